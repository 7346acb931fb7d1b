"""Plain float64 references of the block operators, and their error bounds.

Each reference is the operator's formula, sequential in time, in torch float64 on
the CPU.  With ``absolute=True`` every term enters by its magnitude: the result
is the sum of the magnitudes of an output's terms, the scale its rounding errors
are relative to.

Bounds.  A result is off by at most
    eps(storage)/2 |r|  +  c 2^-24 scale   (+ the grid of fp16's subnormals),
the first for the one rounding on store, the second for c fp32 roundings (half a
step, 2^-24, each) in its longest chain:
  conv   K fused multiply-adds, bias, and 12 for SiLU and its derivative (exp2,
         reciprocal: one step each; products; the argument's own error enters
         times at most 2); sums over B T rows: their number of additions in the
         longest chain, bounded by the number of terms.
  scan   a step multiplies the state by a gate (argument 2 roundings, whose
         effect |x| e^-|x| sums to less than 1 over any run; exp2 one step = 2)
         and adds (1): 4 a step over T steps; 40 for softplus, gates, joins; the
         gradient runs through two such chains.
  norm   two sums of n terms and 16 for the rest.
"""
import torch

F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def bound(r, scale, dtype, c):
    """Elementwise bound for an output stored as `dtype` (see above)."""
    out = half_step(dtype) * r.abs() + c * 2.0 ** -24 * scale
    if dtype == torch.float16:
        out = out + 2.0 ** -25
    # nothing below fp32's normal range is claimed
    return out + 2.0 ** -120


def worst(got, r, scale, dtype, c):
    """Largest error as a fraction of its bound (inf for a non-finite result)."""
    if r.numel() == 0:
        assert tuple(got.shape) == tuple(r.shape)
        return 0.0
    got = got.detach().cpu().to(F64)
    assert tuple(got.shape) == tuple(r.shape), (got.shape, r.shape)
    if not torch.isfinite(got).all():
        return float("inf")
    return float(((got - r).abs() / bound(r, scale, dtype, c)).max())


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x, absolute=False):
    g = torch.sigmoid(x)
    return g * (1 + (x.abs() if absolute else x) * (1 - g))


def _ends(lengths, B, T):
    return [T] * B if lengths is None else [max(0, min(T, int(n))) for n in lengths]


def _a(t, absolute):
    return t.abs() if absolute and t is not None else t


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------

def conv_fwd(x, w, bias=None, x0=None, lengths=None, act=None, absolute=False):
    B, T, D = x.shape
    K = w.shape[1]
    y, xT = torch.zeros(B, T, D, dtype=F64), torch.zeros(B, K - 1, D, dtype=F64)
    for b, n in enumerate(_ends(lengths, B, T)):
        past = x0[b] if x0 is not None else torch.zeros(K - 1, D, dtype=F64)
        xe = torch.cat([past, x[b, :n]], 0)
        xT[b] = xe[n:n + K - 1]
        for t in range(n):
            s = (_a(xe[t:t + K], absolute) * _a(w, absolute).t()).sum(0)
            if bias is not None:
                s = s + _a(bias, absolute)
            if act == "silu" and absolute:
                s = s * 1.1  # |silu'| <= 1.1 and |silu(s)| <= |s|
            elif act == "silu":
                s = silu(s)
            y[b, t] = s
    return y, xT


def conv_bwd(x, w, bias, x0, dy, dxT=None, lengths=None, act=None, absolute=False):
    B, T, D = x.shape
    K = w.shape[1]
    dx, dx0 = torch.zeros(B, T, D, dtype=F64), torch.zeros(B, K - 1, D, dtype=F64)
    dw, db = torch.zeros(D, K, dtype=F64), torch.zeros(D, dtype=F64)
    for b, n in enumerate(_ends(lengths, B, T)):
        past = x0[b] if x0 is not None else torch.zeros(K - 1, D, dtype=F64)
        xe = torch.cat([past, x[b, :n]], 0)
        dxe = torch.zeros(n + K - 1, D, dtype=F64)
        for t in range(n):
            ds = _a(dy[b, t], absolute)
            if act == "silu":
                s = (xe[t:t + K] * w.t()).sum(0) + (bias if bias is not None else 0.0)
                # silu'' is at most 1/2: s's own error, relative to its magnitudes, enters ds times that
                ds = ds * (1.1 + 0.5 * (xe[t:t + K].abs() * w.abs().t()).sum(0) if absolute else dsilu(s))
            db += ds
            dw += (ds[None] * _a(xe[t:t + K], absolute)).t()
            dxe[t:t + K] += ds[None] * _a(w, absolute).t()
        if dxT is not None:
            dxe[n:n + K - 1] += _a(dxT[b], absolute)
        dx0[b], dx[b, :n] = dxe[:K - 1], dxe[K - 1:]
    return dx, dw, db, dx0


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def _rate(delta, delta_bias, softplus):
    raw = delta + (delta_bias if delta_bias is not None else 0.0)
    return (torch.nn.functional.softplus(raw, threshold=500.0), torch.sigmoid(raw)) if softplus else \
        (raw, torch.ones_like(raw))


def scan_fwd(u, delta, A, Bm, Cm, skip=None, z=None, delta_bias=None, h0=None, lengths=None, softplus=True,
             absolute=False):
    """(y, hT, s, H): H[:, t] is the state after t steps, s the output before the gate."""
    B, T, D = u.shape
    N, G = A.shape[1], Bm.shape[2]
    dl, _ = _rate(delta, delta_bias, softplus)
    rep = D // G
    s = torch.zeros(B, T, D, dtype=F64)
    H = torch.zeros(B, T + 1, D, N, dtype=F64)
    ends = _ends(lengths, B, T)
    for b in range(B):
        h = _a(h0[b], absolute) if h0 is not None else torch.zeros(D, N, dtype=F64)
        H[b, 0] = h
        for t in range(ends[b]):
            bt, ct = (_a(m[b, t], absolute).repeat_interleave(rep, 0) for m in (Bm, Cm))
            x = _a(dl[b, t] * u[b, t], absolute)
            h = torch.exp(dl[b, t][:, None] * A) * h + x[:, None] * bt
            H[b, t + 1] = h
            s[b, t] = (ct * h).sum(1)
            if skip is not None:
                s[b, t] += _a(skip * u[b, t], absolute)
        H[b, ends[b] + 1:] = h
    y = s if z is None else s * _a(silu(z), absolute)
    for b in range(B):
        y[b, ends[b]:] = 0
    return y, H[:, T].clone(), s, H


def scan_bwd(u, delta, A, Bm, Cm, dy, dhT=None, skip=None, z=None, delta_bias=None, h0=None, lengths=None,
             softplus=True, absolute=False):
    B, T, D = u.shape
    N, G = A.shape[1], Bm.shape[2]
    rep = D // G
    dl, der = _rate(delta, delta_bias, softplus)
    _, _, s, H = scan_fwd(u, delta, A, Bm, Cm, skip, z, delta_bias, h0, lengths, softplus, absolute)
    du, dd = torch.zeros_like(u), torch.zeros_like(u)
    dz = torch.zeros_like(u) if z is not None else None
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dskip, dbias = torch.zeros(D, dtype=F64), torch.zeros(D, dtype=F64)
    dh0 = torch.zeros(B, D, N, dtype=F64)
    for b, n in enumerate(_ends(lengths, B, T)):
        gam = _a(dhT[b], absolute) if dhT is not None else torch.zeros(D, N, dtype=F64)
        for t in range(n - 1, -1, -1):
            ub, gy = _a(u[b, t], absolute), _a(dy[b, t], absolute)
            bt, ct = (_a(m[b, t], absolute).repeat_interleave(rep, 0) for m in (Bm, Cm))
            ds = gy
            if z is not None:
                ds = gy * _a(silu(z[b, t]), absolute)
                dz[b, t] = gy * s[b, t] * dsilu(z[b, t], absolute)
            x = _a(dl[b, t] * u[b, t], absolute)
            a = torch.exp(dl[b, t][:, None] * A)
            g = ct * ds[:, None] + gam
            gam = a * g
            q = gam * H[b, t]
            dC[b, t] = (ds[:, None] * H[b, t + 1]).view(G, rep, N).sum(1)
            dB[b, t] = (g * x[:, None]).view(G, rep, N).sum(1)
            dx = (g * bt).sum(1)
            dA += q * _a(dl[b, t], absolute)[:, None]
            dd[b, t] = ((q * _a(A, absolute)).sum(1) + ub * dx) * der[b, t]
            du[b, t] = _a(dl[b, t], absolute) * dx
            if skip is not None:
                du[b, t] += _a(skip, absolute) * ds
            dskip += ds * ub
            dbias += dd[b, t]
        dh0[b] = gam
    return du, dd, dA, dB, dC, dskip, dz, dbias, dh0


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def norm_fwd(x, w=None, bias=None, z=None, groups=1, eps=1e-5, centered=True, act=None):
    R, D = x.shape
    xg = x.view(R, groups, D // groups)
    xc = xg - xg.mean(-1, keepdim=True) if centered else xg
    xh = (xc / torch.sqrt(xc.square().mean(-1, keepdim=True) + eps)).reshape(R, D)
    p = xh * w if w is not None else xh
    if bias is not None:
        p = p + bias
    return silu(p) if act == "silu" else p * silu(z) if z is not None else p


def norm_bwd(x, w, bias, dy, z=None, groups=1, eps=1e-5, centered=True, act=None):
    R, D = x.shape
    n = D // groups
    xg = x.view(R, groups, n)
    xc = xg - xg.mean(-1, keepdim=True) if centered else xg
    rstd = 1 / torch.sqrt(xc.square().mean(-1, keepdim=True) + eps)
    xh = (xc * rstd).reshape(R, D)
    p = xh * (w if w is not None else 1.0) + (bias if bias is not None else 0.0)
    dz = dy * p * dsilu(z) if z is not None else None
    dp = dy * dsilu(p) if act == "silu" else dy * silu(z) if z is not None else dy
    dxh = (dp * (w if w is not None else 1.0)).view(R, groups, n)
    xhg = xh.view(R, groups, n)
    dx = dxh - xhg * (dxh * xhg).mean(-1, keepdim=True)
    if centered:
        dx = dx - dxh.mean(-1, keepdim=True)
    return (dx * rstd).reshape(R, D), (dp * xh).sum(0), dp.sum(0), dz
