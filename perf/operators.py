"""Measured cases of the block operators: the short causal convolution, the
selective state-space scan and the gated group norm, each forward, backward
(where it trains) and for single tokens.

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true); ``exact`` computes it in float64.

Conventions (channels last everywhere; parameters and scan states are fp32,
activations have the case's type):
  conv   x (B, T, D), w (D, K), bias (D), x0 (B, K-1, D) -> y, xT
  scan   u, delta, z (B, T, D), A (D, N), Bm, Cm (B, T, G, N), skip, delta_bias
         (D), h0 (B, D, N) -> y, hT
  norm   x, z (R, D), w, bias (D), G groups a row -> y
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-5
# Work bounds of the ranges: channel-steps of the convolution and the norm,
# state-steps of the scan (forward; a training pass stores every state in its
# plain form and stays below a quarter of it).
_MAX_ELEMS = 8 * 8192 * 4096
_MAX_STATES = 8 * 4096 * 4096 * 16


def listed():
    conv = dict(op="conv", K=4, silu=True, x0=False, ragged=False)
    scan = dict(op="scan", N=16, G=1, z=False, h0=False, ragged=False)
    norm = dict(op="norm", gate=True, centered=True)
    return [
        # a batch of long prompts, the benchmark's largest (B, T, D)
        dict(conv, name="conv_prompt", kind="fwd", dtype="bf16", B=8, T=8192, D=4096),
        # a training step at a middle size
        dict(conv, name="conv_train", kind="train", dtype="bf16", B=4, T=4096, D=2048),
        # prompts of unequal lengths continued from carried inputs, odd sizes, training in fp32
        dict(conv, name="conv_ragged_train", kind="train", dtype="f32", B=5, T=1037, D=519, K=3, x0=True,
             ragged=True),
        # one token for each of 64 sequences
        dict(conv, name="conv_step", kind="step", dtype="bf16", B=64, D=4096, x0=True),
        # the smallest prompt: latency
        dict(scan, name="scan_small", kind="fwd", dtype="f32", B=1, T=1024, D=64),
        # one long prompt: few channels, many steps
        dict(scan, name="scan_prompt", kind="fwd", dtype="bf16", B=1, T=8192, D=4096, z=True),
        # a batch of prompts, the largest scan
        dict(scan, name="scan_batch", kind="fwd", dtype="bf16", B=8, T=4096, D=4096),
        # prompts of unequal lengths (one empty) from carried states, two groups, odd sizes
        dict(scan, name="scan_ragged", kind="fwd", dtype="f16", B=5, T=777, D=1030, G=2, N=24, z=True, h0=True,
             ragged=True),
        # a training step
        dict(scan, name="scan_train", kind="train", dtype="bf16", B=4, T=4096, D=2048, z=True),
        # one token for each of 64 sequences
        dict(scan, name="scan_step", kind="step", dtype="bf16", B=64, D=4096, z=True, h0=True),
        # a training step of the norm behind the scan
        dict(norm, name="norm_train", kind="train", dtype="bf16", R=4 * 4096, D=4096, G=32),
        # one token for each of 64 sequences
        dict(norm, name="norm_step", kind="fwd", dtype="bf16", R=64, D=4096, G=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op, kind = rng.choice([("conv", "fwd"), ("conv", "train"), ("conv", "step"), ("scan", "fwd"), ("scan", "train"),
                           ("scan", "step"), ("norm", "fwd"), ("norm", "train")])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    odd = rng.random() < 0.5  # any channel count, or one that whole vectors fit

    def channels(lo, hi):
        d = _log_int(rng, lo, hi)
        return d if odd else max(lo, (d + 31) // 32 * 32)

    if op == "norm":
        G = rng.choice([1, 2, 3, 4, 8, 16, 32])
        D = max(1, channels(32, 4096) // G) * G
        R = min(_log_int(rng, 1, 4 * 4096), _MAX_ELEMS // D)
        return dict(op=op, kind=kind, dtype=dtype, R=R, D=D, G=G, gate=rng.random() < 0.6,
                    centered=rng.random() < 0.6)
    if op == "conv":
        case = dict(op=op, kind=kind, dtype=dtype, K=rng.choice([2, 3, 4, 4, 5, 8]), silu=rng.random() < 0.7,
                    x0=rng.random() < 0.5, ragged=False, D=channels(16, 4096))
        if kind == "step":
            case.update(B=_log_int(rng, 1, 256), x0=True)
        else:
            case.update(B=_log_int(rng, 1, 8), T=_log_int(rng, 1, 8192), ragged=rng.random() < 0.4)
        return case
    N = rng.choice([1, 4, 7, 8, 16, 16, 16, 24, 32, 64])
    G = rng.choice([1, 1, 2, 4])
    D = max(1, channels(16, 4096) // G) * G
    case = dict(op=op, kind=kind, dtype=dtype, N=N, G=G, D=D, z=rng.random() < 0.6, h0=rng.random() < 0.5,
                ragged=False)
    if kind == "step":
        case.update(B=_log_int(rng, 1, 256), h0=True)
        return case
    B = _log_int(rng, 1, 8)
    cap = _MAX_STATES if kind == "fwd" else _MAX_STATES // 4
    T = min(_log_int(rng, 1, 8192), max(1, cap // (B * D * N)))
    case.update(B=B, T=T, ragged=rng.random() < 0.4)
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    def lengths(B, T):
        n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        n[0] = T        # the longest prompt fills the batch's rows
        if B > 1:
            n[B - 1] = 0  # a slot without a prompt
        return n

    D = case["D"]
    s = {"case": case}
    train, step = case["kind"] == "train", case["kind"] == "step"
    if case["op"] == "norm":
        R = case["R"]
        s.update(x=normal(R, D, scale=0.7), w=1.0 + normal(D, scale=0.2, to=torch.float32),
                 bias=normal(D, scale=0.2, to=torch.float32) if case["centered"] else None,
                 z=normal(R, D) if case["gate"] else None)
        if train:
            s["dy"] = normal(R, D)
        return s
    B, T = case["B"], case.get("T", 1)
    if case["op"] == "conv":
        K = case["K"]
        s.update(w=normal(D, K, scale=K ** -0.5, to=torch.float32), bias=normal(D, scale=0.1, to=torch.float32),
                 x=normal(B, D) if step else normal(B, T, D),
                 x0=normal(B, K - 1, D) if case["x0"] else None,
                 lengths=lengths(B, T) if case["ragged"] else None)
        if step:
            s["x_out"] = torch.empty_like(s["x0"])
        if train:
            s["dy"] = normal(B, T, D)
        return s
    N, G = case["N"], case["G"]
    # time constants between 10 and 1000 steps: softplus(delta_bias) in [1e-3, 1e-1], A near -(1..N)
    target = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    act = (B, D) if step else (B, T, D)
    shared = (B, G, N) if step else (B, T, G, N)
    s.update(u=normal(*act), delta=normal(*act, scale=0.5),
             A=-uniform(D, N, lo=0.8, hi=1.2) * torch.arange(1, N + 1, device="cuda", dtype=torch.float32),
             Bm=normal(*shared), Cm=normal(*shared), skip=1.0 + normal(D, scale=0.1, to=torch.float32),
             delta_bias=target + torch.log(-torch.expm1(-target)),
             z=normal(*act) if case["z"] else None,
             h0=normal(B, D, N, scale=0.5, to=torch.float32) if case["h0"] else None,
             lengths=lengths(B, T) if case["ragged"] else None)
    if step:
        s["h_out"] = torch.empty_like(s["h0"])
    if train:
        s["dy"] = normal(B, T, D)
    return s


def run(s):
    case = s["case"]
    return (_OWN if own else _PLAIN)[case["op"]](s, case)


# ---------------------------------------------------------------------------
# through the library
# ---------------------------------------------------------------------------

def _own_conv(s, case):
    import linear_recurrence_scans_amd as lrs
    act = "silu" if case["silu"] else None
    if case["kind"] == "step":
        return lrs.mi_causal_conv_step(s["x"], s["w"], s["bias"], s["x0"], act=act, x_out=s["x_out"])
    y, xT = lrs.mi_causal_conv_fwd(s["x"], s["w"], s["bias"], s["x0"], act=act, lengths=s["lengths"])
    if case["kind"] == "fwd":
        return y, xT
    dx, dw, db, dx0 = lrs.mi_causal_conv_bwd(s["x"], s["w"], s["bias"], s["x0"], s["dy"], act=act,
                                             lengths=s["lengths"])
    return [t for t in (y, xT, dx, dw, db, dx0) if t is not None]


def _own_scan(s, case):
    import linear_recurrence_scans_amd as lrs
    args = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"])
    opt = dict(skip=s["skip"], z=s["z"], delta_bias=s["delta_bias"])
    if case["kind"] == "step":
        return lrs.mi_selective_scan_step(*args, s["h0"], **opt, h_out=s["h_out"])
    train = case["kind"] == "train"
    y, hT, states = lrs.mi_selective_scan_fwd(*args, **opt, h0=s["h0"], lengths=s["lengths"], save_states=train)
    if not train:
        return y, hT
    grads = lrs.mi_selective_scan_bwd(*args, states, s["dy"], **opt, h0=s["h0"], lengths=s["lengths"])
    return [t for t in (y, hT) + tuple(grads) if t is not None]


def _own_norm(s, case):
    import linear_recurrence_scans_amd as lrs
    opt = dict(z=s["z"], groups=case["G"], eps=_EPS, centered=case["centered"], act=None if case["gate"] else "silu")
    y = lrs.mi_group_norm_fwd(s["x"], s["w"], s["bias"], **opt)
    if case["kind"] == "fwd":
        return y
    grads = lrs.mi_group_norm_bwd(s["x"], s["w"], s["bias"], s["dy"], **opt)
    return [y] + [t for t in grads if t is not None]


_OWN = {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}


# ---------------------------------------------------------------------------
# plain form: 32-bit torch operations, rounded once at the end
# ---------------------------------------------------------------------------

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _dsilu(x):
    g = 1.0 / (1.0 + torch.exp(-x))
    return g * (1.0 + x * (1.0 - g))


def _valid(lengths, T):
    """(B, T, 1) mask of the steps that exist, or None for all."""
    if lengths is None:
        return None
    return (torch.arange(T, device=lengths.device)[None, :] < lengths[:, None].clamp(0, T))[..., None]


def _plain_conv(s, case):
    dt = _DTYPES[case["dtype"]]
    w, bias, K, D = s["w"], s["bias"], case["K"], case["D"]
    B = case["B"]
    x0 = s["x0"].float() if s["x0"] is not None else torch.zeros(B, K - 1, D, device=w.device)
    if case["kind"] == "step":
        xe = torch.cat([x0, s["x"].float()[:, None]], 1)
        a = bias + sum(xe[:, k] * w[:, k] for k in range(K))
        return (_silu(a) if case["silu"] else a).to(dt), xe[:, 1:].to(dt)
    T = case["T"]
    ok = _valid(s["lengths"], T)
    x = s["x"].float()
    if ok is not None:
        x = torch.where(ok, x, 0.0)
    xe = torch.cat([x0, x], 1)
    a = bias + sum(xe[:, k:k + T] * w[:, k] for k in range(K))
    y = _silu(a) if case["silu"] else a
    end = s["lengths"].clamp(0, T).long() if ok is not None else torch.full((B,), T, device=w.device)
    rows = end[:, None] + torch.arange(K - 1, device=w.device)[None, :]
    xT = torch.gather(xe, 1, rows[..., None].expand(B, K - 1, D)).to(dt)
    if ok is not None:
        y = torch.where(ok, y, 0.0)
    y = y.to(dt)
    if case["kind"] == "fwd":
        return y, xT
    da = s["dy"].float()
    if ok is not None:
        da = torch.where(ok, da, 0.0)
    if case["silu"]:
        da = da * _dsilu(a)
    dxe = torch.zeros_like(xe)
    dw = torch.empty_like(w)
    for k in range(K):
        dxe[:, k:k + T] += da * w[:, k]
        dw[:, k] = (da * xe[:, k:k + T]).sum((0, 1), dtype=torch.float64).float()
    db = da.sum((0, 1), dtype=torch.float64).float()
    dx = dxe[:, K - 1:]
    if ok is not None:
        dx = torch.where(ok, dx, 0.0)
    out = [y, xT, dx.to(dt), dw, db]
    if s["x0"] is not None:
        out.append(dxe[:, :K - 1].to(dt))
    return out


_CHUNK = 32  # steps whose gates the plain scan forms at once


def _plain_scan(s, case):
    dt = _DTYPES[case["dtype"]]
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    step, train = case["kind"] == "step", case["kind"] == "train"
    T = 1 if step else case["T"]
    A, skip = s["A"], s["skip"]
    u = s["u"].float().view(B, T, D)
    raw = s["delta"].float().view(B, T, D) + s["delta_bias"]
    dl = torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    Bm, Cm = s["Bm"].float().view(B, T, G, N), s["Cm"].float().view(B, T, G, N)
    ok = _valid(s.get("lengths"), T)
    if ok is not None:
        u, dl = torch.where(ok, u, 0.0), torch.where(ok, dl, 0.0)
    x = dl * u

    def spread(m):  # (B, L, G, N) -> one row of N for each channel of a group
        return m.repeat_interleave(D // G, dim=2) if G > 1 else m

    h = s["h0"].clone() if s["h0"] is not None else torch.zeros(B, D, N, device=A.device)
    y = torch.empty(B, T, D, device=A.device)
    H = torch.empty(B, T + 1, D, N, device=A.device) if train else None
    if train:
        H[:, 0] = h
    for t0 in range(0, T, _CHUNK):
        t1 = min(T, t0 + _CHUNK)
        a = torch.exp(dl[:, t0:t1, :, None] * A)
        b = x[:, t0:t1, :, None] * spread(Bm[:, t0:t1])
        hs = H[:, t0 + 1:t1 + 1] if train else torch.empty_like(a)
        for t in range(t1 - t0):
            h = torch.addcmul(b[:, t], a[:, t], h)
            hs[:, t] = h
        y[:, t0:t1] = (hs * spread(Cm[:, t0:t1])).sum(-1)
    sk = y + skip * u
    gate = None
    if s["z"] is not None:
        z = s["z"].float().view(B, T, D)
        gate = _silu(z)
    yo = sk if gate is None else sk * gate
    if ok is not None:
        yo = torch.where(ok, yo, 0.0)
    if step:
        return yo.view(B, D).to(dt), h
    yo = yo.to(dt)
    if not train:
        return yo, h
    dy = s["dy"].float()
    if ok is not None:
        dy = torch.where(ok, dy, 0.0)
    dz = None
    ds = dy
    if gate is not None:
        dz = dy * sk * _dsilu(z)
        if ok is not None:
            dz = torch.where(ok, dz, 0.0)
        ds = torch.where(ok, dy * gate, 0.0) if ok is not None else dy * gate
    dBm, dCm = torch.empty_like(Bm), torch.empty_like(Cm)
    dA = torch.zeros(D, N, device=A.device, dtype=torch.float64)
    dxs, ddl = torch.empty_like(x), torch.empty_like(x)
    g = torch.zeros(B, D, N, device=A.device)  # a_{t+1} g_{t+1}
    for t1 in range(T, 0, -_CHUNK):
        t0 = max(0, t1 - _CHUNK)
        a = torch.exp(dl[:, t0:t1, :, None] * A)
        c = ds[:, t0:t1, :, None] * spread(Cm[:, t0:t1])
        gs = torch.empty_like(a)
        for t in range(t1 - t0 - 1, -1, -1):
            torch.add(c[:, t], g, out=gs[:, t])
            g = a[:, t] * gs[:, t]
        dCm[:, t0:t1] = (ds[:, t0:t1, :, None] * H[:, t0 + 1:t1 + 1]).view(B, t1 - t0, G, D // G, N).sum(3)
        dBm[:, t0:t1] = (x[:, t0:t1, :, None] * gs).view(B, t1 - t0, G, D // G, N).sum(3)
        dxs[:, t0:t1] = (gs * spread(Bm[:, t0:t1])).sum(-1)
        q = gs * a * H[:, t0:t1]
        dA += (q * dl[:, t0:t1, :, None]).sum((0, 1), dtype=torch.float64)
        ddl[:, t0:t1] = (q * A).sum(-1)
    ddl = ddl + u * dxs
    draw_ = ddl / (1.0 + torch.exp(-raw))
    du = dl * dxs + skip * ds
    if ok is not None:
        draw_, du = torch.where(ok, draw_, 0.0), torch.where(ok, du, 0.0)
    out = [yo, h, du.to(dt), draw_.to(dt), dA.float(), dBm.to(dt), dCm.to(dt),
           (ds * u).sum((0, 1), dtype=torch.float64).float()]
    if dz is not None:
        out.append(dz.to(dt))
    out.append(draw_.sum((0, 1), dtype=torch.float64).float())
    if s["h0"] is not None:
        out.append(g)
    return out


def _plain_norm(s, case):
    dt = _DTYPES[case["dtype"]]
    R, D, G = case["R"], case["D"], case["G"]
    x = s["x"].float().view(R, G, D // G)
    w, bias = s["w"], s["bias"]
    mean = x.mean(-1, keepdim=True) if case["centered"] else torch.zeros(R, G, 1, device=w.device)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + _EPS)
    xh = xc * rstd
    p = xh.view(R, D) * w
    if bias is not None:
        p = p + bias
    z = s["z"].float() if s["z"] is not None else None
    y = (_silu(p) if z is None else p * _silu(z)).to(dt)
    if case["kind"] == "fwd":
        return y
    dy = s["dy"].float()
    dz = None
    if z is None:
        dp = dy * _dsilu(p)
    else:
        dz = dy * p * _dsilu(z)
        dp = dy * _silu(z)
    dw = (dp * xh.view(R, D)).sum(0, dtype=torch.float64).float()
    dxh = (dp * w).view(R, G, D // G)
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if case["centered"]:
        dx = dx - dxh.mean(-1, keepdim=True)
    out = [y, (dx * rstd).view(R, D).to(dt), dw]
    if bias is not None:
        out.append(dp.sum(0, dtype=torch.float64).float())
    if dz is not None:
        out.append(dz.to(dt))
    return out


_PLAIN = {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}


# ---------------------------------------------------------------------------
# work a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    D = case["D"]
    train, step = case["kind"] == "train", case["kind"] == "step"
    if case["op"] == "norm":
        n = case["R"] * D
        tensors = 2 + case["gate"] + (2 + case["gate"] if train else 0)  # x, y, z; dy, dx, dz
        params = 4 * D * (1 + case["centered"]) * (2 if train else 1)
        return {"bytes": n * e * tensors + params, "flops": n * (12 + (24 if train else 0))}
    B, T = case["B"], case.get("T", 1)
    if case["op"] == "conv":
        K, n = case["K"], case["B"] * T * D
        carried = B * (K - 1) * D * e * (1 + (1 + train) * bool(case["x0"]))  # xT; x0 and its gradient
        params = 4 * D * (K + 1) * (2 if train else 1)
        flops = n * (2 * K + (6 if case["silu"] else 0)) * (3 if train else 1)
        return {"bytes": n * e * (4 if train else 2) + carried + params, "flops": flops}
    N, G, n = case["N"], case["G"], B * T * D
    # u, delta, y; z; dy, du, ddelta; dz
    acts = 3 + case["z"] + (3 + case["z"] if train else 0)
    shared = 2 * B * T * G * N * e * (2 if train else 1)
    states = 4 * B * D * N * (1 + (1 + train) * bool(case["h0"]))
    params = 4 * D * (N + 2) * (2 if train else 1)
    # a state and step: gate (2), update (3), output (2); training: 16 more
    return {"bytes": n * e * acts + shared + states + params,
            "flops": n * (7 * N + 12) + (n * (16 * N + 24) if train else 0)}


# ---------------------------------------------------------------------------
# float64 from the definitions: gradients by differentiation of the forward
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    train = case["kind"] == "train"
    leaves = {"norm": ("x", "w", "bias", "z"), "conv": ("x", "w", "bias", "x0"),
              "scan": ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias", "h0")}[case["op"]]
    d = {k: s[k].double() if s.get(k) is not None else None for k in leaves}
    if train and case["op"] != "scan":
        for k in leaves:
            if d[k] is not None:
                d[k].requires_grad_(True)
    with torch.set_grad_enabled(train):
        if case["op"] == "scan":
            return _exact_scan(s, case, d, leaves)
        if case["op"] == "conv":
            y, xT = _exact_conv(s, case, d)
            outs = [y, xT]
        else:
            y = _exact_norm(case, d)
            outs = [y]
        if not train:
            return tuple(outs) if len(outs) > 1 else outs[0]
        live = [k for k in leaves if d[k] is not None]
        grads = torch.autograd.grad(y, [d[k] for k in live], s["dy"].double())
    return [t.detach() for t in outs] + list(grads)


def _exact_conv(s, case, d):
    B, K, D = case["B"], case["K"], case["D"]
    step = case["kind"] == "step"
    T = 1 if step else case["T"]
    x = d["x"].view(B, T, D)
    n = [T] * B if s.get("lengths") is None else [max(0, min(T, int(v))) for v in s["lengths"].tolist()]
    ys, ends = [], []
    for b in range(B) if s.get("lengths") is not None else [slice(None)]:
        one = isinstance(b, int)
        nb = n[b] if one else T
        xb = x[b:b + 1, :nb] if one else x
        rows = xb.shape[0]
        past = (d["x0"][b:b + 1] if one else d["x0"]) if d["x0"] is not None else xb.new_zeros(rows, K - 1, D)
        xe = torch.cat([past, xb], 1)
        ends.append(xe[:, nb:nb + K - 1])
        # window k of a step holds the input K - 1 - k steps before it
        acc = d["bias"].expand(rows, nb, D)
        for back in range(K):
            acc = acc + xe[:, K - 1 - back:K - 1 - back + nb] * d["w"][:, K - 1 - back]
        if case["silu"]:
            acc = acc * torch.sigmoid(acc)
        ys.append(torch.cat([acc, acc.new_zeros(rows, T - nb, D)], 1))
    y, xT = torch.cat(ys, 0), torch.cat(ends, 0)
    return (y.view(B, D) if step else y), xT


def _exact_norm(case, d):
    R, D, G = case["R"], case["D"], case["G"]
    x = d["x"].view(R, G, D // G)
    if case["centered"]:
        v, m = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
    else:
        m, v = 0.0, x.square().mean(-1, keepdim=True)
    p = ((x - m) / torch.sqrt(v + _EPS)).reshape(R, D) * d["w"]
    if d["bias"] is not None:
        p = p + d["bias"]
    if d["z"] is None:
        return p * torch.sigmoid(p)
    return p * (d["z"] * torch.sigmoid(d["z"]))


def _exact_scan(s, case, d, leaves):
    """Blocks of channels, each by recursive doubling over time."""
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    step, train = case["kind"] == "step", case["kind"] == "train"
    T = 1 if step else case["T"]
    per = D // G
    block = max(1, min(per, (1 << (23 if train else 26)) // (B * T * N)))
    dev = s["A"].device
    keep = None if s.get("lengths") is None else \
        (torch.arange(T, device=dev)[None, :, None] < s["lengths"].view(B, 1, 1))
    y = torch.empty(B, T, D, device=dev, dtype=torch.float64)
    hT = torch.empty(B, D, N, device=dev, dtype=torch.float64)
    grads = {k: torch.zeros_like(d[k]) if d[k] is not None else None for k in leaves}
    last = torch.full((B,), T, device=dev) if keep is None else s["lengths"].clamp(0, T).long()
    for g in range(G):
        for c0 in range(g * per, (g + 1) * per, block):
            ch = slice(c0, min(c0 + block, (g + 1) * per))
            cut = {}
            for k in leaves:
                if d[k] is None:
                    cut[k] = None
                    continue
                t = d[k]
                if k in ("u", "delta", "z"):
                    t = t.view(B, T, D)[..., ch]
                elif k in ("Bm", "Cm"):
                    t = t.view(B, T, G, N)[:, :, g]
                elif k == "h0":
                    t = t[:, ch]
                else:
                    t = t[ch]
                cut[k] = t.detach().clone().requires_grad_(train)
            rate = torch.nn.functional.softplus(cut["delta"] + cut["delta_bias"], threshold=700.0)
            if keep is not None:
                rate = rate * keep
            decay = (rate[..., None] * cut["A"]).exp()                       # (B, T, c, N)
            state = (rate * cut["u"])[..., None] * cut["Bm"][:, :, None, :]
            if cut["h0"] is not None:
                first = state[:, :1] + decay[:, :1] * cut["h0"][:, None]
                state = torch.cat([first, state[:, 1:]], 1)
            hop = 1
            while hop < T:
                state = torch.cat([state[:, :hop], state[:, hop:] + decay[:, hop:] * state[:, :-hop]], 1)
                decay = torch.cat([decay[:, :hop], decay[:, hop:] * decay[:, :-hop]], 1)
                hop *= 2
            out = (state * cut["Cm"][:, :, None, :]).sum(-1) + cut["skip"] * cut["u"]
            if cut["z"] is not None:
                out = out * cut["z"] * torch.sigmoid(cut["z"])
            if keep is not None:
                out = torch.where(keep, out, 0.0)
            y[..., ch] = out.detach()
            # steps past a prompt's end leave its state as it was
            hT[:, ch] = state.detach()[:, -1]
            if train:
                live = [k for k in leaves if cut[k] is not None]
                got = torch.autograd.grad(out, [cut[k] for k in live], s["dy"].double()[..., ch])
                for k, t in zip(live, got):
                    if k in ("u", "delta", "z"):
                        grads[k].view(B, T, D)[..., ch] = t
                    elif k in ("Bm", "Cm"):
                        grads[k].view(B, T, G, N)[:, :, g] += t
                    elif k == "h0":
                        grads[k][:, ch] = t
                    else:
                        grads[k][ch] = t
            del cut, rate, decay, state, out
    if step:
        return y.view(B, D), hT
    if not train:
        return y, hT
    order = ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias", "h0")
    return [y, hT] + [grads[k] for k in order if grads[k] is not None]
