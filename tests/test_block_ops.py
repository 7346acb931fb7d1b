"""Block operators (causal convolution, selective scan, group norm): the
references against differences, the refusals, and the GPU results against the
references within the bounds of tests/block_ref.py."""
import itertools
import sys

import pytest
import torch

import block_ref as R
import linear_recurrence_scans_amd as lrs

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
(MI_OK, MI_ERR_INVALID_ARG, MI_ERR_UNSUPPORTED, MI_ERR_WORKSPACE) = range(4)
P, STEP = 1 << 20, 1 << 30  # fake device addresses, far apart; never dereferenced

gpu = pytest.mark.gpu


def say(*args):
    print("[case]", *args, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def quant(t, dtype):
    """The values an input of this type really holds, in float64."""
    return None if t is None else t.to(dtype).to(torch.float64)


def dev(t, dtype):
    return None if t is None else t.to(dtype).cuda()


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def conv_inputs(B, T, D, K, dtype, seed, bias=True, x0=True, lengths=None):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    d = dict(x=quant(n(B, T, D), dtype), w=quant(n(D, K) * K ** -0.5, F32), bias=quant(n(D) * 0.3, F32) if bias else None,
             x0=quant(n(B, K - 1, D), dtype) if x0 else None, dy=quant(n(B, T, D), dtype),
             dxT=quant(n(B, K - 1, D), dtype))
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return d


def scan_inputs(B, T, D, G, N, dtype, seed, skip=True, z=True, bias=True, h0=True, lengths=None):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    r = lambda *s: torch.rand(*s, generator=g, dtype=torch.float64)
    target = torch.exp(r(D) * 4.6 - 6.9)  # rates of 1e-3 to 1e-1
    d = dict(u=quant(n(B, T, D), dtype), delta=quant(n(B, T, D) * 0.5 + (0 if bias else -3.0), dtype),
             A=quant(-(0.8 + 0.4 * r(D, N)) * torch.arange(1, N + 1, dtype=torch.float64), F32),
             Bm=quant(n(B, T, G, N), dtype), Cm=quant(n(B, T, G, N), dtype),
             skip=quant(1 + 0.1 * n(D), F32) if skip else None, z=quant(n(B, T, D), dtype) if z else None,
             delta_bias=quant(target + torch.log(-torch.expm1(-target)), F32) if bias else None,
             h0=quant(n(B, D, N) * 0.5, F32) if h0 else None, dy=quant(n(B, T, D), dtype),
             dhT=quant(n(B, D, N), F32))
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return d


def norm_inputs(rows, D, dtype, seed, w=True, bias=True, z=False, mean=0.0):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    return dict(x=quant(n(rows, D) * 0.7 + mean, dtype), w=quant(1 + 0.2 * n(D), F32) if w else None,
                bias=quant(0.2 * n(D), F32) if bias else None, z=quant(n(rows, D), dtype) if z else None,
                dy=quant(n(rows, D), dtype))


# ---------------------------------------------------------------------------
# the references: gradients against differences (CPU)
# ---------------------------------------------------------------------------

def _differences(f, x, grads):
    """Central differences of the scalar f(**x) along random directions."""
    g = gen(99)
    for name, grad in grads.items():
        v = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        e = 1e-6
        up, dn = f(**{**x, name: x[name] + e * v}), f(**{**x, name: x[name] - e * v})
        want, got = float(up - dn) / (2 * e), float((grad * v).sum())
        assert abs(got - want) <= 1e-6 * (abs(want) + float((grad * v).abs().sum())) + 1e-9, (name, got, want)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("K,lengths", [(4, None), (3, [5, 0, 1]), (1, [2, 5, 0])])
def test_conv_reference_gradient_is_the_difference(K, lengths, act):
    d = conv_inputs(3, 5, 4, K, torch.float64, 1, lengths=lengths)
    ln, dy, dxT = d.pop("lengths"), d.pop("dy"), d.pop("dxT")

    def f(x, w, bias, x0):
        y, xT = R.conv_fwd(x, w, bias, x0, ln, act)
        return (y * dy).sum() + (xT * dxT).sum()

    dx, dw, db, dx0 = R.conv_bwd(d["x"], d["w"], d["bias"], d["x0"], dy, dxT, ln, act)
    grads = dict(x=dx, w=dw, bias=db)
    if K > 1:
        grads["x0"] = dx0
    _differences(f, d, grads)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("G,N,lengths", [(1, 3, None), (2, 4, [6, 0, 1])])
def test_scan_reference_gradient_is_the_difference(G, N, lengths, softplus):
    d = scan_inputs(3, 6, 4, G, N, torch.float64, 2, lengths=lengths)
    ln, dy, dhT = d.pop("lengths"), d.pop("dy"), d.pop("dhT")
    if not softplus:
        d["delta"], d["delta_bias"] = d["delta"].abs() * 0.1, d["delta_bias"].abs() * 0.01

    def f(u, delta, A, Bm, Cm, skip, z, delta_bias, h0):
        y, hT, _, _ = R.scan_fwd(u, delta, A, Bm, Cm, skip, z, delta_bias, h0, ln, softplus)
        return (y * dy).sum() + (hT * dhT).sum()

    names = ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias", "h0")
    got = R.scan_bwd(d["u"], d["delta"], d["A"], d["Bm"], d["Cm"], dy, dhT, d["skip"], d["z"], d["delta_bias"],
                     d["h0"], ln, softplus)
    _differences(f, d, dict(zip(names, got)))


@pytest.mark.parametrize("centered,act,z", [(True, None, True), (True, "silu", False), (False, None, False),
                                            (False, None, True)])
def test_norm_reference_gradient_is_the_difference(centered, act, z):
    d = norm_inputs(5, 12, torch.float64, 3, z=z)
    dy = d.pop("dy")
    opt = dict(groups=3, eps=1e-5, centered=centered, act=act)

    def f(x, w, bias, z):
        return (R.norm_fwd(x, w, bias, z, **opt) * dy).sum()

    dx, dw, db, dz = R.norm_bwd(d["x"], d["w"], d["bias"], dy, d["z"], **opt)
    grads = dict(x=dx, w=dw, bias=db)
    if z:
        grads["z"] = dz
    _differences(f, d, grads)


# ---------------------------------------------------------------------------
# refusals (CPU: nothing is launched)
# ---------------------------------------------------------------------------

def ptrs(n):
    return [P + i * STEP for i in range(n)]


BIG = 1 << 40


def test_conv_refusals():
    L = lrs._load()
    x, w, b, x0, ln, y, xT, dy, dxT, dx, dw, db, dx0, ws = ptrs(14)

    def fwd(x=x, w=w, b=b, x0=x0, ln=ln, y=y, xT=xT, sz=(2, 8, 16, 4), act=1, dt=0):
        return L.mi_causal_conv_fwd(x, w, b, x0, ln, y, xT, *sz, act, dt, None)

    assert fwd(sz=(-1, 8, 16, 4)) == MI_ERR_INVALID_ARG
    assert fwd(sz=(2, 8, 16, 0)) == MI_ERR_UNSUPPORTED
    assert fwd(sz=(2, 8, 16, 9)) == MI_ERR_UNSUPPORTED
    assert fwd(act=2) == MI_ERR_UNSUPPORTED
    assert fwd(dt=3) == MI_ERR_UNSUPPORTED
    assert fwd(x=None) == MI_ERR_INVALID_ARG
    assert fwd(w=None) == MI_ERR_INVALID_ARG
    assert fwd(y=None) == MI_ERR_INVALID_ARG
    assert fwd(x=x + 2) == MI_ERR_INVALID_ARG      # misaligned float
    assert fwd(ln=ln + 1) == MI_ERR_INVALID_ARG
    assert fwd(y=x) == MI_ERR_INVALID_ARG          # output on its input
    assert fwd(xT=x0) == MI_ERR_INVALID_ARG
    assert fwd(xT=y + 16) == MI_ERR_INVALID_ARG    # outputs on each other
    assert fwd(sz=(1 << 40, 1 << 20, 1 << 10, 4)) == MI_ERR_INVALID_ARG  # size overflow
    assert fwd(x=None, y=None, w=None, xT=None, sz=(0, 8, 16, 4)) == MI_OK
    assert fwd(sz=(2, 8, 0, 4)) == MI_OK

    def bwd(dx=dx, dw=dw, db=db, dx0=dx0, ws=ws, wsb=BIG, dy=dy, sz=(2, 8, 16, 4), dt=0):
        return L.mi_causal_conv_bwd(x, w, b, x0, ln, dy, dxT, dx, dw, db, dx0, *sz, 1, dt, ws, wsb, None)

    need = L.mi_causal_conv_bwd_workspace(2, 8, 16, 4, 0)
    assert need > 0
    assert bwd(ws=None) == MI_ERR_WORKSPACE
    assert bwd(wsb=need - 1) == MI_ERR_WORKSPACE
    assert bwd(ws=ws + 64) == MI_ERR_INVALID_ARG
    assert bwd(dw=None) == MI_ERR_INVALID_ARG
    assert bwd(dy=None) == MI_ERR_INVALID_ARG
    assert bwd(dx=dy) == MI_ERR_INVALID_ARG
    assert bwd(db=dw) == MI_ERR_INVALID_ARG
    assert bwd(ws=x) == MI_ERR_INVALID_ARG
    assert bwd(sz=(2, 8, 16, 9)) == MI_ERR_UNSUPPORTED

    def step(x0=x0, y=y, xo=xT, sz=(2, 16, 4)):
        return L.mi_causal_conv_step(x, w, b, x0, y, xo, *sz, 0, 0, None)

    assert step(x0=None) == MI_ERR_INVALID_ARG
    assert step(xo=None) == MI_ERR_INVALID_ARG
    assert step(xo=x0 + 16) == MI_ERR_INVALID_ARG  # neither in place nor apart
    assert step(y=x0) == MI_ERR_INVALID_ARG
    assert step(sz=(0, 16, 4)) == MI_OK


def test_scan_refusals():
    L = lrs._load()
    (u, delta, A, Bm, Cm, skip, z, db, h0, ln, y, hT, st, dy, dhT, du, dd, dA, dB, dC, dsk, dz, ddb, dh0,
     ws) = ptrs(25)

    def fwd(u=u, delta=delta, A=A, Bm=Bm, Cm=Cm, y=y, hT=hT, st=st, sz=(2, 8, 16, 2, 4), dt=0, h0=h0,
            wsp=ws, wsb=BIG):
        return L.mi_selective_scan_fwd(u, delta, A, Bm, Cm, skip, z, db, h0, ln, y, hT, st, *sz, 1, dt, wsp, wsb, None)

    assert fwd(sz=(2, 8, 16, 2, 0)) == MI_ERR_UNSUPPORTED
    assert fwd(sz=(2, 8, 16, 2, 65)) == MI_ERR_UNSUPPORTED
    assert fwd(sz=(2, 8, 16, 3, 4)) == MI_ERR_INVALID_ARG   # groups do not divide the channels
    assert fwd(sz=(2, 8, 16, 0, 4)) == MI_ERR_INVALID_ARG
    assert fwd(sz=(2, -8, 16, 2, 4)) == MI_ERR_INVALID_ARG
    assert fwd(dt=5) == MI_ERR_UNSUPPORTED
    for k in ("u", "delta", "A", "Bm", "Cm", "y"):
        assert fwd(**{k: None}) == MI_ERR_INVALID_ARG, k
    assert fwd(A=A + 2) == MI_ERR_INVALID_ARG
    assert fwd(hT=h0) == MI_ERR_INVALID_ARG
    assert fwd(st=hT) == MI_ERR_INVALID_ARG
    assert fwd(y=z) == MI_ERR_INVALID_ARG
    assert fwd(sz=(0, 8, 16, 2, 4), u=None, y=None) == MI_OK
    assert fwd(sz=(1 << 40, 1 << 20, 1 << 10, 1, 4)) == MI_ERR_INVALID_ARG
    long = (1, 4096, 16, 1, 16)  # one channel tile: segments of the sequence
    need = L.mi_selective_scan_fwd_workspace(*long, 0)
    assert need > 0
    assert fwd(sz=long, wsp=None) == MI_ERR_WORKSPACE
    assert fwd(sz=long, wsb=need - 1) == MI_ERR_WORKSPACE
    assert fwd(sz=long, wsp=u) == MI_ERR_INVALID_ARG
    assert fwd(sz=long, wsp=ws + 4) == MI_ERR_INVALID_ARG
    for N in range(1, 65):
        assert L.mi_selective_scan_block(N) > 0
    assert L.mi_selective_scan_block(0) == 0 and L.mi_selective_scan_block(65) == 0

    def bwd(skip=skip, dsk=dsk, z=z, dz=dz, db=db, ddb=ddb, st=st, ws=ws, wsb=BIG, du=du, sz=(2, 8, 16, 2, 4)):
        return L.mi_selective_scan_bwd(u, delta, A, Bm, Cm, skip, z, db, st, ln, dy, dhT, du, dd, dA, dB, dC, dsk, dz,
                                       ddb, dh0, *sz, 1, 0, ws, wsb, None)

    need = L.mi_selective_scan_bwd_workspace(2, 8, 16, 2, 4, 0)
    assert need > 0
    assert bwd(ws=None) == MI_ERR_WORKSPACE
    assert bwd(wsb=need - 1) == MI_ERR_WORKSPACE
    assert bwd(dsk=None) == MI_ERR_INVALID_ARG   # gradients go with their inputs
    assert bwd(z=None) == MI_ERR_INVALID_ARG
    assert bwd(ddb=None) == MI_ERR_INVALID_ARG
    assert bwd(st=None) == MI_ERR_INVALID_ARG
    assert bwd(du=u) == MI_ERR_INVALID_ARG
    assert bwd(ws=u) == MI_ERR_INVALID_ARG
    assert bwd(sz=(2, 8, 16, 2, 65)) == MI_ERR_UNSUPPORTED

    def step(h=h0, ho=hT, sz=(2, 16, 2, 4)):
        return L.mi_selective_scan_step(u, delta, A, Bm, Cm, h, skip, z, db, y, ho, *sz, 1, 0, None)

    assert step(h=None) == MI_ERR_INVALID_ARG
    assert step(ho=h0 + 64) == MI_ERR_INVALID_ARG
    assert step(sz=(2, 16, 2, 65)) == MI_ERR_UNSUPPORTED
    assert step(sz=(2, 0, 2, 4)) == MI_OK


def test_norm_refusals():
    L = lrs._load()
    x, w, b, z, y, dy, dx, dw, db, dz, ws = ptrs(11)

    def fwd(x=x, z=z, y=y, sz=(8, 16, 4), eps=1e-5, act=0, dt=0):
        return L.mi_group_norm_fwd(x, w, b, z, y, *sz, eps, 1, act, dt, None)

    assert fwd(sz=(8, 16, 3)) == MI_ERR_INVALID_ARG
    assert fwd(sz=(8, 16, 0)) == MI_ERR_INVALID_ARG
    assert fwd(sz=(-8, 16, 4)) == MI_ERR_INVALID_ARG
    assert fwd(eps=-1.0) == MI_ERR_INVALID_ARG
    assert fwd(eps=float("nan")) == MI_ERR_INVALID_ARG
    assert fwd(act=1) == MI_ERR_INVALID_ARG          # an activation and a gate
    assert fwd(act=7) == MI_ERR_UNSUPPORTED
    assert fwd(dt=9) == MI_ERR_UNSUPPORTED
    assert fwd(x=None) == MI_ERR_INVALID_ARG
    assert fwd(y=x) == MI_ERR_INVALID_ARG
    assert fwd(sz=(0, 16, 4), x=None, y=None) == MI_OK

    def bwd(dw=dw, dz=dz, dx=dx, ws=ws, wsb=BIG):
        return L.mi_group_norm_bwd(x, w, b, z, dy, dx, dw, db, dz, 8, 16, 4, 1e-5, 1, 0, 0, ws, wsb, None)

    need = L.mi_group_norm_bwd_workspace(8, 16, 4, 0)
    assert need > 0
    assert bwd(ws=None) == MI_ERR_WORKSPACE
    assert bwd(wsb=need - 1) == MI_ERR_WORKSPACE
    assert bwd(dw=None) == MI_ERR_INVALID_ARG
    assert bwd(dz=None) == MI_ERR_INVALID_ARG
    assert bwd(dx=dy) == MI_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors_of_the_block_operators():
    x = torch.rand(1, 4, 4)
    with pytest.raises(ValueError, match="GPU"):
        lrs.mi_causal_conv_fwd(x, torch.rand(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        lrs.mi_selective_scan_fwd(x, x, torch.rand(4, 2), x, x)
    with pytest.raises(ValueError, match="GPU"):
        lrs.mi_group_norm_fwd(x)


# ---------------------------------------------------------------------------
# GPU: causal convolution
# ---------------------------------------------------------------------------

def poison(t, lengths):
    """NaN in the steps past each length."""
    if lengths is None:
        return t
    t = t.clone()
    for b, n in enumerate(lengths):
        t[b, max(0, int(n)):] = float("nan")
    return t


def _len(d):
    return None if d["lengths"] is None else d["lengths"].cuda()


def check_conv(B, T, D, K, dtype, act, seed, **kw):
    say("conv", (B, T, D, K), dtype, act, kw)
    d = conv_inputs(B, T, D, K, dtype, seed, **kw)
    ln = d["lengths"]
    x, dy = dev(poison(d["x"], ln), dtype), dev(poison(d["dy"], ln), dtype)
    w, bias, x0, dxT = dev(d["w"], F32), dev(d["bias"], F32), dev(d["x0"], dtype), dev(d["dxT"], dtype)
    y, xT = lrs.mi_causal_conv_fwd(x, w, bias, x0, act=act, lengths=_len(d))
    ry, rxT = R.conv_fwd(d["x"], d["w"], d["bias"], d["x0"], ln, act)
    sy, _ = R.conv_fwd(d["x"], d["w"], d["bias"], d["x0"], ln, act, absolute=True)
    e = {"y": R.worst(y, ry, sy, dtype, K + 13)}
    assert torch.equal(xT.cpu().double(), rxT)
    got = lrs.mi_causal_conv_bwd(x, w, bias, x0, dy, dxT, act=act, lengths=_len(d))
    args = (d["x"], d["w"], d["bias"], d["x0"], d["dy"], d["dxT"], ln, act)
    ref, sc = R.conv_bwd(*args), R.conv_bwd(*args, absolute=True)
    c = 2 * K + 26
    for name, gt, r, s, t in zip(("dx", "dw", "dbias", "dx0"), got, ref, sc, (dtype, F32, F32, dtype)):
        if gt is not None:
            e[name] = R.worst(gt, r, s, t, c + (B * T if t is F32 and name in ("dw", "dbias") else 0))
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_widths(K, dtype):
    check_conv(2, 37, 40, K, dtype, "silu", K, lengths=[37, 20])


@gpu
@pytest.mark.parametrize("T", [0, 1, 2, 3, 15, 16, 17, 63, 64, 65, 130, 300])
def test_conv_lengths(T):
    check_conv(2, T, 24, 4, BF16, None, T)
    check_conv(3, T, 8, 3, F32, "silu", T, lengths=[T, 0, min(T, 1)], bias=False, x0=False)


@gpu
@pytest.mark.parametrize("D", [1, 2, 3, 4, 7, 8, 63, 64, 100, 257, 520])
def test_conv_channels(D):
    check_conv(1, 20, D, 4, F16, "silu", D)
    check_conv(2, 20, D, 4, F32, None, D, x0=False)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D", [2, 6, 70, 126, 130, 258])
def test_conv_pairs(D, dtype):
    """Even widths that hold no whole 8-byte vectors in 16-bit types, and their steps."""
    check_conv(2, 70, D, 4, dtype, "silu", D, lengths=[70, 33])
    d = conv_inputs(3, 5, D, 4, dtype, D)
    x, w, b = dev(d["x"], dtype), dev(d["w"], F32), dev(d["bias"], F32)
    y, xT = lrs.mi_causal_conv_fwd(x, w, b, act="silu")
    st = torch.zeros(3, 3, D, dtype=dtype, device="cuda")
    for t in range(5):
        yt, st = lrs.mi_causal_conv_step(x[:, t], w, b, st, act="silu")
        assert torch.equal(yt, y[:, t])
    assert torch.equal(st, xT)


@gpu
def test_conv_continues_and_steps():
    """Pieces and single steps give the whole's results, and the same carried inputs."""
    say("conv pieces and steps B=3 T=29 D=72 K=4 bf16")
    d = conv_inputs(3, 29, 72, 4, BF16, 5)
    x, w, b = dev(d["x"], BF16), dev(d["w"], F32), dev(d["bias"], F32)
    y, xT = lrs.mi_causal_conv_fwd(x, w, b, act="silu")
    y1, c1 = lrs.mi_causal_conv_fwd(x[:, :11], w, b, act="silu")
    y2, c2 = lrs.mi_causal_conv_fwd(x[:, 11:], w, b, c1, act="silu")
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(c2, xT)
    st = torch.zeros(3, 3, 72, dtype=BF16, device="cuda")
    for t in range(29):
        yt, out = lrs.mi_causal_conv_step(x[:, t], w, b, st, act="silu", x_out=st)
        assert out is st
        assert torch.equal(yt, y[:, t]), t
    assert torch.equal(st, xT)


# ---------------------------------------------------------------------------
# GPU: selective scan
# ---------------------------------------------------------------------------

NAMES = ("u", "delta", "A", "Bm", "Cm", "skip", "z", "delta_bias", "h0")


def check_scan(B, T, D, G, N, dtype, seed, softplus=True, **kw):
    say("scan", (B, T, D, G, N), dtype, kw)
    d = scan_inputs(B, T, D, G, N, dtype, seed, **kw)
    if not softplus:
        d["delta"], d["delta_bias"] = quant(d["delta"].abs() * 0.05, dtype), None
    ln = d["lengths"]
    acts = {k: dev(poison(d[k], ln) if d[k] is not None else None, dtype)
            for k in ("u", "delta", "z", "Bm", "Cm", "dy")}
    par = {k: dev(d[k], F32) for k in ("A", "skip", "delta_bias", "h0", "dhT")}
    args = (acts["u"], acts["delta"], par["A"], acts["Bm"], acts["Cm"])
    opt = dict(skip=par["skip"], z=acts["z"], delta_bias=par["delta_bias"], h0=par["h0"], lengths=_len(d),
               softplus=softplus)
    y, hT, st = lrs.mi_selective_scan_fwd(*args, **opt, save_states=True)
    rin = [d[k] for k in ("u", "delta", "A", "Bm", "Cm")]
    ropt = dict(skip=d["skip"], z=d["z"], delta_bias=d["delta_bias"], h0=d["h0"], lengths=ln, softplus=softplus)
    ry, rh, _, H = R.scan_fwd(*rin, **ropt)
    sy, sh, _, SH = R.scan_fwd(*rin, **ropt, absolute=True)
    c = 4 * T + 40 + N
    e = {"y": R.worst(y, ry, sy, dtype, c), "hT": R.worst(hT, rh, sh, F32, c)}
    blk = lrs.mi_selective_scan_block(N)
    e["states"] = R.worst(st, H[:, :T:blk] if T else H[:, :0], SH[:, :T:blk] if T else SH[:, :0], F32, c)
    got = lrs.mi_selective_scan_bwd(*args, st, acts["dy"], par["dhT"], **opt)
    ref = R.scan_bwd(*rin, d["dy"], d["dhT"], **ropt)
    sc = R.scan_bwd(*rin, d["dy"], d["dhT"], **ropt, absolute=True)
    types = (dtype, dtype, F32, dtype, dtype, F32, dtype, F32, F32)
    extra = dict(A=B * T, Bm=D, Cm=D, skip=B * T, delta_bias=B * T)
    for name, gt, r, s, t in zip(NAMES, got, ref, sc, types):
        assert (gt is None) == (d[name] is None), name
        if gt is not None:
            e["d" + name] = R.worst(gt, r, s, t, 2 * c + 40 + extra.get(name, 0))
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 12, 16, 17, 32, 33, 64])
def test_scan_states(N, dtype):
    check_scan(2, 35, 20, 1, N, dtype, N, lengths=[35, 17])


@gpu
@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 31, 63, 64, 65, 128, 129, 150])
def test_scan_lengths(T):
    check_scan(2, T, 34, 1, 16, F32, T)
    check_scan(3, T, 12, 2, 4, BF16, T, lengths=[T, 0, min(T, 1)], h0=False, z=False)


@gpu
@pytest.mark.parametrize("D,G", [(1, 1), (2, 2), (3, 1), (16, 1), (31, 1), (32, 1), (33, 1), (66, 2), (70, 5),
                                 (96, 3), (130, 1)])
def test_scan_channels(D, G):
    check_scan(2, 21, D, G, 16, BF16, D, skip=False)
    check_scan(1, 21, D, G, 20, F32, D, bias=False)


@gpu
def test_scan_without_softplus():
    check_scan(2, 40, 24, 1, 16, F32, 7, softplus=False)


@gpu
def test_scan_bad_lengths_are_clamped():
    say("scan lengths outside [0, T]")
    check_scan(3, 20, 8, 1, 4, F32, 8, lengths=[-5, 1000, 20])


@gpu
def test_scan_extreme_rates():
    """Gates that underflow to zero and gates of exactly one."""
    say("scan extreme rates")
    d = scan_inputs(1, 70, 16, 1, 16, F32, 9)
    d["delta"][:, ::3] = 40.0    # softplus = x: exp(-40 n) vanishes
    d["delta"][:, 1::3] = -200.0  # rate 0: the state stays
    a = {k: dev(v, F32) for k, v in d.items() if v is not None and k != "lengths"}
    y, hT, st = lrs.mi_selective_scan_fwd(*(a[k] for k in NAMES[:5]), *(a[k] for k in NAMES[5:]), save_states=True)
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin)
    sy, sh, _, _ = R.scan_fwd(*rin, absolute=True)
    # a rate of 40 and A of -19 put the gate's argument near 800: its roundings count |argument|
    e = {"y": R.worst(y, ry, sy, F32, 400), "hT": R.worst(hT, rh, sh, F32, 400)}
    got = lrs.mi_selective_scan_bwd(*(a[k] for k in NAMES[:5]), st, a["dy"], a["dhT"], a["skip"], a["z"],
                                    a["delta_bias"], a["h0"])
    assert all(bool(torch.isfinite(t).all()) for t in got)
    print(e)
    assert max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,G,N", [(40, 1, 16), (33, 3, 7), (20, 2, 64), (5, 1, 1), (64, 1, 18)])
def test_scan_step(D, G, N, dtype):
    say("scan step", (D, G, N), dtype)
    d = scan_inputs(3, 6, D, G, N, dtype, D + N)
    acts = {k: dev(d[k], dtype) for k in ("u", "delta", "z", "Bm", "Cm")}
    par = {k: dev(d[k], F32) for k in ("A", "skip", "delta_bias", "h0")}
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin)
    sy, sh, _, _ = R.scan_fwd(*rin, absolute=True)
    h, ys = par["h0"].clone(), []
    for t in range(6):
        args = [acts[k][:, t] for k in ("u", "delta")] + [par["A"]] + [acts[k][:, t] for k in ("Bm", "Cm")]
        y, out = lrs.mi_selective_scan_step(*args, h, par["skip"], acts["z"][:, t], par["delta_bias"], h_out=h)
        assert out is h
        ys.append(y)
    e = {"y": R.worst(torch.stack(ys, 1), ry, sy, dtype, 4 * 6 + 40 + N), "h": R.worst(h, rh, sh, F32, 64 + N)}
    keep = par["h0"].clone()
    y1, h1 = lrs.mi_selective_scan_step(acts["u"][:, 0], acts["delta"][:, 0], par["A"], acts["Bm"][:, 0],
                                        acts["Cm"][:, 0], par["h0"])
    assert torch.equal(keep, par["h0"]) and h1 is not par["h0"]
    print(e)
    assert max(e.values()) <= 1.0, e


@gpu
def test_scan_continues_from_its_state():
    say("scan pieces B=2 T=300 D=48 N=16")
    d = scan_inputs(2, 300, 48, 1, 16, F32, 11)
    a = {k: dev(v, F32) for k, v in d.items() if v is not None}
    cut = lambda s: [a[k][:, s] if k in ("u", "delta", "Bm", "Cm") else a[k] for k in NAMES[:5]]
    rest = lambda s, h: dict(skip=a["skip"], z=a["z"][:, s], delta_bias=a["delta_bias"], h0=h)
    one, two, whole = slice(0, 117), slice(117, 300), slice(0, 300)
    y, hT, _ = lrs.mi_selective_scan_fwd(*cut(whole), **rest(whole, a["h0"]))
    y1, h1, _ = lrs.mi_selective_scan_fwd(*cut(one), **rest(one, a["h0"]))
    y2, h2, _ = lrs.mi_selective_scan_fwd(*cut(two), **rest(two, h1))
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin)
    sy, sh, _, _ = R.scan_fwd(*rin, absolute=True)
    for g, r, s in ((y, ry, sy), (torch.cat([y1, y2], 1), ry, sy), (hT, rh, sh), (h2, rh, sh)):
        assert R.worst(g, r, s, F32, 4 * 300 + 56) <= 1.0


# ---------------------------------------------------------------------------
# GPU: group norm
# ---------------------------------------------------------------------------

def check_norm(rows, D, G, dtype, seed, centered=True, act=None, eps=1e-5, **kw):
    say("norm", (rows, D, G), dtype, centered, act, kw)
    d = norm_inputs(rows, D, dtype, seed, **kw)
    t = {k: dev(d[k], F32 if k in ("w", "bias") else dtype) for k in d}
    opt = dict(groups=G, eps=eps, centered=centered, act=act)
    y = lrs.mi_group_norm_fwd(t["x"], t["w"], t["bias"], t["z"], **opt)
    ry = R.norm_fwd(d["x"], d["w"], d["bias"], d["z"], **opt)
    n = D // G
    # magnitudes: xh is off by (n + 16) roundings relative to |x| / std (the mean's
    # terms do not shrink with x - mean) and to itself; everything else multiplies it
    xg = d["x"].view(rows, G, n)
    xc = xg - xg.mean(-1, keepdim=True) if centered else xg
    rstd = 1 / torch.sqrt(xc.square().mean(-1, keepdim=True) + eps)
    mag = ((xg.abs() + (xg.abs().mean(-1, keepdim=True) if centered else 0)) * rstd).reshape(rows, D)
    aw = d["w"].abs() if d["w"] is not None else torch.ones(D, dtype=torch.float64)
    ap = mag * aw + (d["bias"].abs() if d["bias"] is not None else 0)
    gate = R.silu(d["z"]).abs() if d["z"] is not None else 1.1
    c = 2 * n + 40
    e = {"y": R.worst(y, ry, ap * gate, dtype, c)}
    got = lrs.mi_group_norm_bwd(t["x"], t["w"], t["bias"], t["dy"], t["z"], **opt)
    ref = R.norm_bwd(d["x"], d["w"], d["bias"], d["dy"], d["z"], **opt)
    # dp: silu'' <= 1/2 lets p's error into dp
    dp = d["dy"].abs() * (1.1 + 0.5 * ap if act else gate)
    dxh = (dp * aw).view(rows, G, n)
    mg = mag.view(rows, G, n)
    sx = ((dxh + mg * (dxh * mg).mean(-1, keepdim=True) * 3 + dxh.mean(-1, keepdim=True)) * rstd).reshape(rows, D)
    scales = (sx, (dp * mag).sum(0), dp.sum(0),
              d["dy"].abs() * ap * R.dsilu(d["z"], absolute=True) if d["z"] is not None else None)
    for name, gt, r, s, ty in zip(("dx", "dw", "dbias", "dz"), got, ref, scales, (dtype, F32, F32, dtype)):
        if gt is not None:
            e[name] = R.worst(gt, r, s, ty, 2 * c + (rows if ty is F32 and name in ("dw", "dbias") else 0))
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,G", [(1, 1), (8, 8), (8, 1), (16, 4), (30, 3), (64, 1), (96, 3), (256, 2), (264, 1),
                                 (1030, 2), (1024, 1), (2048, 1), (4096, 1), (4096, 32), (6144, 1), (10240, 1),
                                 (16384, 1)])
def test_norm_groups(D, G, dtype):
    check_norm(5, D, G, dtype, D + G, z=True)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,G", [(2, 1), (10, 5), (24, 4), (512, 64), (600, 75), (3, 3), (130, 65), (2047, 1), (2050, 1),
                                 (4095, 1), (4094, 2), (4098, 1), (8190, 1), (8194, 1), (16390, 1)])
def test_norm_odd_widths(D, G, dtype):
    """Groups of single elements, pairs and whole vectors, one vector a group, both sides of each limit."""
    check_norm(4, D, G, dtype, D + G, z=True)
    check_norm(71, D, G, dtype, D + G + 1, centered=False, act="silu")


@gpu
@pytest.mark.parametrize("rows", [0, 1, 2, 3, 7, 16, 33, 130])
def test_norm_rows(rows):
    check_norm(rows, 48, 3, F32, rows, act="silu")
    check_norm(rows, 24, 4, BF16, rows, centered=False, bias=False)
    check_norm(rows, 515, 1, F16, rows, w=False, bias=False)


@gpu
def test_norm_wide_groups():
    """Groups beyond the register kernels: any width."""
    check_norm(3, 20000, 1, F32, 1, z=True)
    check_norm(4, 33000, 1, BF16, 2, act="silu")
    check_norm(2, 2 * 9001, 2, F16, 3, centered=False)


@gpu
def test_norm_constant_group_and_offset():
    """A constant group normalises to the bias; an offset costs what its magnitude costs."""
    say("norm constant group, offset")
    x = torch.full((4, 64), 3.0, device="cuda")
    b = torch.linspace(-1, 1, 64, device="cuda")
    y = lrs.mi_group_norm_fwd(x, None, b, groups=4)
    assert torch.equal(y, b.expand(4, 64))
    check_norm(6, 128, 2, F32, 4, mean=100.0)


# ---------------------------------------------------------------------------
# GPU: what holds for all of them
# ---------------------------------------------------------------------------

def _everything(stream=None, seed=21):
    """All outputs of a small block, forward and backward."""
    kw = dict(stream=stream)
    c = conv_inputs(2, 90, 72, 4, BF16, seed)
    s = scan_inputs(2, 90, 72, 1, 16, BF16, seed)
    n = norm_inputs(180, 72, BF16, seed, z=True)
    out = []
    x, w, b, x0 = dev(c["x"], BF16), dev(c["w"], F32), dev(c["bias"], F32), dev(c["x0"], BF16)
    out += lrs.mi_causal_conv_fwd(x, w, b, x0, act="silu", **kw)
    out += lrs.mi_causal_conv_bwd(x, w, b, x0, dev(c["dy"], BF16), act="silu", **kw)
    a = {k: dev(v, F32 if k in ("A", "skip", "delta_bias", "h0", "dhT") else BF16) for k, v in s.items() if v is not None}
    args = [a[k] for k in NAMES[:5]]
    opt = {k: a[k] for k in ("skip", "z", "delta_bias", "h0")}
    y, hT, st = lrs.mi_selective_scan_fwd(*args, **opt, save_states=True, **kw)
    out += [y, hT]
    out += lrs.mi_selective_scan_bwd(*args, st, a["dy"], a["dhT"], **opt, **kw)
    nx, nw, nb, nz = dev(n["x"], BF16), dev(n["w"], F32), dev(n["bias"], F32), dev(n["z"], BF16)
    out.append(lrs.mi_group_norm_fwd(nx, nw, nb, nz, groups=3, **kw))
    out += lrs.mi_group_norm_bwd(nx, nw, nb, dev(n["dy"], BF16), nz, groups=3, **kw)
    out += lrs.mi_causal_conv_step(x[:, 0], w, b, x0, act="silu", **kw)
    out += lrs.mi_selective_scan_step(*[t[:, 0] if i != 2 else t for i, t in enumerate(args)], a["h0"], a["skip"],
                                      a["z"][:, 0], a["delta_bias"], **kw)
    return out


@gpu
def test_repeated_runs_and_side_stream_are_bitwise_equal():
    say("block operators repeated, and on a side stream")
    first = _everything()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, _everything()))
    side = torch.cuda.Stream()
    got = _everything(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, got))


@gpu
def test_strided_and_misaligned_inputs():
    """Slices of a wider projection and views off the vector alignment."""
    say("block operators on slices and misaligned views")
    wide = torch.randn(2, 40, 200, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF16)
    w = torch.randn(64, 4, device="cuda")
    part = wide[..., 70:134]
    y, _ = lrs.mi_causal_conv_fwd(part, w, act="silu")
    y2, _ = lrs.mi_causal_conv_fwd(part.contiguous(), w, act="silu")
    assert torch.equal(y, y2)
    flat = torch.randn(1 + 2 * 40 * 64, device="cuda").to(BF16)
    odd = flat[1:].view(2, 40, 64)
    assert odd.data_ptr() % 16 != 0
    a, _ = lrs.mi_causal_conv_fwd(odd, w)
    b, _ = lrs.mi_causal_conv_fwd(odd.clone(), w)
    assert torch.equal(a, b)
    assert torch.equal(lrs.mi_group_norm_fwd(odd, groups=2), lrs.mi_group_norm_fwd(odd.clone(), groups=2))
    A = -torch.rand(64, 16, device="cuda")
    bc = torch.randn(2, 40, 1, 16, device="cuda").to(BF16)
    p, q = (lrs.mi_selective_scan_fwd(t, t, A, bc, bc) for t in (odd, odd.clone()))
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@gpu
def test_graph_capture_replays():
    """Forward, backward and step captured once, replayed with new inputs, with
    eager work between the replays."""
    say("block operators under a captured graph")
    g = torch.Generator("cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x, dy, w, b = rnd(2, 70, 64).to(BF16), rnd(2, 70, 64).to(BF16), rnd(64, 4), rnd(64)
    A, bc = -torch.rand(64, 16, device="cuda", generator=g), rnd(2, 70, 1, 16).to(BF16)
    lrs.set_checked(False)
    try:
        def work():
            v, xT = lrs.mi_causal_conv_fwd(x, w, b, act="silu")
            y, hT, st = lrs.mi_selective_scan_fwd(v, v, A, bc, bc, save_states=True)
            o = lrs.mi_group_norm_fwd(y, groups=2)
            dn = lrs.mi_group_norm_bwd(y, None, None, dy, groups=2)[0]
            gr = lrs.mi_selective_scan_bwd(v, v, A, bc, bc, st, dn)
            cg = lrs.mi_causal_conv_bwd(x, w, b, None, gr[0], act="silu")
            return [o, xT, hT] + [t for t in (*gr, *cg) if t is not None]

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static = work()
        for i in range(4):
            x.copy_(rnd(2, 70, 64))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in static]
            eager = work()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, eager)), i
    finally:
        lrs.set_checked(True)


@gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements: the tail equals the tail run by itself."""
    say("conv and scan forward, T = 540000, D = 4000 bf16 (2.16e9 elements)")
    T, D, k = 540000, 4000, 200
    x = torch.empty(1, T, D, dtype=BF16, device="cuda")
    g = torch.Generator("cuda").manual_seed(4)
    for i in range(0, T, 60000):
        x[:, i:i + 60000] = torch.randn(1, 60000, D, device="cuda", generator=g)
    w = torch.randn(D, 4, device="cuda", generator=g)
    y, xT = lrs.mi_causal_conv_fwd(x, w, act="silu")
    y2, xT2 = lrs.mi_causal_conv_fwd(x[:, -k:], w, None, x[:, -k - 3:-k], act="silu")
    assert torch.equal(y[:, -k:], y2) and torch.equal(xT, xT2)
    A = -(0.5 + torch.rand(D, 4, device="cuda", generator=g))
    bc = torch.randn(1, T, 1, 4, device="cuda", generator=g).to(BF16)
    blk = lrs.mi_selective_scan_block(4)
    cut = T - 3 * blk - 5
    z = x
    h0 = lrs.mi_selective_scan_fwd(x[:, :cut], x[:, :cut], A, bc[:, :cut], bc[:, :cut], y=y[:, :cut])[1]
    ys, hT, _ = lrs.mi_selective_scan_fwd(x, x, A, bc, bc, z=z, y=y)
    t2, h2, _ = lrs.mi_selective_scan_fwd(x[:, cut:], x[:, cut:], A, bc[:, cut:], bc[:, cut:], z=z[:, cut:], h0=h0)
    # both ran the same steps from states that differ by fp32 roundings: two
    # roundings on store, and (4 a step over a decay of at most 20 steps) of the largest value
    for p, q, t in ((ys[:, cut:], t2, BF16), (hT, h2, F32)):
        p, q = p.double(), q.double()
        assert bool(torch.isfinite(p).all())
        lim = 2 * R.half_step(t) * p.abs() + 2 * 120 * 2.0 ** -24 * float(p.abs().max())
        assert bool(((p - q).abs() <= lim).all())


# ---------------------------------------------------------------------------
# GPU: every way a scan is cut over workgroups, and the operators together
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("B,T,D,G,N,lengths", [
    (1, 1000, 16, 1, 16, None),            # segments of the sequence
    (2, 700, 24, 1, 4, [700, 333]),        # ... that end inside one, or before it
    (1, 650, 40, 2, 6, None),
    (2, 500, 20, 1, 40, [0, 257]),
    (1, 300, 33, 1, 64, None),
    (4, 70, 800, 1, 16, [70, 1, 0, 65]),   # narrow tiles
    (5, 150, 650, 1, 20, None),
    (16, 40, 1280, 1, 16, None),           # wide tiles, no segments in the backward
])
def test_scan_cuts(B, T, D, G, N, lengths):
    check_scan(B, T, D, G, N, F32, T + D, lengths=lengths)


@gpu
def test_example_trains_and_serves():
    """The example block: training lowers the loss, steps equal one pass.

    Logits are fp32 sums over the blocks' outputs, of order 1 to 10, through 13
    operators a block and layer; 1e-3 is 10^3 roundings of the largest."""
    say("examples/sequence_block.py")
    import os
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sequence_block as ex
    torch.manual_seed(0)
    model = ex.Model().cuda()
    losses = ex.train(model, 60)
    assert losses[-1] < 0.7 * losses[0], (losses[0], losses[-1])
    assert ex.serve(model, [40, 17, 0, 33], 12) < 1e-3
