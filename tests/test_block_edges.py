"""Block operators where they can go wrong: gates that grow, rates that vanish,
limits of a launch, and the ways a call is cut that small shapes do not reach.

References and bounds are those of tests/block_ref.py."""
import pytest
import torch

import block_ref as R
import linear_recurrence_scans_amd as lrs
from test_block_ops import (BF16, F16, F32, NAMES, check_norm, check_scan, conv_inputs, dev, poison, quant, say,
                            scan_inputs)

gpu = pytest.mark.gpu


def run_scan(d, dtype, softplus=True, lengths=None, backward=True):
    """Forward (and backward) of the library on the float64 inputs d: (outputs, gradients)."""
    par = ("A", "skip", "delta_bias", "h0", "dhT")
    t = {k: dev(v, F32 if k in par else dtype) for k, v in d.items() if k != "lengths"}
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args, rest = [t[k] for k in NAMES[:5]], {k: t[k] for k in NAMES[5:]}
    out = lrs.mi_selective_scan_fwd(*args, **rest, softplus=softplus, lengths=ln, save_states=True)
    if not backward:
        return out, None
    return out, lrs.mi_selective_scan_bwd(*args, out[2], t["dy"], t["dhT"], **rest, softplus=softplus, lengths=ln)


# ---------------------------------------------------------------------------
# gates above one
# ---------------------------------------------------------------------------

# One shape for each number of states a lane holds, in every way that the forward
# is cut: segments of the sequence, narrow tiles, wide tiles.
CUTS = [(B, T, D, N) for N in (1, 6, 16, 20, 40)
        for B, T, D in ((1, 600, 16), (4, 70, 800), (16, 40, 1280))]


def _growing(B, T, D, N, dtype):
    """Every gate is e^30, and only the last two inputs and the first two upstream
    gradients are not zero: states and gradients stay below e^60 although the
    product of any three gates is past fp32's range."""
    d = scan_inputs(B, T, D, 1, N, dtype, B + T + N, skip=False, z=False, bias=False, h0=True)
    d["delta"], d["A"] = torch.full_like(d["delta"], 0.5), quant(60.0 + 0.1 * torch.rand(D, N, dtype=torch.float64,
                                                                 generator=torch.Generator().manual_seed(N)), F32)
    d["u"][:, :-2] = 0
    d["dy"][:, 2:] = 0
    d["h0"].zero_()
    d["dhT"].zero_()
    return d


@gpu
@pytest.mark.parametrize("B,T,D,N", CUTS)
def test_scan_gates_that_grow(B, T, D, N):
    """The product of a run of gates overflows where nothing that it multiplies does."""
    say("scan growing gates", (B, T, D, N))
    d = _growing(B, T, D, N, F32)
    (y, hT, _), got = run_scan(d, F32, softplus=False)
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin, softplus=False)
    sy, sh, _, _ = R.scan_fwd(*rin, softplus=False, absolute=True)
    # a gate's argument is near 30 (43 as a power of two): its two roundings count that often, for two gates
    c = 4 * 2 + 40 + N + 2 * 2 * 44
    e = {"y": R.worst(y, ry, sy, F32, c), "hT": R.worst(hT, rh, sh, F32, c)}
    ref = R.scan_bwd(*rin[:5], d["dy"], d["dhT"], *rin[5:], softplus=False)
    sc = R.scan_bwd(*rin[:5], d["dy"], d["dhT"], *rin[5:], softplus=False, absolute=True)
    # dBm and dCm add up the channels, dA the steps (two of them are not zero) of all sequences
    extra = dict(A=2 * B, Bm=D, Cm=D)
    for name, gt, r, s in zip(NAMES, got, ref, sc):
        if gt is not None:
            e["d" + name] = R.worst(gt, r, s, F32, 2 * c + 40 + extra.get(name, 0))
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


def check_grown(d, argument):
    """Forward against the reference where gates only multiply a carried state: each
    rounding of a gate's argument counts |argument| (as a power of two), twice a step."""
    (y, hT, _), _ = run_scan(d, F32, softplus=False, backward=False)
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin, softplus=False)
    sy, sh, _, _ = R.scan_fwd(*rin, softplus=False, absolute=True)
    T, N = d["u"].shape[1], d["A"].shape[1]
    c = 4 * T + 40 + N + 2 * T * argument
    e = {"y": R.worst(y, ry, sy, F32, c), "hT": R.worst(hT, rh, sh, F32, c)}
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("N", [1, 6, 16, 20, 40])
def test_scan_small_state_that_grows(N):
    """A state of 2^-100 under 16 gates of e^9: the product is 2^207, the state ends at 2^107."""
    say("scan small growing state", N)
    d = scan_inputs(2, 16, 24, 1, N, F32, N, skip=False, z=False, bias=False)
    d["delta"], d["A"] = torch.full_like(d["delta"], 0.5), torch.full_like(d["A"], 18.0)
    d["u"].zero_()
    d["h0"] = quant(torch.sign(d["h0"]) * 2.0 ** -100, F32)
    check_grown(d, 13)


@gpu
def test_scan_segments_that_grow_and_shrink():
    """Segments of 512 steps over which the state grows by 2^216 and shrinks again."""
    say("scan segments that grow and shrink, B=1 T=4096 D=3056 N=1")
    T, D = 4096, 3056
    d = scan_inputs(1, T, D, 1, 1, F32, 5, skip=False, z=False, bias=False)
    d["A"] = torch.full_like(d["A"], 1.0)
    up = (torch.arange(T) // 256 % 2 == 0).double() * 2 - 1
    d["delta"] = quant((up * 0.5859375)[None, :, None].expand(1, T, D), F32)
    d["u"].zero_()
    d["h0"] = quant(torch.sign(d["h0"]) * 2.0 ** -120, F32)
    assert lrs.mi_selective_scan_fwd_workspace(1, T, D, 1, 1) == 2 * 8 * D * 4  # eight segments
    check_grown(d, 1)


@gpu
@pytest.mark.parametrize("N", [1, 6, 16, 20, 40])
@pytest.mark.parametrize("T,lengths", [(5, None), (150, [150, 0, 33])])
def test_scan_rates_that_forget_everything(T, lengths, N):
    """A of -inf: a gate is zero wherever the rate is not, also in a block whose last
    steps do not exist.  A of -3e38, finite, has gradients too."""
    say("scan A = -inf and -3e38", T, N, lengths)
    d = scan_inputs(3, T, 24, 1, N, F32, T + N, lengths=lengths)
    for low, backward in ((float("-inf"), False), (-3e38, True)):
        d["A"][:, 0] = low
        d["A"] = quant(d["A"], F32)
        (y, hT, _), got = run_scan(d, F32, lengths=lengths, backward=backward)
        rin = [d[k] for k in NAMES]
        ry, rh, _, _ = R.scan_fwd(*rin, lengths=d["lengths"])
        sy, sh, _, _ = R.scan_fwd(*rin, lengths=d["lengths"], absolute=True)
        c = 4 * T + 40 + N
        e = {"y": R.worst(y, ry, sy, F32, c), "hT": R.worst(hT, rh, sh, F32, c)}
        if backward:
            ref = R.scan_bwd(*rin[:5], d["dy"], d["dhT"], *rin[5:], lengths=d["lengths"])
            sc = R.scan_bwd(*rin[:5], d["dy"], d["dhT"], *rin[5:], lengths=d["lengths"], absolute=True)
            extra = dict(A=3 * T, Bm=24, Cm=24, skip=3 * T, delta_bias=3 * T)
            for name, gt, r, s in zip(NAMES, got, ref, sc):
                e["d" + name] = R.worst(gt, r, s, F32, 2 * c + 40 + extra.get(name, 0))
        print(e, flush=True)
        assert max(e.values()) <= 1.0, e


@gpu
def test_scan_step_that_forgets_everything():
    """The single-token step with A of -3e38: a rate of zero keeps the state, any other replaces it."""
    say("scan step A = -3e38")
    d = scan_inputs(2, 1, 24, 1, 16, F32, 3)
    d["A"][:, 3] = quant(torch.tensor(-3e38, dtype=torch.float64), F32)
    d["delta"][0] = -200.0
    t = {k: dev(v, F32) for k, v in d.items() if v is not None}
    y, h = lrs.mi_selective_scan_step(t["u"][:, 0], t["delta"][:, 0], t["A"], t["Bm"][:, 0], t["Cm"][:, 0], t["h0"],
                                      t["skip"], t["z"][:, 0], t["delta_bias"])
    rin = [d[k] for k in NAMES]
    ry, rh, _, _ = R.scan_fwd(*rin)
    sy, sh, _, _ = R.scan_fwd(*rin, absolute=True)
    e = {"y": R.worst(y, ry[:, 0], sy[:, 0], F32, 60), "h": R.worst(h, rh, sh, F32, 60)}
    print(e, flush=True)
    assert max(e.values()) <= 1.0, e


# ---------------------------------------------------------------------------
# the rate softplus(x)
# ---------------------------------------------------------------------------

@gpu
def test_rate_is_accurate_relative_to_itself():
    """One state, A = 0 and ones elsewhere: y is the rate, ddelta its derivative.  The rate's
    bound, in half steps of 2^-24: two for each of exp2 and log2, one each for the product's
    remainder, the join and the sum with max(x, 0), one for the remainder of 1 + e taken
    without its factor 1 / (1 + e); and ln 2 in fp32 leaves 0.05 |x| of the remainder.  The
    derivative's: exp2 and its remainder as there, two for the reciprocal, one each for
    1 + e and the products.  Rates of 1e-3 to 1e-1 lie at x = -7 to -2."""
    say("softplus rates")
    x = torch.cat([torch.linspace(-80, 80, 8192, dtype=torch.float64), torch.linspace(-16, 4, 16384, dtype=torch.float64),
                   torch.tensor([0.0, -1e-30, 1e-30, 500.0], dtype=torch.float64)]).float().double()
    n = x.numel()
    want = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    one = torch.ones(1, 1, 1, 1, device="cuda")
    u, A = torch.ones(1, 1, n, device="cuda"), torch.zeros(n, 1, device="cuda")
    delta = x.float().cuda().view(1, 1, n)
    y, hT, st = lrs.mi_selective_scan_fwd(u, delta, A, one, one, save_states=True)
    dd = lrs.mi_selective_scan_bwd(u, delta, A, one, one, st, torch.ones_like(u))[1]
    y1, h1 = lrs.mi_selective_scan_step(u[:, 0], delta[:, 0], A, one[:, 0], one[:, 0], torch.zeros(1, n, 1, device="cuda"))
    lim = (8 + 0.05 * x.abs()) * 2.0 ** -24 * want
    worst = {k: float(((g.cpu().double().view(-1) - want).abs() / lim).max())
             for k, g in (("y", y), ("hT", hT), ("y1", y1), ("h1", h1))}
    der = torch.exp(-torch.log1p(torch.exp(-x)))
    worst["ddelta"] = float(((dd.cpu().double().view(-1) - der).abs() / ((8 + 0.05 * x.abs()) * 2.0 ** -24 * der)).max())
    print(worst, flush=True)
    assert max(worst.values()) <= 1.0, worst


@gpu
def test_rate_of_infinities():
    """softplus(-inf) is zero (the state stays, the token leaves no trace); inf and NaN stay
    what they are in the state, and y is not finite either."""
    say("softplus of -inf, inf, NaN")
    x = torch.tensor([float("-inf"), -1000.0, 1000.0, float("inf"), float("nan")], device="cuda")
    one = torch.ones(1, 1, 1, 1, device="cuda")
    h0 = torch.full((1, 5, 1), 3.0, device="cuda")
    y, hT, _ = lrs.mi_selective_scan_fwd(torch.ones(1, 1, 5, device="cuda"), x.view(1, 1, 5),
                                         torch.full((5, 1), -1.0, device="cuda"), one, one, h0=h0)
    y, hT = y.flatten().tolist(), hT.flatten().tolist()
    assert y[:3] == hT[:3] == [3.0, 3.0, 1000.0]
    assert hT[3] == float("inf") and hT[4] != hT[4]
    assert not torch.isfinite(torch.tensor(y[3:])).any()


# ---------------------------------------------------------------------------
# limits of a launch (CPU: nothing is launched, the addresses are never read)
# ---------------------------------------------------------------------------

def test_calls_beyond_one_launch_are_refused():
    """2^32 threads or more: refused as unsupported before any launch."""
    L = lrs._load()
    UNSUPPORTED = 2
    p = [(1 << 42) * (i + 1) for i in range(22)]
    far = 1 << 60
    assert L.mi_causal_conv_fwd(p[0], p[1], None, None, None, p[2], None, 1 << 24, 1, 4, 4, 0, 0, None) == UNSUPPORTED
    assert L.mi_causal_conv_bwd(p[0], p[1], None, None, None, p[2], None, p[3], p[4], None, None, 1 << 24, 1, 4, 4, 0, 0,
                                far, 1 << 50, None) == UNSUPPORTED
    assert L.mi_causal_conv_step(p[0], p[1], None, p[2], p[3], p[4], 1 << 32, 1, 2, 0, 0, None) == UNSUPPORTED
    assert L.mi_selective_scan_fwd(*p[:5], None, None, None, None, None, p[5], p[6], None, 1 << 24, 1, 1, 1, 1, 1, 0,
                                   None, 0, None) == UNSUPPORTED
    assert L.mi_selective_scan_bwd(*p[:5], None, None, None, p[5], None, p[6], None, *p[7:12], None, None, None, None,
                                   1 << 23, 1, 1, 1, 1, 1, 0, far, 1 << 50, None) == UNSUPPORTED
    assert L.mi_selective_scan_step(*p[:6], None, None, None, p[6], p[7], 1 << 24, 1, 1, 1, 1, 0, None) == UNSUPPORTED
    G = 1 << 24
    assert L.mi_group_norm_fwd(p[0], None, None, None, p[1], 1, 260 * G, G, 1e-5, 1, 0, 0, None) == UNSUPPORTED
    assert L.mi_group_norm_bwd(p[0], None, None, None, p[1], p[2], None, None, None, 1, 260 * G, G, 1e-5, 1, 0, 0, far,
                               1 << 50, None) == UNSUPPORTED


def test_outputs_that_are_no_tensors():
    """An output given by the caller is checked for what it is before its shape is."""
    from linear_recurrence_scans_amd import block_ops
    like = torch.zeros(2, 3)
    for bad in ([0.0] * 6, 1, "y"):
        with pytest.raises(TypeError, match="y must be a torch.Tensor"):
            block_ops._new(bad, like, (2, 3), "y")
        with pytest.raises(TypeError, match="y must be a torch.Tensor"):
            block_ops._out(bad, like, "y")
    with pytest.raises(ValueError, match="y must be a contiguous"):
        block_ops._new(torch.zeros(3, 2).t(), like, (2, 3), "y")
    ok = torch.zeros(2, 3)
    assert block_ops._out(ok, like, "y") is ok


# ---------------------------------------------------------------------------
# non-finite inputs
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("what,value", [("u", float("inf")), ("u", float("nan")), ("delta", float("inf"))])
@pytest.mark.parametrize("B,T,D,N", [(2, 300, 16, 6), (4, 70, 800, 16), (16, 40, 1280, 16), (2, 70, 16, 40)])
def test_scan_nonfinite_inputs_stay_in_their_channel(B, T, D, N, what, value):
    """One bad token of one channel: what the formulas do not make of it keeps its bits, and
    what they do is not finite."""
    say("scan with", what, value, (B, T, D, N))
    b, t, c = 1, 21, 5
    d = scan_inputs(B, T, D, 1, N, F32, N)
    (y, hT, st), g = run_scan(d, F32)
    d[what][b, t, c] = value
    (y2, hT2, st2), g2 = run_scan(d, F32)
    seen = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    seen[b, t:, c] = True
    assert torch.equal(y[~seen], y2[~seen]) and not torch.isfinite(y2[seen]).any()
    own = torch.zeros(B, D, dtype=torch.bool, device="cuda")
    own[b, c] = True
    assert torch.equal(hT[~own], hT2[~own]) and not torch.isfinite(hT2[own]).any()
    same = lambda i, keep: torch.equal(g[i][keep], g2[i][keep])
    for i, name in enumerate(NAMES):
        if name in ("u", "delta", "z"):
            keep = torch.ones(B, T, D, dtype=torch.bool, device="cuda")
            keep[b, :, c] = False
        elif name in ("Bm", "Cm"):  # sums over the channels
            keep = torch.ones(B, T, dtype=torch.bool, device="cuda")
            keep[b] = False
            if name == "Cm":
                keep[b, :t] = True  # the states before
            elif what == "u":
                keep[b] = True      # g of the other tokens does not depend on u
                keep[b, t] = False
        elif name == "h0":
            keep = ~own
        else:
            keep = torch.ones(D, dtype=torch.bool, device="cuda")
            keep[c] = False
        assert same(i, keep), name
    if what == "u":  # neither du nor dh0 depends on u
        assert same(0, slice(None)) and same(8, slice(None))


# ---------------------------------------------------------------------------
# every way a call is cut, over several blocks and turns
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("T,N,dtype", [(600, 3, F32), (600, 4, F16), (300, 7, F32), (300, 8, BF16), (300, 16, F32),
                                       (300, 16, BF16), (300, 16, F16), (200, 24, BF16), (110, 33, F32), (110, 64, F16)])
def test_scan_narrow_tiles_over_several_blocks(T, N, dtype):
    """Narrow tiles of the forward, at least three blocks of 32 to 256 steps, each number of
    states a lane holds; the states it saves; the backward in segments and without."""
    check_scan(4, T, 800, 1, N, dtype, T + N, lengths=[T, 0, T // 2 + 3, 1])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,T,D,G,N,lengths", [(1, 1000, 16, 1, 16, None), (2, 700, 24, 1, 4, [700, 333]),
                                               (1, 650, 40, 2, 6, None), (2, 500, 20, 1, 40, [0, 257]),
                                               (1, 600, 31, 1, 20, None), (16, 40, 1280, 1, 8, None)])
def test_scan_cuts_in_16_bits(B, T, D, G, N, lengths, dtype):
    """Segments of both directions and wide tiles."""
    check_scan(B, T, D, G, N, dtype, T + D, lengths=lengths)


def conv_all(d, act, absolute=False):
    """R.conv_fwd and R.conv_bwd with all steps at once: y, xT, dx, dw, dbias, dx0."""
    ab = (lambda t: t.abs()) if absolute else (lambda t: t)
    x, w, K, ln = d["x"], d["w"], d["w"].shape[1], d["lengths"].long()
    B, T, D = x.shape
    ok = (torch.arange(T)[None] < ln[:, None])[..., None]
    xe = torch.cat([d["x0"], torch.where(ok, x, 0.0)], 1)
    rows = ln[:, None] + torch.arange(K - 1)[None]
    pick = rows[..., None].expand(B, K - 1, D)
    win = lambda e, k: e[:, k:k + T]
    s = d["bias"] + sum(win(xe, k) * w[:, k] for k in range(K))
    mag = sum(win(xe, k).abs() * w[:, k].abs() for k in range(K))
    sa = mag + d["bias"].abs() if absolute else s
    y = (sa * 1.1 if absolute else R.silu(s)) if act else sa
    ds = ab(d["dy"])
    if act:
        ds = ds * (1.1 + 0.5 * mag if absolute else R.dsilu(s))
    ds = torch.where(ok, ds, 0.0)
    dxe = torch.zeros_like(xe)
    for k in range(K):
        dxe[:, k:k + T] += ds * ab(w)[:, k]
    dxe.scatter_add_(1, pick, ab(d["dxT"]))
    dw = torch.stack([(ds * win(ab(xe), k)).sum((0, 1)) for k in range(K)], 1)
    return (torch.where(ok, y, 0.0), torch.gather(xe, 1, pick), torch.where(ok, dxe[:, K - 1:], 0.0), dw,
            ds.sum((0, 1)), dxe[:, :K - 1])


@pytest.mark.parametrize("absolute", [False, True])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("K", [2, 4])
def test_conv_all_is_the_reference(K, act, absolute):
    d = conv_inputs(3, 7, 4, K, F32, K, lengths=[7, 0, 2])
    args = (d["x"], d["w"], d["bias"], d["x0"])
    want = R.conv_fwd(*args, d["lengths"], act, absolute)[:1] + \
        R.conv_fwd(*args, d["lengths"], act)[1:] + \
        R.conv_bwd(*args, d["dy"], d["dxT"], d["lengths"], act, absolute)
    for name, g, r in zip(("y", "xT", "dx", "dw", "dbias", "dx0"), conv_all(d, act, absolute), want):
        assert float((g - r).abs().max()) <= 1e-12, name


@gpu
@pytest.mark.parametrize("B,T,D,K,dtype,run", [(1400, 70, 12, 4, BF16, 32), (2100, 70, 10, 3, F32, 64),
                                               (900, 300, 8, 5, F16, 64), (1400, 70, 9, 4, F32, 32)])
def test_conv_backward_long_runs(B, T, D, K, dtype, run):
    """Runs of 32 and 64 steps a wave (shorter ones are all that few sequences get), lengths
    that end inside them."""
    say("conv backward, runs of", run, (B, T, D, K), dtype)
    g = torch.Generator().manual_seed(B)
    d = conv_inputs(B, T, D, K, dtype, K, lengths=torch.randint(0, T + 1, (B,), generator=g).tolist())
    ln, lnd = d["lengths"], d["lengths"].cuda()
    # the partial rows that the workspace holds tell the run: four waves a workgroup
    rows = lrs.mi_causal_conv_bwd_workspace(B, T, D, K, dtype) // ((K + 1) * D * 4)
    assert rows == B * -(-T // (4 * run))
    x, dy = dev(poison(d["x"], ln), dtype), dev(poison(d["dy"], ln), dtype)
    w, bias, x0, dxT = dev(d["w"], F32), dev(d["bias"], F32), dev(d["x0"], dtype), dev(d["dxT"], dtype)
    y, xT = lrs.mi_causal_conv_fwd(x, w, bias, x0, act="silu", lengths=lnd)
    got = (y, xT) + tuple(lrs.mi_causal_conv_bwd(x, w, bias, x0, dy, dxT, act="silu", lengths=lnd))
    ref, sc = conv_all(d, "silu"), conv_all(d, "silu", absolute=True)
    e, c = {}, 2 * K + 26
    for name, gt, r, s, ty, n in zip(("y", "xT", "dx", "dw", "dbias", "dx0"), got, ref, sc,
                                     (dtype, dtype, dtype, F32, F32, dtype), (K + 13, 0, c, c + B * T, c + B * T, c)):
        e[name] = R.worst(gt, r, s, ty, n)
    print(e, flush=True)
    assert torch.equal(xT.cpu().double(), ref[1]) and max(e.values()) <= 1.0, e


@gpu
@pytest.mark.parametrize("rows,D,G,dtype", [(1100, 515, 1, F32), (4099, 515, 1, F16), (1100, 264, 1, BF16),
                                            (4099, 64, 1, F32), (4099, 64, 4, F16), (40003, 64, 1, BF16),
                                            (1031, 4097, 1, F32), (2061, 4097, 1, BF16), (9001, 24, 24, F32),
                                            (1027, 6144, 1, BF16), (1030, 10240, 2, F16)])
def test_norm_workgroups_walk_several_rows(rows, D, G, dtype):
    """More rows than workgroups take at once, in each kind of team and in the kernel for any
    width: parameters' gradients add up over the turns, and the last turn is not whole."""
    check_norm(rows, D, G, dtype, rows + D, z=True)
    check_norm(rows, D, G, dtype, rows + D + 1, centered=False, act="silu")


# ---------------------------------------------------------------------------
# single tokens under a captured graph
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_replay_under_a_graph(dtype):
    """Convolution step, scan step and norm of one token captured once, states updated in
    place, replayed token by token with eager work between: each replay equals the eager step."""
    say("token steps under a captured graph", dtype)
    B, D, K, N, T = 3, 72, 4, 16, 6
    c = conv_inputs(B, T, D, K, dtype, 31)
    s = scan_inputs(B, T, D, 1, N, dtype, 32)
    x, z, delta = (dev(t, dtype) for t in (c["x"], s["z"], s["delta"]))
    Bm, Cm = dev(s["Bm"], dtype), dev(s["Cm"], dtype)
    w, b, A, skip, bias = (dev(t, F32) for t in (c["w"], c["bias"], s["A"], s["skip"], s["delta_bias"]))
    token = [t[:, 0].clone() for t in (x, z, delta, Bm, Cm)]

    def step(taps, h):
        v, _ = lrs.mi_causal_conv_step(token[0], w, b, taps, act="silu", x_out=taps)
        y, _ = lrs.mi_selective_scan_step(v, token[2], A, token[3], token[4], h, skip, None, bias, h_out=h)
        return lrs.mi_group_norm_fwd(y, None, None, token[1], groups=3, centered=False)

    fresh = lambda: (torch.zeros(B, K - 1, D, dtype=dtype, device="cuda"), torch.zeros(B, D, N, device="cuda"))
    held, mine = fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*fresh())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held)
    for t in held:
        t.zero_()  # (capturing ran nothing; the states start where the eager ones do)
    for t in range(T):
        for dst, src in zip(token, (x, z, delta, Bm, Cm)):
            dst.copy_(src[:, t])
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = step(*mine)
        torch.cuda.synchronize()
        assert torch.equal(got, want), t
        assert torch.equal(held[0], mine[0]) and torch.equal(held[1], mine[1]), t
