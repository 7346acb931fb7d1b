"""Block operators: the short causal convolution, the selective state-space scan
and the gated group norm (C ABI in ``include/miscan.h``, section "Block
operators").

Activations are (B, T, D), or (B, D) for one step, in float32, bfloat16 or
float16; parameters (w, bias, A, skip, delta_bias) and scan states are float32.
`lengths` is an int32 tensor (B,) on the GPU, clamped to [0, T]: steps at or
past a sequence's length are ignored and give zero.  As for the scans, inputs
are made contiguous, outputs and workspaces are allocated with torch and the
kernels run on `stream` (default: torch's current stream).
"""
from __future__ import annotations

import torch

from . import _Call, _check, _device, _dt, _load, _workspace

__all__ = [
    "mi_causal_conv_fwd", "mi_causal_conv_bwd", "mi_causal_conv_bwd_workspace", "mi_causal_conv_step",
    "mi_selective_scan_block", "mi_selective_scan_fwd", "mi_selective_scan_fwd_workspace", "mi_selective_scan_bwd",
    "mi_selective_scan_bwd_workspace", "mi_selective_scan_step",
    "mi_group_norm_fwd", "mi_group_norm_bwd", "mi_group_norm_bwd_workspace",
]

_ACTS = {None: 0, "silu": 1}
_F32, _I32 = torch.float32, torch.int32


# A step of a few microseconds on the GPU is bound by what the host does to
# launch it, so the common call (torch's current stream and device) goes
# without the context managers of a side stream.
class _Here:
    """Call on the current stream of the current device."""

    __slots__ = ("handle",)
    side = False

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


# (tensors on a GPU have initialised torch's runtime, so the raw lookups are safe;
# a torch without GPU support has none, and no such tensors)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(stream, device):
    index = device.index
    if stream is None and index == _current_device():
        return _Here(_current_raw_stream(index))
    return _Call(stream, device)


def _act(act) -> int:
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError("act must be None or 'silu', not %r" % (act,)) from None


def _dev_tensor(t, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _device(t, name)
    return t if t.is_contiguous() else t.contiguous()


def _need(t, like: torch.Tensor, shape, name: str, dtype=None):
    """An input of the given shape on `like`'s device (dtype: `like`'s by default)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _device(t, name)
    if t.shape != shape or t.dtype != (dtype or like.dtype) or t.device != like.device:
        raise ValueError("%s must be a %s tensor of shape %s on %s"
                         % (name, dtype or like.dtype, tuple(shape), like.device))
    return t if t.is_contiguous() else t.contiguous()


def _opt(t, like: torch.Tensor, shape, name: str, dtype=None):
    return None if t is None else _need(t, like, shape, name, dtype)


def _new(t, like: torch.Tensor, shape, name: str, dtype=None):
    """An output: the caller's `t`, checked, or a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != shape or t.dtype != (dtype or like.dtype) or t.device != like.device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype or like.dtype, tuple(shape), like.device))
    return t


def _out(t, like: torch.Tensor, name: str):
    return torch.empty_like(like) if t is None else _new(t, like, like.shape, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------

def _conv_shape(x, w, dims):
    if x.dim() != dims:
        raise ValueError("x must be (B, %sD)" % ("T, " if dims == 3 else ""))
    if w.dim() != 2 or w.shape[0] != x.shape[-1] or w.dtype != _F32 or w.device != x.device:
        raise ValueError("w must be a float32 (D, K) tensor on x's device")
    return w.shape[1]


def mi_causal_conv_fwd(x, w, bias=None, x0=None, *, act=None, lengths=None, y=None, xT=None, stream=None):
    """(y, xT): depthwise causal convolution of x (B, T, D) with w (D, K), plus
    bias (D), through `act` (None or "silu").  x0 (B, K-1, D) holds the inputs
    before the first step (None = zeros); xT (B, K-1, D) is the x0 of the
    sequence's continuation."""
    with _call(stream, _device(x, "x")) as c:
        x, w = _dev_tensor(x, "x"), _dev_tensor(w, "w")
        K = _conv_shape(x, w, 3)
        Bn, T, D = x.shape
        bias = None if bias is None else _need(bias, x, (D,), "bias", _F32)
        x0 = None if x0 is None else _need(x0, x, (Bn, K - 1, D), "x0")
        lengths = None if lengths is None else _need(lengths, x, (Bn,), "lengths", _I32)
        y, xT = _out(y, x, "y"), _new(xT, x, (Bn, max(K - 1, 0), D), "xT")
        if c.side:
            c.keep(x, w, bias, x0, lengths, y, xT)
        st = _load().mi_causal_conv_fwd(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(x0), _ptr(lengths),
                                        y.data_ptr(), xT.data_ptr(), Bn, T, D, K, _act(act), _dt(x), c.handle)
        if st:
            _check(st, "mi_causal_conv_fwd")
    return y, xT


def mi_causal_conv_bwd_workspace(B: int, T: int, D: int, K: int, dtype=torch.float32) -> int:
    from . import _DTYPES
    return int(_load().mi_causal_conv_bwd_workspace(B, T, D, K, _DTYPES[dtype]))


def mi_causal_conv_bwd(x, w, bias, x0, dy, dxT=None, *, act=None, lengths=None, dx=None, dw=None, dbias=None,
                       dx0=None, ws=None, stream=None):
    """(dx, dw, dbias, dx0): gradient of mi_causal_conv_fwd for dy (B, T, D) and,
    optionally, dxT (B, K-1, D); dbias and dx0 are None without bias and x0."""
    with _call(stream, _device(x, "x")) as c:
        x, w, dy = _dev_tensor(x, "x"), _dev_tensor(w, "w"), _dev_tensor(dy, "dy")
        K = _conv_shape(x, w, 3)
        Bn, T, D = x.shape
        dy = _need(dy, x, x.shape, "dy")
        bias = None if bias is None else _need(bias, x, (D,), "bias", _F32)
        x0 = None if x0 is None else _need(x0, x, (Bn, K - 1, D), "x0")
        dxT = None if dxT is None else _need(dxT, x, (Bn, K - 1, D), "dxT")
        lengths = None if lengths is None else _need(lengths, x, (Bn,), "lengths", _I32)
        dx, dw = _out(dx, x, "dx"), _out(dw, w, "dw")
        dbias = _out(dbias, bias, "dbias") if bias is not None else None
        dx0 = _out(dx0, x0, "dx0") if x0 is not None else None
        dt = _dt(x)
        ws = _workspace(ws, _load().mi_causal_conv_bwd_workspace(Bn, T, D, K, dt), x.device)
        if c.side:
            c.keep(x, w, bias, x0, lengths, dy, dxT, dx, dw, dbias, dx0, ws)
        st = _load().mi_causal_conv_bwd(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(x0), _ptr(lengths),
                                        dy.data_ptr(), _ptr(dxT), dx.data_ptr(), dw.data_ptr(), _ptr(dbias),
                                        _ptr(dx0), Bn, T, D, K, _act(act), dt, ws.data_ptr(), _nbytes(ws), c.handle)
        if st:
            _check(st, "mi_causal_conv_bwd")
    return dx, dw, dbias, dx0


def mi_causal_conv_step(x, w, bias, x0, *, act=None, y=None, x_out=None, stream=None):
    """(y, x_out): one step, x (B, D) with the carried inputs x0 (B, K-1, D).
    x_out (default: a new tensor) may be x0 itself, which is then updated in place."""
    with _call(stream, _device(x, "x")) as c:
        x, w = _dev_tensor(x, "x"), _dev_tensor(w, "w")
        K = _conv_shape(x, w, 2)
        Bn, D = x.shape
        bias = None if bias is None else _need(bias, x, (D,), "bias", _F32)
        own = x0
        x0 = _need(x0, x, (Bn, K - 1, D), "x0")
        if x_out is own and x0 is not own:
            raise ValueError("x0 must be contiguous to be updated in place")
        y, x_out = _out(y, x, "y"), _out(x_out, x0, "x_out")
        if c.side:
            c.keep(x, w, bias, x0, y, x_out)
        st = _load().mi_causal_conv_step(x.data_ptr(), w.data_ptr(), _ptr(bias), x0.data_ptr(), y.data_ptr(),
                                         x_out.data_ptr(), Bn, D, K, _act(act), _dt(x), c.handle)
        if st:
            _check(st, "mi_causal_conv_step")
    return y, x_out


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def mi_selective_scan_block(N: int) -> int:
    """Steps between two of the states that the forward saves for the backward."""
    return int(_load().mi_selective_scan_block(N))


def _scan_args(u, delta, A, Bm, Cm, skip, z, delta_bias, dims):
    """Checked, contiguous inputs and (B, T, D, G, N); T = 1 for one step."""
    u, A, Bm = _dev_tensor(u, "u"), _dev_tensor(A, "A"), _dev_tensor(Bm, "Bm")
    if u.dim() != dims:
        raise ValueError("u must be (B, %sD)" % ("T, " if dims == 3 else ""))
    D = u.shape[-1]
    if A.dim() != 2 or A.shape[0] != D or A.dtype != _F32 or A.device != u.device:
        raise ValueError("A must be a float32 (D, N) tensor on u's device")
    N = A.shape[1]
    if Bm.dim() != dims + 1 or Bm.shape[:-2] != u.shape[:-1] or Bm.shape[-1] != N or Bm.shape[-2] < 1:
        raise ValueError("Bm and Cm must be (B, %sG, N)" % ("T, " if dims == 3 else ""))
    G = Bm.shape[-2]
    if D % G:
        raise ValueError("G = %d must divide D = %d" % (G, D))
    delta = _need(delta, u, u.shape, "delta")
    Cm = _need(Cm, u, Bm.shape, "Cm")
    if Bm.dtype != u.dtype or Bm.device != u.device:
        raise ValueError("u, delta, Bm, Cm and z must share device and dtype (%s, %s)" % (u.device, u.dtype))
    skip, delta_bias = _opt(skip, u, (D,), "skip", _F32), _opt(delta_bias, u, (D,), "delta_bias", _F32)
    z = None if z is None else _need(z, u, u.shape, "z")
    T = u.shape[1] if dims == 3 else 1
    return (u, delta, A, Bm, Cm, skip, z, delta_bias), (u.shape[0], T, D, G, N)


def mi_selective_scan_fwd_workspace(B: int, T: int, D: int, G: int, N: int, dtype=torch.float32) -> int:
    from . import _DTYPES
    return int(_load().mi_selective_scan_fwd_workspace(B, T, D, G, N, _DTYPES[dtype]))


def mi_selective_scan_fwd(u, delta, A, Bm, Cm, skip=None, z=None, delta_bias=None, h0=None, *, softplus=True,
                          lengths=None, save_states=False, y=None, hT=None, states=None, ws=None, stream=None):
    """(y, hT, states): the selective scan of u (B, T, D) with rates
    softplus(delta + delta_bias), A (D, N), Bm, Cm (B, T, G, N), y gated by
    silu(z), from the state h0 (B, D, N) to hT.  `states` is what the backward
    needs, or None unless save_states is set (or a tensor for it is given)."""
    with _call(stream, _device(u, "u")) as c:
        args, (Bn, T, D, G, N) = _scan_args(u, delta, A, Bm, Cm, skip, z, delta_bias, 3)
        u = args[0]
        h0 = None if h0 is None else _need(h0, u, (Bn, D, N), "h0", _F32)
        lengths = None if lengths is None else _need(lengths, u, (Bn,), "lengths", _I32)
        y, hT = _out(y, u, "y"), _new(hT, u, (Bn, D, N), "hT", _F32)
        if save_states or states is not None:
            blk = max(1, mi_selective_scan_block(N))
            states = _new(states, u, (Bn, (T + blk - 1) // blk, D, N), "states", _F32)
        lib, dt = _load(), _dt(u)
        need = lib.mi_selective_scan_fwd_workspace(Bn, T, D, G, N, dt)
        if need:
            ws = _workspace(ws, need, u.device)
        if c.side:
            c.keep(*args, h0, lengths, y, hT, states, ws)
        st = lib.mi_selective_scan_fwd(*(_ptr(t) for t in args), _ptr(h0), _ptr(lengths), y.data_ptr(),
                                       hT.data_ptr(), _ptr(states), Bn, T, D, G, N, int(bool(softplus)), dt,
                                       _ptr(ws), 0 if ws is None else _nbytes(ws), c.handle)
        if st:
            _check(st, "mi_selective_scan_fwd")
    return y, hT, states


def mi_selective_scan_bwd_workspace(B: int, T: int, D: int, G: int, N: int, dtype=torch.float32) -> int:
    from . import _DTYPES
    return int(_load().mi_selective_scan_bwd_workspace(B, T, D, G, N, _DTYPES[dtype]))


def mi_selective_scan_bwd(u, delta, A, Bm, Cm, states, dy, dhT=None, skip=None, z=None, delta_bias=None, h0=None, *,
                          softplus=True, lengths=None, ws=None, stream=None):
    """(du, ddelta, dA, dBm, dCm, dskip, dz, ddelta_bias, dh0): gradient of
    mi_selective_scan_fwd for dy (B, T, D) and, optionally, dhT (B, D, N), given
    the forward's `states`; None for inputs that were None."""
    with _call(stream, _device(u, "u")) as c:
        args, (Bn, T, D, G, N) = _scan_args(u, delta, A, Bm, Cm, skip, z, delta_bias, 3)
        u, delta, A, Bm, Cm, skip, z, delta_bias = args
        blk = max(1, mi_selective_scan_block(N))
        states = _need(states, u, (Bn, (T + blk - 1) // blk, D, N), "states", _F32)
        dy = _need(dy, u, u.shape, "dy")
        dhT = None if dhT is None else _need(dhT, u, (Bn, D, N), "dhT", _F32)
        h0 = None if h0 is None else _need(h0, u, (Bn, D, N), "h0", _F32)
        lengths = None if lengths is None else _need(lengths, u, (Bn,), "lengths", _I32)
        grads = [torch.empty_like(t) if t is not None else None
                 for t in (u, delta, A, Bm, Cm, skip, z, delta_bias, h0)]
        du, ddelta, dA, dBm, dCm, dskip, dz, dbias, dh0 = grads
        dt = _dt(u)
        ws = _workspace(ws, _load().mi_selective_scan_bwd_workspace(Bn, T, D, G, N, dt), u.device)
        if c.side:
            c.keep(*args, states, dy, dhT, lengths, *grads, ws)
        st = _load().mi_selective_scan_bwd(*(_ptr(t) for t in args), states.data_ptr(), _ptr(lengths), dy.data_ptr(),
                                           _ptr(dhT), du.data_ptr(), ddelta.data_ptr(), dA.data_ptr(),
                                           dBm.data_ptr(), dCm.data_ptr(), _ptr(dskip), _ptr(dz), _ptr(dbias),
                                           _ptr(dh0), Bn, T, D, G, N, int(bool(softplus)), dt, ws.data_ptr(),
                                           _nbytes(ws), c.handle)
        if st:
            _check(st, "mi_selective_scan_bwd")
    return tuple(grads)


def mi_selective_scan_step(u, delta, A, Bm, Cm, h, skip=None, z=None, delta_bias=None, *, softplus=True, y=None,
                           h_out=None, stream=None):
    """(y, h_out): one step, u, delta, z (B, D), Bm, Cm (B, G, N), from the state
    h (B, D, N).  h_out (default: a new tensor) may be h itself, which is then
    updated in place."""
    with _call(stream, _device(u, "u")) as c:
        args, (Bn, _, D, G, N) = _scan_args(u, delta, A, Bm, Cm, skip, z, delta_bias, 2)
        u, delta, A, Bm, Cm, skip, z, delta_bias = args
        own = h
        h = _need(h, u, (Bn, D, N), "h", _F32)
        if h_out is own and h is not own:
            raise ValueError("h must be contiguous to be updated in place")
        y, h_out = _out(y, u, "y"), _out(h_out, h, "h_out")
        if c.side:
            c.keep(*args, h, y, h_out)
        st = _load().mi_selective_scan_step(u.data_ptr(), delta.data_ptr(), A.data_ptr(), Bm.data_ptr(),
                                            Cm.data_ptr(), h.data_ptr(), _ptr(skip), _ptr(z), _ptr(delta_bias),
                                            y.data_ptr(), h_out.data_ptr(), Bn, D, G, N, int(bool(softplus)),
                                            _dt(u), c.handle)
        if st:
            _check(st, "mi_selective_scan_step")
    return y, h_out


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def _norm_args(x, w, bias, z, groups, act):
    x = _dev_tensor(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    D = x.shape[-1]
    if groups < 1 or D % groups:
        raise ValueError("groups = %d must divide D = %d" % (groups, D))
    if z is not None and act is not None:
        raise ValueError("act and z exclude each other")
    w, bias = _opt(w, x, (D,), "w", _F32), _opt(bias, x, (D,), "bias", _F32)
    z = None if z is None else _need(z, x, x.shape, "z")
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return x, w, bias, z, rows, D


def mi_group_norm_fwd(x, w=None, bias=None, z=None, *, groups=1, eps=1e-5, centered=True, act=None, y=None,
                      stream=None):
    """y: x (..., D) normalised over the D / groups channels of each group of
    each row (mean and variance, or the root mean square if not centered), times
    w plus bias, through `act` or gated by silu(z)."""
    with _call(stream, _device(x, "x")) as c:
        x, w, bias, z, R, D = _norm_args(x, w, bias, z, groups, act)
        y = _out(y, x, "y")
        if c.side:
            c.keep(x, w, bias, z, y)
        st = _load().mi_group_norm_fwd(x.data_ptr(), _ptr(w), _ptr(bias), _ptr(z), y.data_ptr(), R, D, groups, eps,
                                       int(bool(centered)), _act(act), _dt(x), c.handle)
        if st:
            _check(st, "mi_group_norm_fwd")
    return y


def mi_group_norm_bwd_workspace(R: int, D: int, groups: int, dtype=torch.float32) -> int:
    from . import _DTYPES
    return int(_load().mi_group_norm_bwd_workspace(R, D, groups, _DTYPES[dtype]))


def mi_group_norm_bwd(x, w, bias, dy, z=None, *, groups=1, eps=1e-5, centered=True, act=None, dx=None, ws=None,
                      stream=None):
    """(dx, dw, dbias, dz): gradient of mi_group_norm_fwd for dy (..., D); None
    for inputs that were None."""
    with _call(stream, _device(x, "x")) as c:
        x, w, bias, z, R, D = _norm_args(x, w, bias, z, groups, act)
        dy = _need(dy, x, x.shape, "dy")
        dx = _out(dx, x, "dx")
        dw, dbias, dz = (torch.empty_like(t) if t is not None else None for t in (w, bias, z))
        dt = _dt(x)
        ws = _workspace(ws, _load().mi_group_norm_bwd_workspace(R, D, groups, dt), x.device)
        if c.side:
            c.keep(x, w, bias, z, dy, dx, dw, dbias, dz, ws)
        st = _load().mi_group_norm_bwd(x.data_ptr(), _ptr(w), _ptr(bias), _ptr(z), dy.data_ptr(), dx.data_ptr(),
                                       _ptr(dw), _ptr(dbias), _ptr(dz), R, D, groups, eps, int(bool(centered)),
                                       _act(act), dt, ws.data_ptr(), _nbytes(ws), c.handle)
        if st:
            _check(st, "mi_group_norm_bwd")
    return dx, dw, dbias, dz
