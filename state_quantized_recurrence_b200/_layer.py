"""Binding of the operators around and beside the gated delta rule
(``include/gdn_layer.h``): argument marshalling only, as in ``_binding``."""

from __future__ import annotations

import ctypes
import functools
import inspect

import torch

from ._binding import GDN_DTYPE, GdnError, _need, lib

GDN_ACT = {None: 0, "none": 0, "silu": 1}
GDN_NORM_OUT = {"none": 0, "fp8_row": 1, "int8_g32": 2, "int8_g16": 3, "int8_g64": 4}


def _declare() -> None:
    P, I, L, F, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                     ctypes.c_size_t)
    scan = [P, L, P, L, P, P, L, P, L, P, P]      # x, dt, A, B, C, D, dt_bias
    for name, args, res in (
            ("gdn_conv_prefill", [P, L, P, P, P, P] + [I] * 6 + [P, P, P], I),
            ("gdn_conv_decode", [P, L, P, P, P] + [I] * 5 + [P, P], I),
            ("gdn_conv_backward_workspace_bytes", [I] * 5, Z),
            ("gdn_conv_backward", [P, L, P, P, P, P] + [I] * 6 + [P, P, P, Z] + [P] * 5, I),
            ("gdn_scan_prefill_workspace_bytes", [I] * 8, Z),
            ("gdn_scan_prefill", scan + [P, P] + [I] * 7 + [P, Z, P, P, P], I),
            ("gdn_scan_decode", scan + [P] + [I] * 6 + [P, P], I),
            ("gdn_scan_backward_workspace_bytes", [I] * 8, Z),
            ("gdn_scan_backward", scan + [P, P] + [I] * 7 + [P, P, P, Z] + [P] * 9, I),
            ("gdn_norm", [P, L, P, L, P, L, P, L, I, I, F, I, I] + [P] * 4, I),
            ("gdn_norm_backward_workspace_bytes", [L, I, I], Z),
            ("gdn_norm_backward", [P, L, P, L, P, P, L, P, L, L, I, I, F, I, P, Z] + [P] * 4, I)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_declare()


# ------------------------------------------------------------------ checks ----
# Single-token calls are as short as their launch: messages are formatted
# only when they are raised, and the device is switched only when it differs.
def _device(*ts) -> int:
    """The index of the one CUDA device that holds every given tensor."""
    dev = -1
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("tensors must be CUDA tensors")
            if dev >= 0:
                raise ValueError(f"tensors on different devices (cuda:{dev} and cuda:{d})")
            dev = d
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _call(f, name: str, dev: int, stream, *args) -> None:
    """The C call on ``dev`` and on ``stream`` (default: the current stream
    of ``dev``), which has to be one of ``dev``."""
    _check_stream(stream, dev)
    if dev == torch.cuda.current_device():
        status = f(*args, _handle(stream, dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _handle(stream, dev))
    if status != 0:
        raise GdnError(status, name)


# The current stream's handle without a Stream object around it, where this
# torch has the call.
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _handle(stream, dev: int) -> int:
    return _current_raw(dev) if stream is None else stream.cuda_stream


def _check_stream(stream, dev: int) -> None:
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is of cuda:{stream.device_index}, the tensors are on cuda:{dev}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _f32(shape, name, t) -> None:
    if t is not None and not (t.dtype == torch.float32 and t.shape == shape
                              and t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous fp32 {list(shape)}")


def _token_stride(t: torch.Tensor, inner: int, name: str) -> int:
    """Elements between consecutive tokens of ``t``, whose last ``inner``
    dimensions are one token's contiguous row and whose leading ones are the
    tokens, equally far apart (a slice of a projection's output qualifies)."""
    shape = t.shape
    if t.is_contiguous():
        row = 1
        for d in shape[len(shape) - inner:]:
            row *= d
        return row
    strides, row = t.stride(), 1
    for d in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        if shape[d] != 1 and strides[d] != row:
            raise ValueError(f"{name}: a token's row must be contiguous")
        row *= shape[d]
    stride, span = None, 1
    for d in range(len(shape) - 1 - inner, -1, -1):
        if shape[d] == 1:
            continue
        if stride is None:
            stride = strides[d]
        if strides[d] != stride * span:
            raise ValueError(f"{name}: tokens must be equally far apart")
        span *= shape[d]
    if stride is None or row == 0 or span == 0:
        return row
    if stride < row:
        raise ValueError(f"{name}: tokens must not overlap")
    return stride


def _like(t, x, name) -> None:
    if not (t.shape == x.shape and t.dtype == x.dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous, x's shape and dtype")


def _sequences(lead, cu_seqlens):
    """(n_seq, T) of [B, T] leading dimensions."""
    if cu_seqlens is None:
        return lead[0], lead[1]
    _need(lead[0] == 1 and cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1
          and cu_seqlens.numel() >= 1 and cu_seqlens.is_contiguous(),
          "packed layout needs B == 1 and int32 cu_seqlens")
    return cu_seqlens.numel() - 1, lead[1]


def _streamed(f):
    """With a ``stream``, the whole call runs with it as the current one: the
    outputs and the workspace made here are then that stream's, and none of
    them is memory that another stream still works on."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream") if kw else None
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _new(shape, dtype, x, like):
    """An output on x's device; like ``like``, where a tensor of its shape
    and type is at hand (torch makes those in half the time).  The inputs that
    outputs are made like of are contiguous or refused, slices apart, whose
    likes are contiguous."""
    if like is not None and like.shape == shape and like.dtype == dtype:
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype, device=x.device)


def _scratch(need: int, workspace, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev)) if need else None
    _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(),
          "workspace must be a contiguous uint8 tensor")
    return workspace


# -------------------------------------------------------------------- conv ----
def _conv_args(x, weight, bias, state, lead_dims: int, activation, name):
    _need(activation in GDN_ACT, "activation must be 'silu' or 'none'")
    if x.dim() != lead_dims + 1:
        raise ValueError(f"{name}: x must have {lead_dims + 1} dimensions")
    _need(x.dtype in GDN_DTYPE, "x must be bf16 or fp32")
    C = x.shape[-1]
    _need(weight.dim() == 2 and weight.shape[0] == C, "weight must be [C, W]")
    W = weight.shape[1]
    _f32((C, W), "weight", weight)
    _f32((C,), "bias", bias)
    return C, W, _token_stride(x, 1, "x")


def _conv_state(t, shape, x, name):
    if t is not None and not (t.shape == shape and t.dtype == x.dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {list(shape)} in x's dtype")


def gdn_conv_prefill_into(x, weight, bias, state_in, cu_seqlens, y, state_out,
                          activation: str = "silu", stream=None) -> None:
    """gdn_conv_prefill into preallocated ``y`` and ``state_out`` (which may
    be ``state_in`` itself)."""
    dev = _device(x, weight, bias, state_in, cu_seqlens, y, state_out)
    C, W, xs = _conv_args(x, weight, bias, state_in, 2, activation, "gdn_conv_prefill")
    n, T = _sequences(x.shape[:2], cu_seqlens)
    shape = (n, W - 1, C)
    _conv_state(state_in, shape, x, "state_in")
    _need(state_out is not None, "state_out is needed")
    _conv_state(state_out, shape, x, "state_out")
    _like(y, x, "y")
    _call(lib.gdn_conv_prefill, "gdn_conv_prefill", dev, stream, _ptr(x), xs, _ptr(weight),
          _ptr(bias), _ptr(state_in), _ptr(cu_seqlens), n, T, C, W, GDN_DTYPE[x.dtype],
          GDN_ACT[activation], _ptr(y), _ptr(state_out))


@_streamed
def gdn_conv_prefill(x, weight, bias=None, state_in=None, cu_seqlens=None,
                     activation: str = "silu", stream=None):
    """Causal convolution of every channel: x [B, T, C] (packed: [1, T, C]
    with int32 ``cu_seqlens``), weight fp32 [C, W] with W = 2, 3 or 4, bias
    fp32 [C], state [n_seq, W - 1, C] (the last inputs, oldest first).  x may
    be a slice of wider rows.  Returns ``(y, state_out)``."""
    _need(x.dim() == 3 and weight.dim() == 2, "x must be [B, T, C], weight [C, W]")
    n, _ = _sequences(x.shape[:2], cu_seqlens)
    y = torch.empty_like(x)
    state_out = _new((n, weight.shape[-1] - 1, x.shape[-1]), x.dtype, x, state_in)
    gdn_conv_prefill_into(x, weight, bias, state_in, cu_seqlens, y, state_out, activation, stream)
    return y, state_out


def gdn_conv_decode_into(x, weight, bias, state, y, activation: str = "silu",
                         stream=None) -> None:
    """One token a sequence: x, y [N, C]; ``state`` [N, W - 1, C] moves up by
    one row in place."""
    dev = _device(x, weight, bias, state, y)
    C, W, xs = _conv_args(x, weight, bias, state, 1, activation, "gdn_conv_decode")
    _conv_state(state, (x.shape[0], W - 1, C), x, "state")
    _like(y, x, "y")
    _call(lib.gdn_conv_decode, "gdn_conv_decode", dev, stream, _ptr(x), xs, _ptr(weight),
          _ptr(bias), _ptr(state), x.shape[0], C, W, GDN_DTYPE[x.dtype], GDN_ACT[activation],
          _ptr(y))


@_streamed
def gdn_conv_decode(x, weight, bias, state, activation: str = "silu", stream=None):
    y = torch.empty_like(x)
    gdn_conv_decode_into(x, weight, bias, state, y, activation, stream)
    return y


@_streamed
def gdn_conv_backward(x, weight, dy, bias=None, state_in=None, cu_seqlens=None,
                      dstate_out=None, activation: str = "silu", workspace=None, stream=None):
    """Gradients of ``gdn_conv_prefill(x, weight, bias, state_in, cu_seqlens)``
    for ``dy`` and ``dstate_out`` (x's dtype, or None): ``(dx, dweight, dbias,
    dstate_in)``, dx and dstate_in in x's dtype, the weights' in fp32."""
    dev = _device(x, weight, bias, state_in, cu_seqlens, dy, dstate_out, workspace)
    C, W, xs = _conv_args(x, weight, bias, state_in, 2, activation, "gdn_conv_backward")
    n, T = _sequences(x.shape[:2], cu_seqlens)
    shape = (n, W - 1, C)
    _conv_state(state_in, shape, x, "state_in")
    _conv_state(dstate_out, shape, x, "dstate_out")
    _like(dy, x, "dy")
    need = int(lib.gdn_conv_backward_workspace_bytes(n, T, C, W, int(cu_seqlens is not None)))
    ws = _scratch(need, workspace, dev)
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight)
    db = _new((C,), torch.float32, x, bias)
    ds = _new(shape, x.dtype, x, state_in)
    _call(lib.gdn_conv_backward, "gdn_conv_backward", dev, stream, _ptr(x), xs, _ptr(weight),
          _ptr(bias), _ptr(state_in), _ptr(cu_seqlens), n, T, C, W, GDN_DTYPE[x.dtype],
          GDN_ACT[activation], _ptr(dy), _ptr(dstate_out), _ptr(ws), 0 if ws is None else
          ws.numel(), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ds))
    return dx, dw, db, ds


# -------------------------------------------------------------------- scan ----
def _scan_args(x, dt, A, B, C, D, dt_bias, lead: int, name):
    if not (x.dim() == lead + 2 and B.dim() == lead + 2 and C.shape == B.shape
            and dt.dim() == lead + 1):
        raise ValueError(f"{name}: x [.., H, P], dt [.., H], B and C [.., G, N]")
    H, P = x.shape[-2:]
    G, N = B.shape[-2:]
    _need(x.shape[:lead] == B.shape[:lead] and dt.shape == x.shape[:-1],
          "x, dt, B and C must have the same tokens and heads")
    _need(x.dtype in GDN_DTYPE and dt.dtype == x.dtype and B.dtype == x.dtype
          and C.dtype == x.dtype, "x, dt, B and C must share dtype bf16 or fp32")
    _need(G > 0 and H % G == 0, "H must be a multiple of G")
    _need(A is not None, "A is needed")
    for t, n in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
        _f32((H,), n, t)
    args = (_ptr(x), _token_stride(x, 2, "x"), _ptr(dt), _token_stride(dt, 1, "dt"), _ptr(A),
            _ptr(B), _token_stride(B, 2, "B"), _ptr(C), _token_stride(C, 2, "C"), _ptr(D),
            _ptr(dt_bias))
    return H, P, G, N, args


@_streamed
def gdn_scan_prefill_into(x, dt, A, B, C, D, dt_bias, state_in, cu_seqlens, y, state_out,
                          workspace=None, stream=None) -> None:
    """gdn_scan_prefill into preallocated ``y`` and ``state_out`` (which may
    be ``state_in`` itself).  ``workspace``: a CUDA uint8 tensor of
    gdn_scan_prefill_workspace_bytes(...) bytes, or None to allocate it."""
    dev = _device(x, dt, A, B, C, D, dt_bias, state_in, cu_seqlens, y, state_out, workspace)
    H, P, G, N, args = _scan_args(x, dt, A, B, C, D, dt_bias, 2, "gdn_scan_prefill")
    n, T = _sequences(x.shape[:2], cu_seqlens)
    _f32((n, H, N, P), "state_in", state_in)
    _need(state_out is not None, "state_out is needed")
    _f32((n, H, N, P), "state_out", state_out)
    _like(y, x, "y")
    need = int(lib.gdn_scan_prefill_workspace_bytes(n, T, H, P, G, N, GDN_DTYPE[x.dtype],
                                                    int(cu_seqlens is not None)))
    ws = _scratch(need, workspace, dev)
    _call(lib.gdn_scan_prefill, "gdn_scan_prefill", dev, stream, *args, _ptr(state_in),
          _ptr(cu_seqlens), n, T, H, P, G, N, GDN_DTYPE[x.dtype], _ptr(ws), 0 if ws is None else
          ws.numel(), _ptr(y), _ptr(state_out))


@_streamed
def gdn_scan_prefill(x, dt, A, B, C, D=None, dt_bias=None, state_in=None, cu_seqlens=None,
                     workspace=None, stream=None):
    """Selective state space scan, one decay a head: x [B, T, H, P], dt
    [B, T, H] (before its softplus), B, C [B, T, G, N] (packed: B == 1 and
    int32 ``cu_seqlens``), all bf16 or all fp32 and each possibly a slice of
    wider rows; A, D, dt_bias fp32 [H]; states fp32 [n_seq, H, N, P].
    Returns ``(y, state_out)``."""
    _need(x.dim() == 4 and B.dim() == 4, "x must be [B, T, H, P], B and C [B, T, G, N]")
    n, _ = _sequences(x.shape[:2], cu_seqlens)
    y = torch.empty_like(x)
    state_out = _new((n, x.shape[2], B.shape[-1], x.shape[3]), torch.float32, x, state_in)
    gdn_scan_prefill_into.__wrapped__(  # the stream is the current one already
        x, dt, A, B, C, D, dt_bias, state_in, cu_seqlens, y, state_out, workspace, stream)
    return y, state_out


def gdn_scan_decode_into(x, dt, A, B, C, state, y, D=None, dt_bias=None, stream=None) -> None:
    """One token a sequence: x, y [n, H, P], dt [n, H], B, C [n, G, N];
    ``state`` fp32 [n, H, N, P] is advanced in place."""
    dev = _device(x, dt, A, B, C, D, dt_bias, state, y)
    H, P, G, N, args = _scan_args(x, dt, A, B, C, D, dt_bias, 1, "gdn_scan_decode")
    n = x.shape[0]
    _need(state is not None, "state is needed")
    _f32((n, H, N, P), "state", state)
    _like(y, x, "y")
    _call(lib.gdn_scan_decode, "gdn_scan_decode", dev, stream, *args, _ptr(state), n, H, P, G,
          N, GDN_DTYPE[x.dtype], _ptr(y))


@_streamed
def gdn_scan_decode(x, dt, A, B, C, state, D=None, dt_bias=None, stream=None):
    y = torch.empty_like(x)
    gdn_scan_decode_into(x, dt, A, B, C, state, y, D, dt_bias, stream)
    return y


@_streamed
def gdn_scan_backward(x, dt, A, B, C, dy, D=None, dt_bias=None, state_in=None, cu_seqlens=None,
                      dstate_out=None, workspace=None, stream=None):
    """Gradients of ``gdn_scan_prefill`` for ``dy`` (y's shape and dtype) and
    ``dstate_out`` (fp32, or None): ``(dx, ddt, dA, dB, dC, dD, ddt_bias,
    dstate_in)``; dx, ddt, dB and dC in x's dtype, the others fp32."""
    dev = _device(x, dt, A, B, C, D, dt_bias, state_in, cu_seqlens, dy, dstate_out, workspace)
    H, P, G, N, args = _scan_args(x, dt, A, B, C, D, dt_bias, 2, "gdn_scan_backward")
    n, T = _sequences(x.shape[:2], cu_seqlens)
    _f32((n, H, N, P), "state_in", state_in)
    _f32((n, H, N, P), "dstate_out", dstate_out)
    _like(dy, x, "dy")
    need = int(lib.gdn_scan_backward_workspace_bytes(n, T, H, P, G, N, GDN_DTYPE[x.dtype],
                                                     int(cu_seqlens is not None)))
    ws = _scratch(need, workspace, dev)
    dx, ddt = torch.empty_like(x), torch.empty_like(dt)
    dB, dC = torch.empty_like(B), torch.empty_like(B)
    dA, dD, db = torch.empty_like(A), torch.empty_like(A), torch.empty_like(A)
    ds = _new((n, H, N, P), torch.float32, x, state_in)
    _call(lib.gdn_scan_backward, "gdn_scan_backward", dev, stream, *args, _ptr(state_in),
          _ptr(cu_seqlens), n, T, H, P, G, N, GDN_DTYPE[x.dtype], _ptr(dy), _ptr(dstate_out),
          _ptr(ws), 0 if ws is None else ws.numel(), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB),
          _ptr(dC), _ptr(dD), _ptr(db), _ptr(ds))
    return dx, ddt, dA, dB, dC, dD, db, ds


# -------------------------------------------------------------------- norm ----
class QuantizedRows:
    """Rows held in 8 bits: ``codes`` (float8_e4m3fn for "fp8_row", int8 for
    the INT8 groups) in the rows' shape, and fp32 ``scales``: one a row
    ([..]) or one a group ([.., d / G]).  A value is code * scale."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, qdq: str):
        self.codes, self.scales, self.qdq = codes, scales, qdq

    @property
    def shape(self):
        return tuple(self.codes.shape)

    def dequantize(self) -> torch.Tensor:
        """The fp32 values (plain torch; for checks and for reading results)."""
        c = self.codes.float()
        if self.qdq == "fp8_row":
            return c * self.scales[..., None]
        g = int(self.qdq.split("_g")[1])
        return (c.unflatten(-1, (-1, g)) * self.scales[..., None]).flatten(-2)


def _norm_rows(x, *others):
    """(tokens, heads, strides): rows one by one where every tensor's rows
    are equally far apart, else tokens of shape[-2] contiguous heads."""
    ts = (x,) + others
    for t in others:
        _need(t is None or (t.shape == x.shape and t.dtype == x.dtype),
              "the row tensors must share x's shape and dtype")
    rows = x.numel() // x.shape[-1] if x.shape[-1] else 0
    try:
        return rows, 1, [0 if t is None else _token_stride(t, 1, "rows") for t in ts]
    except ValueError:
        if x.dim() < 3:
            raise
    h = x.shape[-2]
    return rows // h, h, [0 if t is None else _token_stride(t, 2, "rows") for t in ts]


@_streamed
def gdn_norm(x, weight, residual=None, gate=None, eps: float = 1e-6, qdq: str = "none",
             stream=None):
    """RMS norm of the rows of x [.., d]: s = x + residual (rounded to x's
    dtype), y = s / sqrt(mean(s^2) + eps) * weight * silu(gate).  x, residual
    and gate share shape and dtype (bf16 or fp32) and may be slices of wider
    rows, also [.., heads, d] slices whose heads are contiguous; weight fp32
    [d].  ``qdq``: "none" returns y in x's dtype, "fp8_row", "int8_g16",
    "int8_g32" or "int8_g64" a QuantizedRows.  A row of zeros is one of zeros
    for eps = 0 too.  Returns ``(y, s)``, s None without a residual."""
    dev = _device(x, weight, residual, gate)
    _need(qdq in GDN_NORM_OUT, "qdq must be 'none', 'fp8_row' or 'int8_g16/32/64'")
    _need(x.dim() >= 1 and x.dtype in GDN_DTYPE, "x must be bf16 or fp32 [.., d]")
    d = x.shape[-1]
    _f32((d,), "weight", weight)
    tokens, heads, (xs, rs, gs) = _norm_rows(x, residual, gate)
    scales = None
    if qdq == "none":
        y = torch.empty_like(x)
    elif qdq == "fp8_row":
        y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        scales = _new(x.shape[:-1], torch.float32, x, None)
    else:
        group = int(qdq.split("_g")[1])
        _need(d % group == 0, "d must be a multiple of the group")
        y = torch.empty_like(x, dtype=torch.int8)
        scales = _new(x.shape[:-1] + (d // group,), torch.float32, x, None)
    s = None if residual is None else torch.empty_like(x)
    _call(lib.gdn_norm, "gdn_norm", dev, stream, _ptr(x), xs, _ptr(residual), rs, _ptr(gate),
          gs, _ptr(weight), tokens, heads, d, float(eps), GDN_DTYPE[x.dtype], GDN_NORM_OUT[qdq],
          _ptr(y), _ptr(scales), _ptr(s))
    return (y if scales is None else QuantizedRows(y, scales, qdq)), s


@_streamed
def gdn_norm_backward(x, weight, dy, gate=None, dresidual=None, eps: float = 1e-6,
                      workspace=None, stream=None):
    """Gradients of ``gdn_norm`` at x (the s it returned, or its x) for
    ``dy`` and ``dresidual`` (the gradient reaching s from elsewhere):
    ``(dx, dweight, dgate)``, dx and dgate in x's dtype, dweight fp32, dgate
    None without a gate.  An 8-bit output passes its gradient straight
    through."""
    dev = _device(x, weight, dy, gate, dresidual, workspace)
    _need(x.dim() >= 1 and x.dtype in GDN_DTYPE, "x must be bf16 or fp32 [.., d]")
    d = x.shape[-1]
    _f32((d,), "weight", weight)
    _need(dy is not None, "dy is needed")
    tokens, heads, (xs, ys, gs, rs) = _norm_rows(x, dy, gate, dresidual)
    ws = _scratch(int(lib.gdn_norm_backward_workspace_bytes(tokens, heads, d)), workspace, dev)
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight)
    dg = None if gate is None else torch.empty_like(x)
    _call(lib.gdn_norm_backward, "gdn_norm_backward", dev, stream, _ptr(x), xs, _ptr(gate), gs,
          _ptr(weight), _ptr(dy), ys, _ptr(dresidual), rs, tokens, heads, d, float(eps),
          GDN_DTYPE[x.dtype], _ptr(ws), 0 if ws is None else ws.numel(), _ptr(dx), _ptr(dw),
          _ptr(dg))
    return dx, dw, dg
