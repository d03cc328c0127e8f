"""B200 (sm_100a) gated delta rule with a fake-quantized recurrent state.

Thin Python binding over the C ABI in ``include/gdn_qdq.h``: it only checks
and marshals arguments (device pointers, sizes, the current CUDA stream);
every step of the computation runs in the library's CUDA kernels.  There is
no CPU or PyTorch fallback - importing this package fails if the compiled
library is missing.

    o, state = gdn_prefill(q, k, v, g, beta, state_in=None, cu_seqlens=None,
                           qdq="fp8_tile64")
    o, state = gdn_prefill(..., neumann_degree=7)   # approximate solve, 2^m - 1
    o, state = gdn_prefill(..., w_qdq="fp8_row")    # + FP8 QDQ of W, a scale per row
    gdn_prefill_schedule(n_seq, H, d_k, d_v)        # which prefill kernel runs
    o = gdn_decode(q, k, v, g, beta, state, qdq="int8_g32")   # state in place
    dq, dk, dv, dg, dbeta, dstate_in = gdn_prefill_backward(q, k, v, g, beta, d_o, ...)

Packed state storage (codes + scales instead of fp32 QDQ values):

    ps = gdn_state_pack(state, qdq="int8_g32")
    o = gdn_decode_packed(q, k, v, g, beta, ps)                # ps in place
    state = gdn_state_unpack(ps)

What stands around and beside the recurrence in a layer (``include/gdn_layer.h``):

    y, state = gdn_conv_prefill(x, weight, bias, state_in=None, cu_seqlens=None)
    y = gdn_conv_decode(x, weight, bias, state)                # state in place
    dx, dweight, dbias, dstate_in = gdn_conv_backward(x, weight, dy, bias, ...)
    y, state = gdn_scan_prefill(x, dt, A, B, C, D=None, dt_bias=None, ...)
    y = gdn_scan_decode(x, dt, A, B, C, state, D=None, dt_bias=None)
    dx, ddt, dA, dB, dC, dD, ddt_bias, dstate_in = gdn_scan_backward(x, dt, A, B, C, dy, ...)
    y, s = gdn_norm(x, weight, residual=None, gate=None, qdq="fp8_row")
    dx, dweight, dgate = gdn_norm_backward(s, weight, dy, gate=None, dresidual=None)
"""

from __future__ import annotations

from ._binding import (  # noqa: F401
    GDN_DTYPE, GDN_GATE, GDN_QDQ, GDN_STATUS, GDN_W_QDQ, GdnError, check_last_error,
    PackedState, gdn_decode, gdn_decode_into, gdn_decode_packed, gdn_decode_packed_into,
    gdn_last_error, gdn_prefill, gdn_prefill_backward, gdn_prefill_backward_static,
    gdn_prefill_into, gdn_prefill_schedule,
    gdn_state_pack, gdn_state_unpack, lib, library_path, packed_state_empty,
)
from ._layer import (  # noqa: F401
    GDN_ACT, GDN_NORM_OUT, QuantizedRows, gdn_conv_backward, gdn_conv_decode,
    gdn_conv_decode_into, gdn_conv_prefill, gdn_conv_prefill_into, gdn_norm, gdn_norm_backward,
    gdn_scan_backward, gdn_scan_decode, gdn_scan_decode_into, gdn_scan_prefill,
    gdn_scan_prefill_into,
)

__all__ = [
    "gdn_prefill", "gdn_prefill_into", "gdn_prefill_backward", "gdn_prefill_backward_static",
    "gdn_prefill_schedule",
    "gdn_decode", "gdn_decode_into",
    "gdn_decode_packed", "gdn_decode_packed_into", "gdn_state_pack", "gdn_state_unpack",
    "PackedState", "packed_state_empty",
    "gdn_conv_prefill", "gdn_conv_prefill_into", "gdn_conv_decode", "gdn_conv_decode_into",
    "gdn_conv_backward",
    "gdn_scan_prefill", "gdn_scan_prefill_into", "gdn_scan_decode", "gdn_scan_decode_into",
    "gdn_scan_backward",
    "gdn_norm", "gdn_norm_backward", "QuantizedRows",
    "gdn_last_error", "check_last_error", "GdnError", "library_path", "lib",
    "GDN_QDQ", "GDN_W_QDQ", "GDN_DTYPE", "GDN_GATE", "GDN_STATUS",
    "GDN_ACT", "GDN_NORM_OUT",
]
