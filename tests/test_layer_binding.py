"""The layer operators' binding on the host: what it refuses before anything
is launched (no GPU needed)."""

import pytest
import torch

from test_layer_host import lib  # noqa: F401  (builds the library, then imports it)


class OtherStream:
    """A stream of device 1 (torch makes its fields from the driver's)."""
    device_index = 1
    device = torch.device("cuda", 1)
    cuda_stream = 0x1234


def calls(lib, **kw):
    """Every entry point that takes a stream, with arguments that are right."""
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    st = torch.zeros(2, 3, 8)
    q, dt, A = torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 2), torch.zeros(2)
    B, ss = torch.zeros(2, 5, 1, 64), torch.zeros(2, 2, 64, 64)
    r, rw = torch.zeros(4, 8), torch.zeros(8)
    scan = (q, dt, A, B, B)
    token = (q[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], ss)
    return {
        "conv_prefill": lambda: lib.gdn_conv_prefill(x, w, **kw),
        "conv_prefill_into": lambda: lib.gdn_conv_prefill_into(
            x, w, None, None, None, torch.empty_like(x), st, **kw),
        "conv_decode": lambda: lib.gdn_conv_decode(x[:, 0], w, None, st, **kw),
        "conv_decode_into": lambda: lib.gdn_conv_decode_into(
            x[:, 0], w, None, st, torch.zeros(2, 8), **kw),
        "conv_backward": lambda: lib.gdn_conv_backward(x, w, x, **kw),
        "scan_prefill": lambda: lib.gdn_scan_prefill(*scan, **kw),
        "scan_prefill_into": lambda: lib.gdn_scan_prefill_into(
            *scan, None, None, None, None, torch.empty_like(q), ss, **kw),
        "scan_decode": lambda: lib.gdn_scan_decode(*token, **kw),
        "scan_decode_into": lambda: lib.gdn_scan_decode_into(*token, torch.zeros(2, 2, 64), **kw),
        "scan_backward": lambda: lib.gdn_scan_backward(*scan, q, **kw),
        "norm": lambda: lib.gdn_norm(r, rw, **kw),
        "norm_backward": lambda: lib.gdn_norm_backward(r, rw, r, **kw),
    }


NAMES = ["conv_prefill", "conv_prefill_into", "conv_decode", "conv_decode_into", "conv_backward",
         "scan_prefill", "scan_prefill_into", "scan_decode", "scan_decode_into", "scan_backward",
         "norm", "norm_backward"]


@pytest.fixture
def on_device_0(monkeypatch):
    """CPU tensors pass for ones of cuda:0; no call gets as far as the library."""
    from state_quantized_recurrence_b200 import _layer
    monkeypatch.setattr(_layer, "_device", lambda *ts: 0)
    monkeypatch.setattr(_layer, "_scratch", lambda need, ws, dev: ws)
    return _layer


@pytest.mark.parametrize("name", NAMES)
def test_stream_of_another_device_is_refused(lib, on_device_0, name):  # noqa: F811
    """Not dropped for the device's current stream."""
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        calls(lib, stream=OtherStream())[name]()


def test_wrong_ranks_are_refused(lib, on_device_0):  # noqa: F811
    """With a ValueError that says what is wanted, as every other argument."""
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    q, dt, A, B = torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 2), torch.zeros(2), \
        torch.zeros(2, 5, 1, 64)
    cu = torch.zeros(3, dtype=torch.int32)
    for f in (lambda: lib.gdn_conv_prefill(x[0], w), lambda: lib.gdn_conv_prefill(x[0, 0], w),
              lambda: lib.gdn_conv_prefill(x, w[0]), lambda: lib.gdn_conv_prefill(x, w[0, 0]),
              lambda: lib.gdn_conv_prefill(x[0, 0], w, cu_seqlens=cu),
              lambda: lib.gdn_conv_decode(x, w, None, x),
              lambda: lib.gdn_conv_backward(x[0, 0], w, x),
              lambda: lib.gdn_scan_prefill(q[0], dt[0], A, B[0], B[0]),
              lambda: lib.gdn_scan_prefill(q[0, 0, 0], dt, A, B, B),
              lambda: lib.gdn_scan_prefill(q, dt, A, B[0, 0, 0, 0], B),
              lambda: lib.gdn_scan_prefill(q, dt, A, B, B[0]),
              lambda: lib.gdn_scan_backward(q[0], dt[0], A, B[0], B[0], q[0]),
              lambda: lib.gdn_scan_decode(q, dt, A, B, B, q),
              lambda: lib.gdn_norm(x[0, 0, 0], w[0]),
              lambda: lib.gdn_norm_backward(x[0, 0, 0], w[0], x[0, 0, 0])):
        with pytest.raises(ValueError):
            f()


def test_scan_runs_by_units(lib):  # noqa: F811
    """Prompts are cut into runs below 100 units, gradients below 50 (either
    side measured beside the rule); a gradient that is not cut has room for
    the chunks' states and adjoints and the heads' sums alone."""
    T, P, N = 4096, 64, 128
    chunks, state = T // 64, N * P * 4
    for H in (1, 48, 49, 50, 64, 99, 100, 128):
        prompt = lib.lib.gdn_scan_prefill_workspace_bytes(1, T, H, P, H, N, 1, 0)
        assert (prompt > 0) == (H < 100)
        grad = lib.lib.gdn_scan_backward_workspace_bytes(1, T, H, P, H, N, 1, 0)
        whole = 2 * chunks * H * state + 2 * T * H * N * 4 + chunks * H * 16
        assert (grad > whole) == (H < 50) and (H < 50 or grad == whole)
