"""Host-only checks of the layer operators' C ABI and binding (no GPU needed,
nothing is launched): argument errors come back with the documented status
before any CUDA call, workspace sizes follow their formulas, empty batches are
no-ops, and the binding refuses what it cannot pass on."""

import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16, F32 = 0, 1
A = 0x10000  # a 16-byte aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "state_quantized_recurrence_b200_build",
        os.path.join(root, "state_quantized_recurrence_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    build.build()
    import state_quantized_recurrence_b200 as sqr
    return sqr


def conv(lib, **kw):
    a = dict(x=A, xs=64, w=A, b=A, si=None, cu=None, n=2, T=9, C=64, W=4, dt=BF16, act=1, y=A,
             so=A)
    a.update(kw)
    return lib.lib.gdn_conv_prefill(a["x"], a["xs"], a["w"], a["b"], a["si"], a["cu"], a["n"],
                                    a["T"], a["C"], a["W"], a["dt"], a["act"], a["y"], a["so"],
                                    None)


def conv_token(lib, **kw):
    a = dict(x=A, xs=64, w=A, b=A, s=A, n=2, C=64, W=4, dt=BF16, act=1, y=A)
    a.update(kw)
    return lib.lib.gdn_conv_decode(a["x"], a["xs"], a["w"], a["b"], a["s"], a["n"], a["C"], a["W"],
                                   a["dt"], a["act"], a["y"], None)


def conv_grad(lib, ws_bytes=None, **kw):
    a = dict(x=A, xs=64, w=A, b=A, si=None, cu=None, n=2, T=9, C=64, W=4, dt=BF16, act=1, dy=A,
             dso=None, ws=A, dx=A, dw=A, db=A, dsi=A)
    a.update(kw)
    need = lib.lib.gdn_conv_backward_workspace_bytes(a["n"], a["T"], a["C"], a["W"],
                                                     int(a["cu"] is not None))
    return lib.lib.gdn_conv_backward(
        a["x"], a["xs"], a["w"], a["b"], a["si"], a["cu"], a["n"], a["T"], a["C"], a["W"], a["dt"],
        a["act"], a["dy"], a["dso"], a["ws"], need if ws_bytes is None else ws_bytes, a["dx"],
        a["dw"], a["db"], a["dsi"], None)


@pytest.mark.parametrize("call", [conv, conv_token, conv_grad])
def test_conv_errors(lib, call):
    assert call(lib, n=-1) == INVALID
    assert call(lib, C=0) == INVALID
    assert call(lib, xs=63) == INVALID               # tokens would overlap
    assert call(lib, W=1) == UNSUPPORTED
    assert call(lib, W=5) == UNSUPPORTED
    assert call(lib, dt=7) == UNSUPPORTED
    assert call(lib, act=2) == UNSUPPORTED
    assert call(lib, x=None) == INVALID
    assert call(lib, w=None) == INVALID
    assert call(lib, w=A + 2) == INVALID
    assert call(lib, x=A + 1) == INVALID             # an element's own alignment
    if call is not conv_grad:
        assert call(lib, n=0) == OK
        assert call(lib, y=None) == INVALID


def test_conv_specific_errors(lib):
    assert conv(lib, T=-1) == INVALID
    assert conv(lib, so=None) == INVALID
    assert conv(lib, cu=A + 2) == INVALID
    assert conv_token(lib, s=None) == INVALID
    assert conv_grad(lib, ws=None) == INVALID
    assert conv_grad(lib, ws=A + 4) == INVALID
    assert conv_grad(lib, ws_bytes=8) == INVALID
    for name in ("dx", "dw", "db", "dsi", "dy"):
        assert conv_grad(lib, **{name: None}) == INVALID
    # one partial row of W + 1 sums for every tile of 128 tokens
    size = lib.lib.gdn_conv_backward_workspace_bytes
    assert size(2, 129, 64, 4, 0) == 2 * 2 * 5 * 64 * 4
    assert size(3, 300, 64, 2, 1) == (3 + 300 // 128) * 3 * 64 * 4
    assert size(1, 0, 64, 4, 0) == 5 * 64 * 4
    assert size(0, 9, 64, 4, 0) == 0 and size(1, 9, 64, 5, 0) == 0


SCAN = dict(x=A, xs=256, raw=A, rs=4, A=A, B=A, bs=128, C=A, cs=128, D=A, bias=A)


def scan_head(a):
    return [a[k] for k in ("x", "xs", "raw", "rs", "A", "B", "bs", "C", "cs", "D", "bias")]


def scan(lib, **kw):
    a = dict(SCAN, si=None, cu=None, n=2, T=70, H=4, P=64, G=1, N=128, dt=BF16, ws=A, y=A, so=A)
    a.update(kw)
    need = lib.lib.gdn_scan_prefill_workspace_bytes(a["n"], a["T"], a["H"], a["P"], a["G"], a["N"],
                                                    a["dt"], int(a["cu"] is not None))
    return lib.lib.gdn_scan_prefill(*scan_head(a), a["si"], a["cu"], a["n"], a["T"], a["H"], a["P"],
                                    a["G"], a["N"], a["dt"], a["ws"], a.get("ws_bytes", need),
                                    a["y"], a["so"], None)


def scan_token(lib, **kw):
    a = dict(SCAN, s=A, n=2, H=4, P=64, G=1, N=128, dt=BF16, y=A)
    a.update(kw)
    return lib.lib.gdn_scan_decode(*scan_head(a), a["s"], a["n"], a["H"], a["P"], a["G"], a["N"],
                                   a["dt"], a["y"], None)


def scan_grad(lib, **kw):
    a = dict(SCAN, si=None, cu=None, n=2, T=70, H=4, P=64, G=1, N=128, dt=BF16, dy=A, dso=None,
             ws=A, dx=A, ddt=A, dA=A, dB=A, dC=A, dD=A, db=A, dsi=A)
    a.update(kw)
    need = lib.lib.gdn_scan_backward_workspace_bytes(a["n"], a["T"], a["H"], a["P"], a["G"],
                                                     a["N"], a["dt"], int(a["cu"] is not None))
    return lib.lib.gdn_scan_backward(
        *scan_head(a), a["si"], a["cu"], a["n"], a["T"], a["H"], a["P"], a["G"], a["N"], a["dt"],
        a["dy"], a["dso"], a["ws"], a.get("ws_bytes", need), a["dx"], a["ddt"], a["dA"], a["dB"],
        a["dC"], a["dD"], a["db"], a["dsi"], None)


@pytest.mark.parametrize("call", [scan, scan_token, scan_grad])
def test_scan_errors(lib, call):
    assert call(lib, n=-1) == INVALID
    assert call(lib, H=0) == INVALID
    assert call(lib, G=3) == INVALID                 # heads do not divide into the groups
    assert call(lib, G=0) == INVALID
    assert call(lib, P=96) == UNSUPPORTED
    assert call(lib, N=256) == UNSUPPORTED
    assert call(lib, N=16) == UNSUPPORTED
    assert call(lib, dt=9) == UNSUPPORTED
    assert call(lib, A=None) == INVALID
    for name in ("x", "B", "C", "raw"):
        assert call(lib, **{name: None}) == INVALID
    for name in ("x", "B", "C"):
        assert call(lib, **{name: A + 8}) == INVALID  # 16-byte alignment
    assert call(lib, raw=A + 1) == INVALID
    assert call(lib, xs=260) == INVALID              # rows that leave the 16-byte grid
    assert call(lib, bs=120) == INVALID              # tokens would overlap
    assert call(lib, cs=132) == INVALID
    assert call(lib, rs=3) == INVALID
    assert call(lib, D=A + 2) == INVALID
    if call is not scan_grad:
        assert call(lib, n=0) == OK
        assert call(lib, y=None) == INVALID
        assert call(lib, y=A + 8) == INVALID


def test_scan_specific_errors(lib):
    assert scan(lib, T=-1) == INVALID
    assert scan(lib, T=0x7fffff80, n=1) == UNSUPPORTED
    assert scan(lib, so=None) == INVALID
    assert scan(lib, si=A + 4) == INVALID
    assert scan(lib, cu=A + 2) == INVALID
    assert scan_token(lib, s=None) == INVALID
    assert scan_grad(lib, ws=None) == INVALID
    assert scan_grad(lib, ws_bytes=64) == INVALID
    assert scan_grad(lib, dso=A + 4) == INVALID
    for name in ("dy", "dx", "ddt", "dA", "dB", "dC", "dD", "db", "dsi"):
        assert scan_grad(lib, **{name: None}) == INVALID
    # a long sequence of few heads is cut into runs and needs their states
    assert scan(lib, n=1, T=8192, H=1, G=1, xs=64, rs=1, ws=None) == INVALID
    assert scan(lib, n=1, T=8192, H=1, G=1, xs=64, rs=1, ws_bytes=4) == INVALID


def test_scan_workspaces(lib):
    size = lib.lib.gdn_scan_prefill_workspace_bytes
    assert size(2, 70, 4, 64, 1, 128, BF16, 0) == 0            # two chunks a sequence
    assert size(256, 8192, 32, 64, 1, 128, BF16, 0) == 0       # units enough for every SM
    # 128 chunks in 32 runs of four: a state and a decay a run (16-byte steps)
    for dtype in (BF16, F32):
        assert size(1, 8192, 1, 64, 1, 128, dtype, 0) == 32 * 128 * 64 * 4 + 32 * 4
    assert size(1, 8192, 1, 96, 1, 128, BF16, 0) == 0
    back = lib.lib.gdn_scan_backward_workspace_bytes
    # fp32: states and adjoints of 2 x 2 chunks, dB and dC of every head, parts
    assert back(2, 70, 4, 64, 1, 128, F32, 0) == \
        2 * (4 * 4 * 128 * 64 * 4) + 2 * (140 * 4 * 128 * 4) + 4 * 4 * 16
    assert back(0, 70, 4, 64, 1, 128, F32, 0) == 0


def norm(lib, **kw):
    a = dict(x=A, xs=128, r=None, rs=0, g=None, gs=0, w=A, tokens=3, heads=1, d=128, eps=1e-6,
             dt=BF16, out=0, y=A, s=None, ro=None)
    a.update(kw)
    return lib.lib.gdn_norm(a["x"], a["xs"], a["r"], a["rs"], a["g"], a["gs"], a["w"], a["tokens"],
                            a["heads"], a["d"], a["eps"], a["dt"], a["out"], a["y"], a["s"],
                            a["ro"], None)


def norm_grad(lib, **kw):
    a = dict(x=A, xs=128, g=None, gs=0, w=A, dy=A, ys=128, dr=None, drs=0, tokens=3, heads=1,
             d=128, eps=1e-6, dt=BF16, ws=A, dx=A, dw=A, dg=None)
    a.update(kw)
    need = lib.lib.gdn_norm_backward_workspace_bytes(a["tokens"], a["heads"], a["d"])
    return lib.lib.gdn_norm_backward(
        a["x"], a["xs"], a["g"], a["gs"], a["w"], a["dy"], a["ys"], a["dr"], a["drs"], a["tokens"],
        a["heads"], a["d"], a["eps"], a["dt"], a["ws"], a.get("ws_bytes", need), a["dx"], a["dw"],
        a["dg"], None)


@pytest.mark.parametrize("call", [norm, norm_grad])
def test_norm_errors(lib, call):
    assert call(lib, tokens=-1) == INVALID
    assert call(lib, heads=0) == INVALID
    assert call(lib, d=0) == INVALID
    assert call(lib, eps=-1.0) == INVALID
    assert call(lib, eps=float("nan")) == INVALID
    assert call(lib, dt=5) == UNSUPPORTED
    assert call(lib, x=None) == INVALID
    assert call(lib, w=None) == INVALID
    assert call(lib, xs=127) == INVALID              # rows would overlap
    assert call(lib, heads=2, xs=128) == INVALID     # a token holds two rows
    assert call(lib, x=A + 1) == INVALID
    assert call(lib, w=A + 2) == INVALID
    assert call(lib, g=A, gs=100) == INVALID


def test_norm_specific_errors(lib):
    assert norm(lib, tokens=0) == OK
    assert norm(lib, y=None) == INVALID
    assert norm(lib, out=9) == UNSUPPORTED
    assert norm(lib, out=1) == INVALID               # 8 bits need scales
    assert norm(lib, out=2, s=A, d=100, xs=100) == INVALID
    assert norm(lib, out=2, s=A, xs=129) == INVALID  # INT8 groups need aligned rows
    assert norm(lib, r=A, rs=128) == INVALID         # residual and its sum come together
    assert norm(lib, ro=A) == INVALID
    assert norm(lib, d=8193, xs=8193) == UNSUPPORTED
    assert norm(lib, d=40000, xs=40000) == UNSUPPORTED
    assert norm_grad(lib, dw=None) == INVALID
    assert norm_grad(lib, dx=None) == INVALID
    assert norm_grad(lib, g=A, gs=128) == INVALID    # a gate and its gradient come together
    assert norm_grad(lib, ws=None) == INVALID
    assert norm_grad(lib, ws_bytes=4) == INVALID
    size = lib.lib.gdn_norm_backward_workspace_bytes
    assert size(3, 1, 128) == 3 * 128 * 4 and size(1 << 20, 2, 64) == 148 * 4 * 64 * 4
    assert size(0, 1, 128) == 0


def test_binding_refuses(lib):
    """What never reaches the library: tensors on the CPU, wrong shapes and
    types, tokens that are not equally far apart or that overlap."""
    x = torch.zeros(2, 5, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError):
        lib.gdn_conv_prefill(x, w)
    with pytest.raises(ValueError):
        lib.gdn_norm(x, torch.zeros(8))
    with pytest.raises(ValueError):
        lib.gdn_norm(x, torch.zeros(8), qdq="fp4")
    from state_quantized_recurrence_b200 import _layer
    assert _layer._token_stride(torch.zeros(3, 4, 6)[..., :5], 1, "x") == 6
    assert _layer._token_stride(torch.zeros(3, 4, 2, 5), 2, "x") == 10
    assert _layer._token_stride(torch.zeros(1, 4, 8)[:, :1], 1, "x") == 8
    assert _layer._token_stride(torch.zeros(0, 4, 8), 1, "x") == 8
    for bad in (torch.zeros(3, 4, 6)[:, :3], torch.zeros(3, 4, 6).transpose(1, 2),
                torch.zeros(4, 6).t(), torch.zeros(1, 6).expand(4, 6),
                torch.zeros(4, 12)[:, ::2], torch.zeros(3, 4, 6).transpose(0, 1)):
        with pytest.raises(ValueError):
            _layer._token_stride(bad, 1, "x")
    assert _layer._norm_rows(torch.zeros(2, 3, 4, 8), None)[:2] == (24, 1)
    z = torch.zeros(2, 3, 64)[..., 16:48].unflatten(-1, (4, 8))
    assert _layer._norm_rows(torch.zeros(2, 3, 4, 8), z) == (6, 4, [32, 64])
    with pytest.raises(ValueError):
        _layer._norm_rows(torch.zeros(2, 3), torch.zeros(3, 2).t())
    with pytest.raises(ValueError):
        _layer._norm_rows(torch.zeros(2, 8), torch.zeros(2, 8, dtype=torch.bfloat16))


def test_types_are_exported(lib):
    assert lib.GDN_NORM_OUT["fp8_row"] == 1 and lib.GDN_ACT["silu"] == 1
    assert ctypes.sizeof(ctypes.c_int64) == 8
    q = lib.QuantizedRows(torch.tensor([[1, -2], [3, 4]], dtype=torch.int8).repeat(1, 8),
                          torch.tensor([[0.5], [2.0]]), "int8_g16")
    assert q.shape == (2, 16) and q.dequantize()[1, 1] == 8.0
