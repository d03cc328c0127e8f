"""The RMS norm against the 64-bit reference.

Tolerances: one rounding to the result's type, plus fp32 roundings: a thread
adds at most d / 8 squares or products one after the other, the lanes and
warps ten more, and 64 stand for the root, the weight, and the gate's
logistic function.  An 8-bit code is the nearest one to y / scale: the value
code * scale is off by half a step of its format at most, and by the fp32
roundings of y."""

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, shape, dtype, residual, gate, pad=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    rows = lambda: r(*shape[:-1], shape[-1] + pad).to(dtype).cuda()[..., pad:]
    x, w = rows(), (torch.rand(shape[-1], generator=g) + 0.5).cuda()
    return x, w, rows() if residual else None, rows() if gate else None, rows(), rows()


SHAPES = [((1, 128), 0), ((5, 64), 8), ((3, 7, 128), 0), ((4, 2048), 16), ((33, 100), 0),
          ((2, 5), 3), ((3, 1), 0), ((2, 4097), 0), ((2, 8192), 0), ((1, 16384), 0), ((9, 1000), 8),
          ((700, 256), 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual,gate", [(False, False), (True, False), (False, True),
                                           (True, True)])
@pytest.mark.parametrize("shape,pad", SHAPES)
def test_norm_and_gradient(cuda_lib, shape, pad, residual, gate, dtype):
    x, w, res, z, dy, dr = make(1, shape, dtype, residual, gate, pad)
    y, s = cuda_lib.gdn_norm(x, w, residual=res, gate=z)
    want, kept = ref.norm(x, w, res, z, dtype=dtype)
    k = shape[-1] // 8 + 74
    ref.within(y, want, want.abs(), k, "y")
    if residual:
        assert torch.equal(s.double().cpu(), kept)
    else:
        assert s is None
    at = x if s is None else s
    dx, dw, dz = cuda_lib.gdn_norm_backward(at, w, dy, gate=z, dresidual=dr if residual else None)
    dr = dr if residual else None
    g = ref.norm_grad(at, w, dy, z, dr)
    m = ref.norm_grad(at, w, dy, z, dr, mag=True)
    rows = at.numel() // shape[-1]
    ref.within(dx, g[0], m[0], 3 * k, "dx")
    ref.within(dw, g[1], m[1], k + rows, "dweight")
    if gate:
        # the slope of silu passes through zero: its own terms are at most 1.1 |dy n w|
        mag = m[2] + (dy.double().cpu() * ref.norm(at, w)[0]).abs() * 1.1
        ref.within(dz, g[2], mag, k, "dgate")
    else:
        assert dz is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("qdq", ["fp8_row", "int8_g16", "int8_g32", "int8_g64"])
@pytest.mark.parametrize("shape,pad", [((3, 64), 0), ((17, 128), 8), ((2, 2048), 0), ((5, 320), 16),
                                       ((1, 8192), 0)])
def test_eight_bits(cuda_lib, shape, pad, qdq, dtype):
    x, w, res, z, _, _ = make(2, shape, dtype, True, True, pad)
    x[0, : shape[-1] // 2] = 0                       # whole groups of zeros
    res[0, : shape[-1] // 2] = 0
    q, s = cuda_lib.gdn_norm(x, w, residual=res, gate=z, qdq=qdq)
    y, _ = ref.norm(x, w, res, z, dtype=dtype)
    k = (shape[-1] // 8 + 74) * ref.U
    G = shape[-1] if qdq == "fp8_row" else int(qdq[6:])
    yg = y.unflatten(-1, (-1, G))
    amax = yg.abs().amax(-1)
    scale = q.scales.double().cpu().reshape(amax.shape)
    top = 448 if qdq == "fp8_row" else 127
    assert ((scale - amax / top).abs() <= (k + ref.U) * amax / top).all()
    code = q.codes.double().cpu().unflatten(-1, (-1, G))
    val, sc = code * scale[..., None], scale[..., None]
    if qdq == "fp8_row":
        step = torch.maximum(yg.abs() * 2.0 ** -4, sc * 2.0 ** -10)
    else:
        step = sc / 2
        assert code.abs().max() <= 127
    assert ((val - yg).abs() <= step * (1 + 1e-6) + 2 * k * yg.abs()).all()
    assert (code[scale == 0] == 0).all() and (scale == 0).any() == (G <= shape[-1] // 2)
    assert torch.allclose(q.dequantize().double().cpu().unflatten(-1, (-1, G)), val, rtol=1e-6)


def test_rows_unaligned_for_fp8(cuda_lib):
    """Rows that no vector load can take: E4M3 rows still work, INT8 groups
    are refused."""
    x, w, _, _, _, _ = make(3, (4, 99), BF16, False, False, 1)
    q, _ = cuda_lib.gdn_norm(x, w, qdq="fp8_row")
    y, _ = ref.norm(x, w)
    val = q.dequantize().double().cpu()
    assert ((val - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4,
                                             q.scales.double().cpu()[:, None] * 2.0 ** -10)
            * (1 + 1e-4)).all()
    x, w, _, _, _, _ = make(3, (4, 64), BF16, False, False, 1)
    with pytest.raises(cuda_lib.GdnError):
        cuda_lib.gdn_norm(x, w, qdq="int8_g32")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_heads_of_a_projection_slice(cuda_lib, dtype):
    """x contiguous a head, the gate a slice of a wider projection: the rows
    of the two are not equally far apart."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn((2, 9, 3, 128), generator=g).to(dtype).cuda()
    z = torch.randn((2, 9, 512), generator=g).to(dtype).cuda()[..., 64:448].unflatten(-1, (3, 128))
    w = torch.rand(128, generator=g).cuda() + 0.5
    dy = torch.randn((2, 9, 3, 128), generator=g).to(dtype).cuda()
    y, _ = cuda_lib.gdn_norm(x, w, gate=z)
    want, _ = ref.norm(x, w, gate=z)
    ref.within(y, want, want.abs(), 90, "y")
    dx, dw, dz = cuda_lib.gdn_norm_backward(x, w, dy, gate=z)
    a, b, c = ref.norm_grad(x, w, dy, z)
    ma, mb, mc = ref.norm_grad(x, w, dy, z, mag=True)
    ref.within(dx, a, ma, 270, "dx")
    ref.within(dw, b, mb, 90 + 54, "dweight")
    ref.within(dz, c, mc + (dy.double().cpu() * ref.norm(x, w)[0]).abs() * 1.1, 90, "dgate")


def test_nan_and_infinite_rows(cuda_lib):
    """A NaN or an infinity stays in its own row and shows in its scale."""
    x, w, _, _, _, _ = make(5, (4, 256), BF16, False, False)
    clean, _ = cuda_lib.gdn_norm(x, w)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y, _ = cuda_lib.gdn_norm(x, w)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
    assert y[1].isnan().all() and y[2, 9].isnan()
    q, _ = cuda_lib.gdn_norm(x, w, qdq="fp8_row")
    assert q.scales[0].isfinite() and q.scales[1].isnan() and q.scales[3].isfinite()
    assert not q.scales[2].isfinite()
    q, _ = cuda_lib.gdn_norm(x, w, qdq="int8_g32")
    assert q.scales[[0, 3]].isfinite().all() and q.scales[1].isnan().all()


def test_empty_and_repeats_and_graph(cuda_lib):
    x, w, res, z, dy, dr = make(6, (1000, 128), BF16, True, True)
    e = x[:0]
    assert cuda_lib.gdn_norm(e, w)[0].shape == (0, 128)
    assert (cuda_lib.gdn_norm_backward(e, w, e)[1] == 0).all()

    def run(x):
        y, s = cuda_lib.gdn_norm(x, w, residual=res, gate=z, qdq="int8_g32")
        return (y.codes, y.scales, s) + cuda_lib.gdn_norm_backward(s, w, dy, gate=z, dresidual=dr)

    want, again = run(x), run(x)
    xs = torch.zeros_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(xs)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, again, out):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("d", [20000, 32768])
def test_longest_rows(cuda_lib, d):
    x, w, res, z, dy, dr = make(7, (3, d), BF16, True, True)
    y, s = cuda_lib.gdn_norm(x, w, residual=res, gate=z)
    want, _ = ref.norm(x, w, res, z, dtype=BF16)
    ref.within(y, want, want.abs(), d // 8 + 74, "y")
    q, _ = cuda_lib.gdn_norm(x, w, residual=res, gate=z, qdq="fp8_row")
    step = torch.maximum(want.abs() * 2.0 ** -4, q.scales.double().cpu()[:, None] * 2.0 ** -10)
    assert ((q.dequantize().double().cpu() - want).abs() <= step * (1 + 1e-3)).all()
    dx, dw, dz = cuda_lib.gdn_norm_backward(s, w, dy, gate=z, dresidual=dr)
    g, m = ref.norm_grad(s, w, dy, z, dr), ref.norm_grad(s, w, dy, z, dr, mag=True)
    ref.within(dx, g[0], m[0], 3 * (d // 8 + 74), "dx")
    ref.within(dw, g[1], m[1], d // 8 + 74 + 3, "dweight")
    ref.within(dz, g[2], m[2] + (dy.double().cpu() * ref.norm(s, w)[0]).abs() * 1.1, d // 8 + 74,
               "dgate")
    with pytest.raises(cuda_lib.GdnError):
        cuda_lib.gdn_norm(torch.zeros(1, 32776, dtype=BF16, device="cuda"),
                          torch.ones(32776, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_off_the_vector_grid(cuda_lib, dtype):
    """A weight that starts 4 bytes past a 16-byte boundary gives the bits of
    an aligned copy; so does a convolution's."""
    x, w, _, _, dy, _ = make(8, (5, 256), dtype, False, False)
    off = torch.cat([w[:1], w])[1:]
    assert off.data_ptr() % 16 == 4 and off.is_contiguous()
    assert torch.equal(cuda_lib.gdn_norm(x, w)[0], cuda_lib.gdn_norm(x, off)[0])
    for a, b in zip(cuda_lib.gdn_norm_backward(x, w, dy)[:2],
                    cuda_lib.gdn_norm_backward(x, off, dy)[:2]):
        assert torch.equal(a, b)
    taps = torch.randn(256, 4, device="cuda")
    far = torch.cat([taps.flatten()[:1], taps.flatten()])[1:].view(256, 4)
    assert far.data_ptr() % 16 == 4
    for a, b in zip(cuda_lib.gdn_conv_prefill(x[None], taps),
                    cuda_lib.gdn_conv_prefill(x[None], far)):
        assert torch.equal(a, b)
