"""The convolution and the norm in the forms that only large calls take, against
the 64-bit reference (tolerances as in ``test_gpu_conv.py`` and
``test_gpu_norm.py``)."""

import pytest
import torch

import layer_ref as ref
from test_gpu_conv import cu_of, make
from test_gpu_norm import make as make_rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SMS = 148

CONV = [  # tokens or packed lengths, sequences, C, W, pad, state
    (7700, 2, 520, 4, 8, True),
    (3500, 2, 333, 3, 1, False),
    ((3000, 0, 2, 257, 5000, 32, 33, 1, 4000), 9, 1032, 4, 0, True),
]


def conv_ctas(T, n, C, dtype):
    """CTAs of the runs of 32 tokens, eight a CTA, 32 lanes of 4 or 1 channels."""
    v = 4 if C % 4 == 0 else 1
    tiles = n * -(-T // 256) if isinstance(T, int) else n + sum(T) // 256
    return tiles * -(-C // (32 * v))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CONV, ids=[str(i) for i in range(len(CONV))])
def test_convolution_in_long_runs(cuda_lib, case, dtype):
    """Enough CTAs for runs of 32 tokens (bf16; fp32 takes runs of 8, here of
    more tiles than in ``test_gpu_conv.py``)."""
    T, n, C, W, pad, state = case
    assert conv_ctas(T, n, C, dtype) >= 2 * SMS
    cu = None if isinstance(T, int) else cu_of(T)
    lead = (n, T) if cu is None else (1, cu[-1])
    x, w, b, st, dy, dl = make(7, lead, C, W, dtype, n, state, True, pad)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = cuda_lib.gdn_conv_prefill(x, w, b, st, cud)
    grads = cuda_lib.gdn_conv_backward(x, w, dy, b, st, cud, dl)
    cuda_lib.check_last_error()
    want = ref.conv(x, w, b, st, cu, True, dy, dl)
    mag = ref.conv(x, w, b, st, cu, True, dy, dl, mag=True)
    k = W + 41
    ref.within(y, want[0], mag[0], k, "y")
    assert torch.equal(last.double().cpu(), want[1])
    ref.within(grads[0], want[2], mag[2], 2 * k, "dx")
    ref.within(grads[1], want[3], mag[3], k + lead[0] * lead[1], "dweight")
    ref.within(grads[2], want[4], mag[4], k + lead[0] * lead[1], "dbias")
    ref.within(grads[3], want[5], mag[5], 2 * k, "dstate_in")
    for i, name in ((1, "dweight"), (2, "dbias")):  # and norm-wise: sums of the tokens' terms
        off = (grads[i].double().cpu() - want[2 + i]).norm() / want[2 + i].norm()
        assert off <= 2e-6, name


@pytest.mark.parametrize("C,W,dtype,n", [(4352, 4, BF16, 121), (4352, 4, BF16, 122),
                                         (4352, 3, F32, 121), (333, 2, BF16, 199),
                                         (332, 4, F32, 1101)])
def test_tokens_of_many_sequences(cuda_lib, C, W, dtype, n):
    """Four sequences a thread, and fewer in the last CTA: the bits of the
    prompt form, token by token."""
    v = 1 if C % 4 else (8 if dtype == BF16 else 4)
    per = -(-C // v)
    threads = 128 if per >= 128 else -(-per // 32) * 32
    assert n * -(-per // threads) >= (2 if dtype == BF16 else 7) * SMS
    T = 3
    x, w, b, st, _, _ = make(3, (n, T), C, W, dtype, n, True, True, 8)
    y, last = cuda_lib.gdn_conv_prefill(x, w, b, st)
    s = torch.cat([st, st[:3]])
    for t in range(T):
        assert torch.equal(cuda_lib.gdn_conv_decode(x[:, t], w, b, s[:n]), y[:, t])
    assert torch.equal(s[:n], last) and torch.equal(s[n:], st[:3])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual,gate", [(False, False), (True, True)])
@pytest.mark.parametrize("rows,d", [(9001, 128), (1500, 2048), (1201, 1000), (5000, 64),
                                    (700, 4096), (1300, 101), (601, 16384)])
def test_norm_gradient_of_many_rows(cuda_lib, rows, d, residual, gate, dtype):
    """More rows than the gradient's 592 CTAs take at once: a thread's rows one
    behind the other, and dweight summed over them."""
    x, w, _, z, dy, dr = make_rows(1, (rows, d), dtype, False, gate)
    dr = dr if residual else None
    got = cuda_lib.gdn_norm_backward(x, w, dy, gate=z, dresidual=dr)
    g = ref.norm_grad(x, w, dy, z, dr)
    m = ref.norm_grad(x, w, dy, z, dr, mag=True)
    k = d // 8 + 74
    ref.within(got[0], g[0], m[0], 3 * k, "dx")
    ref.within(got[1], g[1], m[1], k + rows, "dweight")
    off = (got[1].double().cpu() - g[1]).norm() / g[1].norm()
    assert off <= 2e-6, "dweight"                     # norm-wise: a sum of the rows' terms
    if gate:
        mag = m[2] + (dy.double().cpu() * ref.norm(x, w)[0]).abs() * 1.1
        ref.within(got[2], g[2], mag, k, "dgate")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", [(20011, 128), (3001, 2048)])
def test_norm_of_many_rows(cuda_lib, rows, d, dtype):
    x, w, res, z, _, _ = make_rows(2, (rows, d), dtype, True, True, 8)
    y, s = cuda_lib.gdn_norm(x, w, residual=res, gate=z)
    want, kept = ref.norm(x, w, res, z, dtype=dtype)
    ref.within(y, want, want.abs(), d // 8 + 74, "y")
    assert torch.equal(s.double().cpu(), kept)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,T", [(3000, 3), (300, 70), (257, 1)])
def test_many_packed_sequences(cuda_lib, n, T, dtype):
    """More packed sequences than are ranked by length or found in one probe:
    the bits of the dense call over the same sequences."""
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    H, P, G, N, C = 2, 64, 1, 64, 24
    x, raw, B, Cm, dy = r(n, T, H, P), r(n, T, H), r(n, T, G, N), r(n, T, G, N), r(n, T, H, P)
    A, D = -torch.rand(H, generator=g).cuda() - 0.5, torch.randn(H, generator=g).cuda()
    st = torch.randn(n, H, N, P, generator=g).cuda()
    u, w, b, cs, du = r(n, T, C), torch.randn(C, 4, generator=g).cuda(), \
        torch.randn(C, generator=g).cuda(), r(n, 3, C), r(n, T, C)
    cu = (torch.arange(n + 1, dtype=torch.int32) * T).cuda()
    one = lambda t: t.reshape(1, n * T, *t.shape[2:])

    def scan(f, cu):
        a = (f(x), f(raw), A, f(B), f(Cm))
        kw = dict(D=D, state_in=st, cu_seqlens=cu)
        return cuda_lib.gdn_scan_prefill(*a, **kw) + tuple(
            cuda_lib.gdn_scan_backward(*a, f(dy), dstate_out=st, **kw)[i] for i in (0, 1, 3, 4, 7))

    def conv(f, cu):
        back = cuda_lib.gdn_conv_backward(f(u), w, f(du), b, cs, cu, cs)
        return cuda_lib.gdn_conv_prefill(f(u), w, b, cs, cu) + (back[0], back[3])

    for op in (scan, conv):
        for i, (p, q) in enumerate(zip(op(lambda t: t, None), op(one, cu))):
            assert torch.equal(p.reshape(-1), q.reshape(-1)), (op.__name__, i)
    cuda_lib.check_last_error()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(cuda_lib, dtype):
    """Dense calls of no tokens pass their states and gradients through."""
    n, H, P, N, C = 3, 2, 64, 64, 8
    e = lambda *s: torch.empty(n, 0, *s, dtype=dtype, device="cuda")
    st = torch.randn(n, H, N, P, device="cuda")
    A = -torch.ones(H, device="cuda")
    scan = (e(H, P), e(H), A, e(1, N), e(1, N))
    y, last = cuda_lib.gdn_scan_prefill(*scan, state_in=st)
    assert y.shape == (n, 0, H, P) and torch.equal(last, st)
    got = cuda_lib.gdn_scan_backward(*scan, e(H, P), state_in=st, dstate_out=st)
    assert torch.equal(got[7], st) and all((got[i] == 0).all() for i in (2, 5, 6))
    w, cs = torch.randn(C, 4, device="cuda"), torch.randn(n, 3, C, device="cuda").to(dtype)
    y, last = cuda_lib.gdn_conv_prefill(e(C), w, None, cs)
    assert y.shape == (n, 0, C) and torch.equal(last, cs)
    got = cuda_lib.gdn_conv_backward(e(C), w, e(C), None, cs, None, cs)
    assert torch.equal(got[3], cs) and (got[1] == 0).all() and (got[2] == 0).all()
