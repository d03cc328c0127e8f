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
