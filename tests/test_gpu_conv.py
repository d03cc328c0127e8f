"""The short causal convolution against the 64-bit reference.

Tolerances: one rounding to the result's type, and the fp32 roundings on the
way counted against the sum of the terms' magnitudes: W + 1 products and
sums, 40 for the logistic function (the fast exponential is within
2 + 1.2 |x| steps, |x| < 30 here) and, for the weights' gradients, one for
every token."""

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def make(seed, lead, C, W, dtype, n_seq, state, bias, pad=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = r(*lead, C + pad).to(dtype).cuda()[..., pad:]
    w, b = (r(C, W) * 0.5).cuda(), r(C).cuda() if bias else None
    st = r(n_seq, W - 1, C).to(dtype).cuda() if state else None
    dy = r(*lead, C).to(dtype).cuda()
    dl = r(n_seq, W - 1, C).to(dtype).cuda() if state else None
    return x, w, b, st, dy, dl


CASES = [  # dense T or packed lengths, sequences, C, W, pad, state, bias, activation
    (1, 3, 8, 4, 0, True, True, "silu"),
    (2, 2, 16, 3, 0, True, False, "silu"),
    (3, 1, 5, 4, 0, False, True, "none"),
    (9, 2, 264, 2, 8, True, True, "silu"),
    (67, 2, 40, 4, 64, False, True, "silu"),
    (300, 1, 24, 4, 3, True, True, "silu"),
    (515, 1, 8, 3, 0, False, False, "none"),
    ((1, 0, 2, 3, 0, 4, 70), 7, 24, 4, 8, True, True, "silu"),
    ((256, 257, 1, 255), 4, 16, 4, 0, False, True, "silu"),
    ((0, 0), 2, 8, 4, 0, True, True, "silu"),
    (tuple([3] * 40), 40, 7, 4, 1, True, True, "silu"),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_prefill_and_gradient(cuda_lib, case, dtype):
    T, n, C, W, pad, state, bias, act = case
    cu = None if isinstance(T, int) else cu_of(T)
    lead = (n, T) if cu is None else (1, cu[-1])
    x, w, b, st, dy, dl = make(7, lead, C, W, dtype, n, state, bias, pad)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = cuda_lib.gdn_conv_prefill(x, w, b, st, cud, activation=act)
    grads = cuda_lib.gdn_conv_backward(x, w, dy, b, st, cud, dl, activation=act)
    cuda_lib.check_last_error()
    silu = act == "silu"
    want = ref.conv(x, w, b, st, cu, silu, dy, dl)
    mag = ref.conv(x, w, b, st, cu, silu, dy, dl, mag=True)
    k = W + 41
    ref.within(y, want[0], mag[0], k, "y")
    assert torch.equal(last.double().cpu(), want[1])
    ref.within(grads[0], want[2], mag[2], 2 * k, "dx")
    ref.within(grads[1], want[3], mag[3], k + lead[0] * lead[1], "dweight")
    ref.within(grads[2], want[4], mag[4], k + lead[0] * lead[1], "dbias")
    ref.within(grads[3], want[5], mag[5], 2 * k, "dstate_in")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,W,n,pad", [(8, 4, 1, 0), (24, 3, 5, 8), (7, 4, 3, 2), (520, 2, 2, 0),
                                       (2304, 4, 9, 16)])
def test_decode(cuda_lib, C, W, n, pad, dtype):
    """Tokens one by one: outputs equal the prompt form's bit for bit (the
    same sums in the same order), and the state is the same rows."""
    T = 5
    x, w, b, st, _, _ = make(3, (n, T), C, W, dtype, n, True, True, pad)
    y, last = cuda_lib.gdn_conv_prefill(x, w, b, st)
    s = st.clone()
    for t in range(T):
        assert torch.equal(cuda_lib.gdn_conv_decode(x[:, t], w, b, s), y[:, t])
    assert torch.equal(s, last)


def test_continued_prompt_and_state_in_place(cuda_lib):
    x, w, b, st, _, _ = make(5, (2, 40), 16, 4, BF16, 2, True, True)
    y, last = cuda_lib.gdn_conv_prefill(x, w, b, st)
    for cut in (1, 2, 3, 17):
        s, parts = st.clone(), []
        for piece in (x[:, :cut].contiguous(), x[:, cut:].contiguous()):
            o = torch.empty_like(piece)
            cuda_lib.gdn_conv_prefill_into(piece, w, b, s, None, o, s)
            parts.append(o)
        assert torch.equal(torch.cat(parts, 1), y) and torch.equal(s, last)


def test_malformed_sequences_are_skipped_and_reported(cuda_lib):
    x, w, b, st, dy, _ = make(6, (1, 30), 8, 4, BF16, 3, True, True)
    good = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    y0, s0 = cuda_lib.gdn_conv_prefill(x, w, b, st, good)
    for cu in ([0, 10, 5, 30], [0, 10, 40, 30], [-3, 10, 20, 30], [0, 10, 20, 29],
               [0, 1 << 30, -(1 << 30), 30]):
        y, s = torch.full_like(y0, 3.0), torch.full_like(s0, 3.0)
        cuda_lib.gdn_conv_prefill_into(
            x, w, b, st, torch.tensor(cu, dtype=torch.int32, device="cuda"), y, s)
        assert cuda_lib.gdn_last_error() == 1
        if cu[:2] == [0, 10]:
            assert torch.equal(y[:, :10], y0[:, :10]) and torch.equal(s[0], s0[0])
        for i in range(3):
            ok = 0 <= cu[i] <= cu[i + 1] <= 30 and (i > 0 or cu[0] == 0) and (i < 2 or cu[3] == 30)
            assert ok or torch.equal(s[i], torch.full_like(s[i], 3.0))
        cuda_lib.gdn_conv_backward(x, w, dy, b, st,
                                   torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert cuda_lib.gdn_last_error() == 1
    assert cuda_lib.gdn_last_error() == 0


def test_streams_graphs_and_repeats(cuda_lib):
    """On another stream, captured and replayed with new inputs, and twice
    the same: the same bits."""
    x, w, b, st, dy, dl = make(8, (2, 600), 136, 4, BF16, 2, True, True)
    want = cuda_lib.gdn_conv_prefill(x, w, b, st) + cuda_lib.gdn_conv_backward(
        x, w, dy, b, st, None, dl)
    again = cuda_lib.gdn_conv_prefill(x, w, b, st) + cuda_lib.gdn_conv_backward(
        x, w, dy, b, st, None, dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = cuda_lib.gdn_conv_prefill(x, w, b, st) + cuda_lib.gdn_conv_backward(
            x, w, dy, b, st, None, dl)
    torch.cuda.synchronize()
    xs = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cuda_lib.gdn_conv_prefill(xs, w, b, st) + cuda_lib.gdn_conv_backward(
            xs, w, dy, b, st, None, dl)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for a, p, q, r in zip(want, again, other, out):
        assert torch.equal(a, p) and torch.equal(a, q) and torch.equal(a, r)
