"""The selective state space scan against the 64-bit reference.

Tolerances: one rounding to the result's type, plus fp32 roundings counted
against the sum of the terms' magnitudes.  A state is at most 3 T roundings
old (decay, product, sum a token); sums over N, P, and in the gradients over
the chunk add theirs, and the softplus, exponentials and decays some 64 more.
bf16 calls run on the tensor cores, whose operands are bf16 pairs: each
carries a value to 2^-17 relative, and a term has at most two of them, so
2^-15 covers it."""

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dstate_in")


def cu_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def make(seed, lead, H, P, G, N, dtype, n, state, extra=True, pad=16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    rows = r(*lead, pad + H * P + 2 * G * N).to(dtype).cuda()
    x = rows[..., pad:pad + H * P].unflatten(-1, (H, P))
    B = rows[..., pad + H * P:pad + H * P + G * N].unflatten(-1, (G, N))
    C = rows[..., pad + H * P + G * N:].unflatten(-1, (G, N))
    raw = r(*lead, H + 3).to(dtype).cuda()[..., 3:]
    A = -(torch.rand(H, generator=g) * 15 + 1).cuda()
    D = r(H).cuda() if extra else None
    bias = (r(H) - 3).cuda() if extra else None
    st = r(n, H, N, P).cuda() if state else None
    dy = r(*lead, H, P).to(dtype).cuda()
    dl = r(n, H, N, P).cuda() if state else None
    return (x, raw, A, B, C), D, bias, st, dy, dl


def check(lib, T, n, H, P, G, N, dtype, state, extra=True, seed=11, grads=True):
    cu = None if isinstance(T, int) else cu_of(T)
    lead = (n, T) if cu is None else (1, cu[-1])
    (x, raw, A, B, C), D, bias, st, dy, dl = make(seed, lead, H, P, G, N, dtype, n, state, extra)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = lib.gdn_scan_prefill(x, raw, A, B, C, D=D, dt_bias=bias, state_in=st, cu_seqlens=cud)
    longest = T if cu is None else max(T)
    k = 3 * longest + N + P + 64
    pair = 2.0 ** -15 if dtype == BF16 else 0.0
    args = (x, raw, A, B, C, D, bias, st, cu)
    if not grads:
        lib.check_last_error()
        want, mag = ref.scan(*args), ref.scan(*args, mag=True)
        ref.within(y, want[0], mag[0], k, "y", pair)
        ref.within(last, want[1], mag[1], k, "state_out")
        return
    got = lib.gdn_scan_backward(x, raw, A, B, C, dy, D=D, dt_bias=bias, state_in=st,
                                cu_seqlens=cud, dstate_out=dl)
    lib.check_last_error()
    want, mag = ref.scan(*args, dy, dl), ref.scan(*args, dy, dl, mag=True)
    ref.within(y, want[0], mag[0], k, "y", pair)
    ref.within(last, want[1], mag[1], k, "state_out")
    sums = lead[0] * lead[1]                      # dA, dD, ddt_bias add every token
    for i, name in enumerate(NAMES):
        kk = 2 * k + 128 + (sums if name in ("dA", "dD", "ddt_bias") else 0)
        ref.within(got[i], want[2 + i], mag[2 + i], kk, name, 2 * pair)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,P,G,N", [(2, 64, 1, 64), (2, 128, 2, 64), (3, 64, 1, 128),
                                     (4, 128, 2, 128)])
@pytest.mark.parametrize("T", [1, 63, 64, 65, 130])
def test_dense(cuda_lib, T, H, P, G, N, dtype):
    check(cuda_lib, T, 2, H, P, G, N, dtype, state=T != 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [(5, 0, 64, 1, 129, 0), (0, 0), (200, 7), tuple([2] * 40)])
def test_packed(cuda_lib, lens, dtype):
    check(cuda_lib, lens, len(lens), 4, 64, 2, 128, dtype, state=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,n,N", [(577, 1, 128), (1000, 2, 64), ((600, 0, 321, 64, 1), 5, 128)])
def test_long_sequences_of_few_heads(cuda_lib, T, n, N, dtype):
    """Few heads and many chunks: the sequences are cut into runs."""
    check(cuda_lib, T, n, 2, 64, 1, N, dtype, state=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_state_in_place_over_runs(cuda_lib, dtype):
    (x, raw, A, B, C), D, bias, st, _, _ = make(12, (2, 900), 2, 128, 1, 64, dtype, 2, True)
    y0, s0 = cuda_lib.gdn_scan_prefill(x, raw, A, B, C, D=D, dt_bias=bias, state_in=st)
    for _ in range(20):
        s, y = st.clone(), torch.empty_like(y0)
        cuda_lib.gdn_scan_prefill_into(x, raw, A, B, C, D, bias, s, None, y, s)
        assert torch.equal(s, s0) and torch.equal(y, y0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_skip_and_bias(cuda_lib, dtype):
    check(cuda_lib, 70, 1, 2, 64, 1, 64, dtype, state=False, extra=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,H,P,G,N", [(1, 1, 64, 1, 64), (3, 4, 128, 2, 128), (5, 6, 64, 3, 128)])
def test_decode(cuda_lib, n, H, P, G, N, dtype):
    (x, raw, A, B, C), D, bias, st, _, _ = make(5, (n,), H, P, G, N, dtype, n, True)
    s = st.clone()
    y = cuda_lib.gdn_scan_decode(x, raw, A, B, C, s, D=D, dt_bias=bias)
    one = [t[:, None] for t in (x, raw)] + [A] + [t[:, None] for t in (B, C)]
    want = ref.scan(*one, D, bias, st, None)
    mag = ref.scan(*one, D, bias, st, None, mag=True)
    ref.within(y, want[0][:, 0], mag[0][:, 0], N + 64, "y")
    ref.within(s, want[1], mag[1], 64, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_tokens(cuda_lib, dtype):
    """A prompt's state goes on with single tokens and with a second prompt:
    both stay within the bounds of the whole sequence's reference."""
    T, cut = 90, 70
    (x, raw, A, B, C), D, bias, st, _, _ = make(9, (2, T), 2, 64, 1, 128, dtype, 2, True)
    want = ref.scan(x, raw, A, B, C, D, bias, st, None)
    mag = ref.scan(x, raw, A, B, C, D, bias, st, None, mag=True)
    head = [t[:, :cut].contiguous() for t in (x, raw, B, C)]
    k, pair = 3 * T + 320, 2.0 ** -15 if dtype == BF16 else 0.0
    _, s = cuda_lib.gdn_scan_prefill(head[0], head[1], A, head[2], head[3], D=D, dt_bias=bias,
                                     state_in=st)
    s2 = s.clone()
    for t in range(cut, T):
        y = cuda_lib.gdn_scan_decode(x[:, t], raw[:, t], A, B[:, t], C[:, t], s, D=D, dt_bias=bias)
        ref.within(y, want[0][:, t], mag[0][:, t], k, "token", pair)
    ref.within(s, want[1], mag[1], k, "state after tokens")
    tail = [t[:, cut:].contiguous() for t in (x, raw, B, C)]
    y = torch.empty_like(tail[0])
    cuda_lib.gdn_scan_prefill_into(tail[0], tail[1], A, tail[2], tail[3], D, bias, s2, None, y, s2)
    ref.within(y, want[0][:, cut:], mag[0][:, cut:], k, "second prompt", pair)
    ref.within(s2, want[1], mag[1], k, "state after the second prompt")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_steps_at_the_ends_of_their_range(cuda_lib, dtype):
    """Steps of 60 (the state forgets everything: exp(-960) is 0) and of
    exp(-60) (it keeps everything): no NaN, and the reference's values.

    Values fade below 2^-126 here.  A bf16 operand piece has no bits under
    2^-133, so a term's error is at most 2^-134 times its other factor (6 at
    most in these inputs), and an output has 130 tokens' terms at most:
    130 * 6 * 2^-134 < 2^-124 absolute."""
    (x, raw, A, B, C), D, bias, st, dy, dl = make(4, (1, 130), 2, 64, 1, 64, dtype, 1, True)
    raw = raw.clone()
    raw[:, ::7] = 60.0
    raw[:, 1::7] = -60.0
    cu = None
    y, last = cuda_lib.gdn_scan_prefill(x, raw, A, B, C, D=D, dt_bias=bias, state_in=st)
    got = cuda_lib.gdn_scan_backward(x, raw, A, B, C, dy, D=D, dt_bias=bias, state_in=st,
                                     dstate_out=dl)
    args = (x, raw, A, B, C, D, bias, st, cu)
    want, mag = ref.scan(*args, dy, dl), ref.scan(*args, dy, dl, mag=True)
    k, pair = 3 * 130 + 192, 2.0 ** -15 if dtype == BF16 else 0.0
    floor = 2.0 ** -124 if dtype == BF16 else 0.0
    ref.within(y, want[0], mag[0], k, "y", pair, floor)
    ref.within(last, want[1], mag[1], k, "state_out", 0.0, floor)
    for i, name in enumerate(NAMES):
        ref.within(got[i], want[2 + i], mag[2 + i], 2 * k + 258, name, 2 * pair, floor)


def test_malformed_sequences_are_skipped_and_reported(cuda_lib):
    (x, raw, A, B, C), D, bias, st, dy, _ = make(6, (1, 200), 2, 64, 1, 64, BF16, 3, True)
    ok = torch.tensor([0, 100, 150, 200], dtype=torch.int32, device="cuda")
    y0, s0 = cuda_lib.gdn_scan_prefill(x, raw, A, B, C, state_in=st, cu_seqlens=ok)
    for cu in ([0, 100, 50, 200], [0, 100, 300, 200], [-3, 100, 150, 200], [0, 100, 150, 199],
               [0, 1 << 30, -(1 << 30), 200]):
        y, s = torch.full_like(y0, 3.0), torch.full_like(s0, 3.0)
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        cuda_lib.gdn_scan_prefill_into(x, raw, A, B, C, None, None, st, c, y, s)
        assert cuda_lib.gdn_last_error() == 1
        for i in range(3):
            good = 0 <= cu[i] <= cu[i + 1] <= 200 and (i > 0 or cu[0] == 0) and (
                i < 2 or cu[3] == 200)
            if not good:
                assert torch.equal(s[i], torch.full_like(s[i], 3.0))
        cuda_lib.gdn_scan_backward(x, raw, A, B, C, dy, state_in=st, cu_seqlens=c)
        assert cuda_lib.gdn_last_error() == 1
    assert cuda_lib.gdn_last_error() == 0


def test_rows_behind_the_last_sequence_stay(cuda_lib):
    """y is written where a sequence has tokens and nowhere else: a buffer
    around it keeps its values."""
    (x, raw, A, B, C), D, bias, st, _, _ = make(6, (2, 70), 2, 64, 1, 128, BF16, 2, False)
    buf = torch.full((4, 70, 2, 64), 5.0, dtype=BF16, device="cuda")
    s = torch.full((4, 2, 128, 64), 5.0, device="cuda")
    cuda_lib.gdn_scan_prefill_into(x, raw, A, B, C, D, bias, None, None, buf[1:3], s[1:3])
    torch.cuda.synchronize()
    for t in (buf, s):
        assert (t[0] == 5).all() and (t[3] == 5).all() and not (t[1:3] == 5).all()


def test_streams_graphs_and_repeats(cuda_lib):
    (x, raw, A, B, C), D, bias, st, dy, dl = make(8, (1, 333), 4, 64, 2, 128, BF16, 1, True)

    def run(x):
        return cuda_lib.gdn_scan_prefill(x, raw, A, B, C, D=D, dt_bias=bias, state_in=st) + \
            cuda_lib.gdn_scan_backward(x, raw, A, B, C, dy, D=D, dt_bias=bias, state_in=st,
                                       dstate_out=dl)

    want, again = run(x), run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(x)
    torch.cuda.synchronize()
    xs = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(xs)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for a, p, q, r in zip(want, again, other, out):
        assert torch.equal(a, p) and torch.equal(a, q) and torch.equal(a, r)
