"""The selective scan over thousands of tokens and many heads, norm-wise
against the chunked 64-bit form: what element-wise bounds that count every
token's roundings cannot see.

A bf16 output that is the rounding of a value within a relative eps (2-norm)
of the exact one differs from the exact one's rounding only where the two
straddle a boundary, with probability |d| / step each; a step is 2^-7 of the
value at most, so the squared 2-norm of what differs is at most sum |d| step <=
2^-7 eps of the output's.  fp32 outputs are compared directly."""

import math

import pytest
import torch

import layer_long as long

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, lead, n, H, P, G, N, dtype, step, decay, spread=1.0):
    """Inputs as a projection gives them, the steps around `step` (their
    logarithm spread by `spread`), A between `decay`'s two values."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, B, C = r(*lead, H, P).to(dtype), r(*lead, G, N).to(dtype), r(*lead, G, N).to(dtype)
    raw = (r(*lead, H) * spread).to(dtype)
    A = -(torch.rand(H, generator=g, device="cuda") * (decay[1] - decay[0]) + decay[0])
    bias = torch.full((H,), math.log(math.expm1(step)), device="cuda")
    return dict(x=x, raw=raw, A=A, B=B, C=C, D=r(H), bias=bias, state=r(n, H, N, P),
                dy=r(*lead, H, P).to(dtype), dlast=r(n, H, N, P))


def prefill(lib, t, cu=None):
    return lib.gdn_scan_prefill(t["x"], t["raw"], t["A"], t["B"], t["C"], D=t["D"],
                                dt_bias=t["bias"], state_in=t["state"], cu_seqlens=cu)


def backward(lib, t, cu=None):
    return lib.gdn_scan_backward(t["x"], t["raw"], t["A"], t["B"], t["C"], t["dy"], D=t["D"],
                                 dt_bias=t["bias"], state_in=t["state"], cu_seqlens=cu,
                                 dstate_out=t["dlast"])


def args(t, cu=None):
    return tuple(t[k] for k in ("x", "raw", "A", "B", "C", "D", "bias", "state")) + (cu,)


def rounding(eps):
    return math.sqrt(eps * 2.0 ** -7)


def test_gradients_summed_over_many_heads(cuda_lib):
    """One CTA takes a chunk's sixteen heads.  dB and dC are fp32 sums of
    products whose operands carry 2^-25; a head's products are twelve sums in
    the tensor pipe, which truncates (2^-24 each on average), and four more
    stand for the decays: eps = 2^-20.  dx has M in bf16 pairs, 2^-18."""
    t = make(1, (2, 4096), 2, 16, 64, 1, 128, BF16, 0.01, (1.0, 16.0))
    got = backward(cuda_lib, t)
    want = long.scan_grad(*args(t), t["dy"], t["dlast"])[2:]
    for i, name, eps in ((3, "dB", 2.0 ** -20), (4, "dC", 2.0 ** -20), (0, "dx", 2.0 ** -18),
                         (1, "ddt", 2.0 ** -18)):
        assert long.off(got[i], want[i].to(BF16)) <= rounding(eps), name


@pytest.mark.parametrize("n,T,H,step,decay,spread", [
    (4, 4096, 32, 1e-3, (1.0, 1.0), 1.0), (4, 8192, 32, 1e-4, (0.1, 0.1), 0.0),
    (2, 4096, 64, 1e-2, (1.0, 16.0), 1.0)])
def test_states_of_long_prompts(cuda_lib, n, T, H, step, decay, spread):
    """The state that a prompt leaves, in 32 bits, from quick forgetting to
    none: a chunk adds twelve sums in the tensor pipe (2^-23 at most each) and
    one rounding of the state; the decays of the chunks are products of
    T / 64 of them, whose roundings (2^-24) add up like their root; the step
    and its logarithm's bias are off by 2^-21 at most."""
    t = make(3, (n, T), n, H, 64, 1, 64, BF16, step, decay, spread)
    y, last = prefill(cuda_lib, t)
    want = long.scan(*(v if v is None else v.double() for v in args(t)))
    eps = (12 * 2.0 + 1) * 2.0 ** -24 + math.sqrt(T / 64) * 2.0 ** -24 + 2.0 ** -21
    assert long.off(last, want[1]) <= eps
    # y: M and the state in bf16 pairs, 2^-18
    assert long.off(y, want[0].to(BF16)) <= rounding(2.0 ** -18)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,step", [(16384, 1e-5), (8192, 1e-4)])
def test_a_state_that_forgets_almost_nothing(cuda_lib, T, step, dtype):
    """The same small step in every token, and few heads, so that the sequence
    is cut into runs: neither the chunks' nor the runs' decays may drift.  The
    bound of test_states_of_long_prompts for bf16; fp32 rounds the state once
    a token, T roundings of 2^-25 on average that add up like their root."""
    t = make(4, (1, T), 1, 2, 64, 1, 64, dtype, step, (0.1, 0.1), 0.0)
    last = prefill(cuda_lib, t)[1]
    want = long.scan(*(v if v is None else v.double() for v in args(t)))[1]
    if dtype == BF16:
        eps = (12 * 2.0 + 1) * 2.0 ** -24 + math.sqrt(T / 64) * 2.0 ** -24 + 2.0 ** -21
    else:
        eps = math.sqrt(T) * 2.0 ** -25 + 2.0 ** -21
    assert long.off(last, want) <= eps


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_single_tokens(cuda_lib, dtype):
    """600 single tokens of the same small step: every one rounds the state
    once, 600 roundings of 2^-25 on average that add up like their root; the
    step's logarithm is off by 2^-21 at most."""
    T = 600
    t = make(5, (2, T), 2, 2, 64, 1, 128, dtype, 1e-4, (0.1, 0.1), 0.0)
    s = t["state"].clone()
    for i in range(T):
        y = cuda_lib.gdn_scan_decode(t["x"][:, i], t["raw"][:, i], t["A"], t["B"][:, i],
                                     t["C"][:, i], s, D=t["D"], dt_bias=t["bias"])
    want = long.scan(*(v if v is None else v.double() for v in args(t)))
    assert long.off(s, want[1]) <= math.sqrt(T) * 2.0 ** -25 + 2.0 ** -21
    half = torch.finfo(dtype).eps / 2
    assert long.off(y, want[0][:, -1]) <= half + 2.0 ** -20


def test_infinite_states_stay_infinite(cuda_lib):
    """Whatever a decay's second float is, an infinity in a state is kept."""
    t = make(6, (1, 8), 1, 2, 64, 1, 64, BF16, 1e-3, (0.5, 4.0))
    s = t["state"].clone()
    s[0, 0, 3, 5], s[0, 1, 7, 9] = math.inf, -math.inf
    for i in range(8):
        cuda_lib.gdn_scan_decode(t["x"][:, i], t["raw"][:, i], t["A"], t["B"][:, i], t["C"][:, i],
                                 s, D=t["D"], dt_bias=t["bias"])
    assert s[0, 0, 3, 5] == math.inf and s[0, 1, 7, 9] == -math.inf
    assert int((~s.isfinite()).sum()) == 2


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H", [(70, 2), (600, 2)])
def test_infinite_states_stay_infinite_in_prompts(cuda_lib, T, H, dtype):
    """An infinity in the state that a prompt starts from, or in the gradient
    of the one that it leaves, is in the state it leaves, or in the gradient of
    the one it starts from, and in no other element of either."""
    t = make(7, (1, T), 1, H, 64, 1, 64, dtype, 1e-3, (0.5, 4.0))
    t["state"][0, 0, 3, 5], t["state"][0, 1, 7, 9] = math.inf, -math.inf
    last = prefill(cuda_lib, t)[1]
    assert last[0, 0, 3, 5] == math.inf and last[0, 1, 7, 9] == -math.inf
    assert int((~last.isfinite()).sum()) == 2
    t["state"], t["dlast"] = t["dlast"], t["state"]
    first = backward(cuda_lib, t)[7]
    assert first[0, 0, 3, 5] == math.inf and first[0, 1, 7, 9] == -math.inf
    assert int((~first.isfinite()).sum()) == 2


FORMS = [  # tokens or packed lengths, sequences, heads, P, G, N, cut into runs
    (5000, 1, 1, 64, 1, 64, True),                        # 20 runs of a sequence
    ((3000, 0, 700, 64, 1, 1500), 6, 2, 64, 1, 128, True),   # packed, and cut
    (2210, 2, 12, 128, 2, 128, True),                     # six heads a CTA of the gradient
    (1150, 2, 12, 64, 2, 64, True),                       # three, two CTAs a group
    ((1000, 0, 4000, 33, 65), 5, 8, 64, 1, 128, True),    # eight, packed
    (700, 4, 32, 64, 4, 64, False),                       # not cut: 128 units
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", FORMS, ids=[str(i) for i in range(len(FORMS))])
def test_runs_heads_and_packed_sequences(cuda_lib, case, dtype):
    """Every output and gradient in the forms that long calls and many heads
    take.  bf16: M and W as in test_gradients_summed_over_many_heads; states
    and sums over all tokens within the bound of test_states_of_long_prompts,
    twice where a state meets an adjoint.  fp32: the state is rounded T times,
    as in test_a_state_that_forgets_almost_nothing.  ddt is the sum of A l and
    x . du, which can cancel: four times the bound of its terms."""
    T, n, H, P, G, N, cut = case
    cu, lead = None, (n, T)
    if not isinstance(T, int):
        cu, lead = [0], (1, sum(T))
        for v in T:
            cu.append(cu[-1] + v)
        T = max(T)
    bytes_ = cuda_lib.lib.gdn_scan_prefill_workspace_bytes(
        n, lead[1], H, P, G, N, cuda_lib.GDN_DTYPE[dtype], int(cu is not None))
    assert (bytes_ > 0) == cut
    t = make(8, lead, n, H, P, G, N, dtype, 0.01, (1.0, 16.0))
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = prefill(cuda_lib, t, cud) + backward(cuda_lib, t, cud)
    cuda_lib.check_last_error()
    want = long.scan_grad(*args(t, cu), t["dy"], t["dlast"])
    if dtype == BF16:
        state = (12 * 2.0 + 1) * 2.0 ** -24 + math.sqrt(T / 64) * 2.0 ** -24 + 2.0 ** -21
        pair, sums, step = (rounding(2.0 ** -k) for k in (18, 20, 18))
    else:
        state = pair = math.sqrt(T) * 2.0 ** -25 + 2.0 ** -21
        sums, step = 2 * state, 4 * state
    bounds = (("y", pair), ("state_out", state), ("dx", 2 * pair), ("ddt", 2 * step),
              ("dA", 2 * state), ("dB", sums), ("dC", sums), ("dD", state),
              ("ddt_bias", 2 * state), ("dstate_in", state))
    for (name, bound), a, b in zip(bounds, got, want):
        assert long.off(a, b.to(a.dtype)) <= bound, name


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_operands_of_three_pieces(cuda_lib, dtype):
    """Sums over all tokens stay fp32 quantities: bounds that operands of fewer
    bf16 pieces are beyond (``test_layer_long.py``)."""
    x, raw, A, B, C, D, bias, h, dy, dl = (t.cuda() for t in long.pieces_case())
    t = dict(x=x.to(dtype), raw=raw.to(dtype), A=A, B=B.to(dtype), C=C.to(dtype), D=D, bias=bias,
             state=h, dy=dy.to(dtype), dlast=dl)
    want = long.scan_grad(*args(t), t["dy"], t["dlast"])
    last, got = prefill(cuda_lib, t)[1], backward(cuda_lib, t)
    assert long.off(last, want[1]) <= long.STATE_BOUND
    assert long.off(got[7], want[9]) <= long.STATE_BOUND
    assert long.off(got[2], want[4]) <= long.DA_BOUND
    assert long.off(got[6], want[8]) <= long.DA_BOUND
    assert long.off(got[5], want[7]) <= long.STATE_BOUND


@pytest.mark.parametrize("n,T", [(1, 64), (2, 2048)])
def test_sums_of_products_are_not_truncated(cuda_lib, n, T):
    """All inputs positive, so that a truncating sum shows as what it is, a bias.
    dD sums dy x over P and the tokens: a step of sixteen products in the tensor
    pipe drops 2^-24 at most, and the fp32 sums of steps, tokens and chunks round
    either way, half as much together.  (Eight steps truncated one on top of the
    other lose 1.6e-7 to 1.9e-7.)"""
    t = make(3, (n, T), n, 2, 128, 1, 128, BF16, 0.01, (1.0, 16.0))
    for k in ("x", "B", "C", "state", "dy", "dlast", "D"):
        t[k] = t[k].abs()
    got = backward(cuda_lib, t)
    want = long.scan_grad(*args(t), t["dy"], t["dlast"])[2:]
    assert long.off(got[5], want[5]) <= 1.5 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,T,H,step,A", [(1, 8192, 2, 1e-4, 0.1), (2, 2048, 32, 1e-3, 1.0)])
def test_gradients_of_slowly_forgetting_states(cuda_lib, n, T, H, step, A, dtype):
    """The adjoint runs back over thousands of tokens as the state runs forward:
    the bounds of test_states_of_long_prompts (bf16) and
    test_a_state_that_forgets_almost_nothing (fp32), and for dB and dC those of
    test_gradients_summed_over_many_heads, where a state or an adjoint enters
    with its own bound."""
    t = make(9, (n, T), n, H, 64, 1, 64, dtype, step, (A, A))
    got = backward(cuda_lib, t)
    want = long.scan_grad(*args(t), t["dy"], t["dlast"])[2:]
    if dtype == BF16:
        state = (12 * 2.0 + 1) * 2.0 ** -24 + math.sqrt(T / 64) * 2.0 ** -24 + 2.0 ** -21
        sums = rounding(2.0 ** -20 + state)
    else:
        state = math.sqrt(T) * 2.0 ** -25 + 2.0 ** -21
        sums = 2 * state
    for i, name, bound in ((7, "dstate_in", state), (5, "dD", state), (3, "dB", sums),
                           (4, "dC", sums)):
        assert long.off(got[i], want[i].to(got[i].dtype)) <= bound, name
