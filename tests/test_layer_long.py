"""Pins the chunked 64-bit scan to the token-by-token one (CPU)."""

import pytest
import torch

import layer_long as long
import layer_ref as ref


@pytest.mark.parametrize("lens", [None, (5, 0, 64, 131)])
def test_chunks_are_the_tokens(lens):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    H, P, G, N = 4, 3, 2, 5
    cu, lead, n = None, (2, 150), 2
    if lens:
        cu, lead, n = [0], (1, sum(lens)), len(lens)
        for v in lens:
            cu.append(cu[-1] + v)
    args = (r(*lead, H, P), r(*lead, H), -torch.rand(H, generator=g, dtype=torch.float64) * 3,
            r(*lead, G, N), r(*lead, G, N), r(H), r(H) - 2, r(n, H, N, P), cu)
    dy, dl = r(*lead, H, P), r(n, H, N, P)
    for a, b in zip(long.scan_grad(*args, dy, dl), ref.scan(*args, dy, dl)):
        assert (a - b).abs().max() <= 1e-11 * b.abs().max()


def test_bounds_tell_pieces_apart():
    """The bounds that the library's states and gradients of A are held to:
    operands of one bf16 piece are far beyond them, ones of three far within.  A
    state of two is beyond as well; a gradient of A of two need not be, whose
    errors have random signs and average out over the tokens (5e-7 here)."""
    case = long.pieces_case()
    x, raw, A, B, C, D, bias, h, dy, dl = (t.double() for t in case)
    want = long.scan_grad(x, raw, A, B, C, D, bias, h, None, dy, dl)
    off = {}
    for k in (1, 2, 3):
        state, dA = long.with_pieces(case, k)
        off[k] = long.off(state, want[1]), long.off(dA, want[4])
    assert off[1][0] > 100 * long.STATE_BOUND and off[1][1] > 100 * long.DA_BOUND
    assert off[2][0] > 2 * long.STATE_BOUND
    assert off[3][0] < long.STATE_BOUND / 20 and off[3][1] < long.DA_BOUND / 20
