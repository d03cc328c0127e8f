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
