"""Packed calls whose cu_seqlens steps back: what the sequences that are in order
receive does not depend on which of the others' CTAs comes last."""

import pytest
import torch

import test_gpu_scan as scan
from test_gpu_conv import make

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_convolution_steps_back(cuda_lib, dtype):
    x, w, b, st, dy, _ = make(6, (1, 30), 8, 4, dtype, 3, True, True)
    good = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    y0, s0 = cuda_lib.gdn_conv_prefill(x, w, b, st, good)
    back = torch.tensor([0, 10, 5, 30], dtype=torch.int32, device="cuda")
    bad = 0
    for _ in range(300):
        y, s = torch.full_like(y0, 3.0), torch.full_like(s0, 3.0)
        cuda_lib.gdn_conv_prefill_into(x, w, b, st, back, y, s)
        bad += not (torch.equal(y[:, :10], y0[:, :10]) and torch.equal(s[0], s0[0])
                    and (y[:, 10:] == 3).all() and (s[1:] == 3).all())
        assert cuda_lib.gdn_last_error() == 1
    assert bad == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_steps_back(cuda_lib, dtype):
    (x, raw, A, B, C), D, bias, st, _, _ = scan.make(6, (1, 200), 2, 64, 1, 64, dtype, 3, True)
    good = torch.tensor([0, 100, 150, 200], dtype=torch.int32, device="cuda")
    y0, s0 = cuda_lib.gdn_scan_prefill(x, raw, A, B, C, D=D, dt_bias=bias, state_in=st,
                                       cu_seqlens=good)
    back = torch.tensor([0, 100, 50, 200], dtype=torch.int32, device="cuda")
    bad = 0
    for _ in range(300):
        y, s = torch.full_like(y0, 3.0), torch.full_like(s0, 3.0)
        cuda_lib.gdn_scan_prefill_into(x, raw, A, B, C, D, bias, st, back, y, s)
        bad += not (torch.equal(y[:, :100], y0[:, :100]) and torch.equal(s[0], s0[0])
                    and (y[:, 100:] == 3).all() and (s[1:] == 3).all())
        assert cuda_lib.gdn_last_error() == 1
    assert bad == 0
