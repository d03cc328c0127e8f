"""The RMS norm where its formula has no value, and in the forms that only
many or long rows take, against the 64-bit reference (tolerances as in
``test_gpu_norm.py``)."""

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rows(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 2048, 8192])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_zeros(cuda_lib, d, eps, dtype):
    """A row of zeros stays one, in every type of output and with eps = 0, and
    lets only the residual's gradient through; its neighbours do not notice."""
    x, z, dy, dr = (rows(i, 5, d, dtype=dtype) for i in range(4))
    w = torch.rand(d, device="cuda") + 0.5
    x[2] = 0
    y, _ = cuda_lib.gdn_norm(x, w, gate=z, eps=eps)
    want, _ = ref.norm(x, w, gate=z, eps=eps)
    want[2] = 0
    ref.within(y, want, want.abs(), d // 8 + 74, "y")
    assert (y[2] == 0).all()
    for qdq in ("fp8_row", "int8_g16", "int8_g32", "int8_g64"):
        q, _ = cuda_lib.gdn_norm(x, w, gate=z, eps=eps, qdq=qdq)
        assert (q.scales[2] == 0).all() and (q.codes[2].float() == 0).all()
        assert (q.scales[[0, 1, 3, 4]] > 0).all() and q.scales.isfinite().all()
    dx, dw, dz = cuda_lib.gdn_norm_backward(x, w, dy, gate=z, dresidual=dr, eps=eps)
    keep = [0, 1, 3, 4]
    g = ref.norm_grad(x[keep], w, dy[keep], z[keep], dr[keep], eps=eps)
    m = ref.norm_grad(x[keep], w, dy[keep], z[keep], dr[keep], eps=eps, mag=True)
    ref.within(dx[keep], g[0], m[0], 3 * (d // 8 + 74), "dx")
    ref.within(dw, g[1], m[1], d // 8 + 74 + 5, "dweight")
    assert (dz[2] == 0).all() and dz.isfinite().all() and dx.isfinite().all()
    if eps == 0:
        assert torch.equal(dx[2], dr[2])
