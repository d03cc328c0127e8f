"""CPU checks of the 64-bit reference that the layer operators are tested
against: the written-out gradients equal central differences of the forward
definitions, and every planted mistake is noticed by the comparison."""

import pytest
import torch

import layer_ref as ref


def rnd(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float64)


def differences(f, x, d=1e-5):
    """Central differences of the scalar f at x."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + d
        hi = f()
        flat[i] = v - d
        lo = f()
        flat[i] = v
        out[i] = (hi - lo) / (2 * d)
    return g


def close(a, b):
    # the differences' own error: d^2 f''' / 6 ~ 1e-10 f''', and 1e-16 f / d ~ 1e-11 f
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), float((a - b).abs().max())


@pytest.mark.parametrize("packed", [False, True])
def test_conv_gradient(packed):
    g = torch.Generator().manual_seed(1)
    C, W = 3, 4
    cu = [0, 5, 5, 7] if packed else None
    x = rnd(g, 1, 7, C) if packed else rnd(g, 2, 5, C)
    n = 3 if packed else 2
    w, b, st = rnd(g, C, W), rnd(g, C), rnd(g, n, W - 1, C)
    dy, dl = rnd(g, *x.shape), rnd(g, n, W - 1, C)

    def f():
        y, last = ref.conv(x, w, b, st, cu)
        return float((y * dy).sum() + (last * dl).sum())

    _, _, dx, dw, db, ds = ref.conv(x, w, b, st, cu, dy=dy, dlast=dl)
    for t, grad in ((x, dx), (w, dw), (b, db), (st, ds)):
        close(differences(f, t), grad)


@pytest.mark.parametrize("packed", [False, True])
def test_scan_gradient(packed):
    g = torch.Generator().manual_seed(2)
    H, P, G, N = 4, 2, 2, 3
    cu = [0, 4, 4, 7] if packed else None
    lead = (1, 7) if packed else (2, 4)
    n = 3 if packed else 2
    x, raw = rnd(g, *lead, H, P), rnd(g, *lead, H)
    B, C = rnd(g, *lead, G, N), rnd(g, *lead, G, N)
    A, D, bias = -rnd(g, H).abs(), rnd(g, H), rnd(g, H)
    st, dl, dy = rnd(g, n, H, N, P), rnd(g, n, H, N, P), rnd(g, *x.shape)

    def f():
        y, last = ref.scan(x, raw, A, B, C, D, bias, st, cu)
        return float((y * dy).sum() + (last * dl).sum())

    out = ref.scan(x, raw, A, B, C, D, bias, st, cu, dy, dl)[2:]
    for t, grad in zip((x, raw, A, B, C, D, bias, st), out):
        close(differences(f, t), grad)


@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradient(gated):
    g = torch.Generator().manual_seed(3)
    x, w, dy, dr = rnd(g, 4, 5), rnd(g, 5), rnd(g, 4, 5), rnd(g, 4, 5)
    z = rnd(g, 4, 5) if gated else None

    def f():
        y, s = ref.norm(x, w, gate=z)
        return float((y * dy).sum() + (s * dr).sum())

    ds, dw, dz = ref.norm_grad(x, w, dy, z, dr)
    for t, grad in ((x, ds), (w, dw)) + (((z, dz),) if gated else ()):
        close(differences(f, t), grad)


def test_e4m3_reference():
    """Every E4M3 value is its own nearest, and midpoints go to the even code."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[codes.isfinite()]
    assert torch.equal(ref.e4m3(codes), codes)
    pos = codes[codes >= 0].unique()
    mid = (pos[1:] + pos[:-1]) / 2
    even = torch.where(torch.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])
    assert torch.equal(ref.e4m3(mid), even)
    assert float(ref.e4m3(torch.tensor(1e9, dtype=torch.float64))) == 448


def test_comparison_notices_mistakes():
    """`within` refuses a result that misses one term, one step, or a NaN."""
    g = torch.Generator().manual_seed(4)
    a = rnd(g, 100)
    for dtype in (torch.float32, torch.bfloat16):
        got = a.to(dtype)
        ref.within(got, a, a.abs(), 4, "rounded")
        for bad in (got * (1 + 2 * torch.finfo(dtype).eps),
                    torch.where(torch.arange(100) == 7, torch.nan, got.double()).to(dtype),
                    got.roll(1)):
            with pytest.raises(AssertionError):
                ref.within(bad, a, a.abs(), 1, "mistake")
