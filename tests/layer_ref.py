"""64-bit reference of the convolution, the scan and the norm, token by token
from their definitions, with the gradients written out.

Every gradient and output is a sum of products whose signs are those of the
inputs, so the same function on the inputs' absolute values gives the sum of
the terms' magnitudes: what rounding errors are measured against.
"""

import torch


def ranges(n_seq, T, cu):
    """(batch row, first token, one past the last) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(n_seq)]
    cu = [int(v) for v in cu]
    return [(0, cu[i], cu[i + 1]) for i in range(n_seq)]


def dbl(*ts):
    return [None if t is None else t.detach().double().cpu() for t in ts]


# -------------------------------------------------------------------- conv ----
def conv(x, w, b, state, cu, silu=True, dy=None, dlast=None, mag=False):
    """y, last (and dx, dw, db, dstate for dy).  mag: magnitudes - the
    activation's slope (at most 1.1) and value bounded by those of |x|."""
    x, w, b, state, dy, dlast = dbl(x, w, b, state, dy, dlast)
    if mag:
        x, w, b, state, dy, dlast = [None if t is None else t.abs()
                                     for t in (x, w, b, state, dy, dlast)]
    C, W = w.shape
    n_seq = x.shape[0] if cu is None else len(cu) - 1
    b = torch.zeros(C, dtype=torch.float64) if b is None else b
    y = torch.zeros_like(x)
    last = torch.zeros((n_seq, W - 1, C), dtype=torch.float64)
    dx, dw, db, ds = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b), last.clone()
    for i, (r, lo, hi) in enumerate(ranges(n_seq, x.shape[1], cu)):
        h = torch.zeros((W - 1, C), dtype=torch.float64) if state is None else state[i]
        h = torch.cat([h, x[r, lo:hi]])
        n = hi - lo
        last[i] = h[n:]
        pre = sum((h[j:j + n] * w[:, j] for j in range(W)), b.expand(n, C))
        sig = torch.sigmoid(pre)
        if not silu or mag:
            act, slope = pre, torch.full_like(pre, 1.1 if silu else 1.0)
        else:
            act, slope = pre * sig, sig * (1 + pre * (1 - sig))
        y[r, lo:hi] = act
        if dy is not None:
            dh = torch.zeros_like(h)
            if dlast is not None:
                dh[n:] += dlast[i]
            dp = dy[r, lo:hi] * slope
            for j in range(W):
                dh[j:j + n] += dp * w[:, j]
                dw[:, j] += (dp * h[j:j + n]).sum(0)
            db += dp.sum(0)
            ds[i], dx[r, lo:hi] = dh[:W - 1], dh[W - 1:]
    return (y, last) if dy is None else (y, last, dx, dw, db, ds)


# -------------------------------------------------------------------- scan ----
def scan(x, raw, A, B, C, D, bias, state, cu, dy=None, dlast=None, mag=False):
    """y, last (and dx, draw, dA, dB, dC, dD, dbias, dstate for dy)."""
    x, raw, A, B, C, D, bias, state, dy, dlast = dbl(x, raw, A, B, C, D, bias, state, dy, dlast)
    if mag:
        x, B, C, D, state, dy, dlast = [None if t is None else t.abs()
                                        for t in (x, B, C, D, state, dy, dlast)]
    H, P = x.shape[2:]
    G, N = B.shape[2:]
    R = H // G
    n_seq = x.shape[0] if cu is None else len(cu) - 1
    z = torch.zeros(H, dtype=torch.float64)
    D, bias = z if D is None else D, z if bias is None else bias
    v = raw + bias
    dt = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    a, u = torch.exp(dt * A), dt[..., None] * x
    Bh, Ch = B.repeat_interleave(R, 2), C.repeat_interleave(R, 2)
    y = torch.zeros_like(x)
    last = torch.zeros((n_seq, H, N, P), dtype=torch.float64)
    da = torch.zeros_like(dt)                    # of the log decay dt A
    du, dBh, dCh, ds = torch.zeros_like(x), torch.zeros_like(Bh), torch.zeros_like(Ch), last.clone()
    for i, (r, lo, hi) in enumerate(ranges(n_seq, x.shape[1], cu)):
        h = last[i].clone() if state is None else state[i]
        hs = [h]
        for t in range(lo, hi):
            h = a[r, t, :, None, None] * h + Bh[r, t, :, :, None] * u[r, t, :, None, :]
            y[r, t] = (Ch[r, t, :, :, None] * h).sum(1) + D[:, None] * x[r, t]
            if dy is not None:
                hs.append(h)
        last[i] = h
        if dy is not None:
            g = torch.zeros_like(h) if dlast is None else dlast[i].clone()
            for t in reversed(range(lo, hi)):
                g = g + Ch[r, t, :, :, None] * dy[r, t, :, None, :]
                dCh[r, t] = (hs[t - lo + 1] * dy[r, t, :, None, :]).sum(-1)
                dBh[r, t] = (g * u[r, t, :, None, :]).sum(-1)
                du[r, t] = (g * Bh[r, t, :, :, None]).sum(1)
                g = g * a[r, t, :, None, None]
                da[r, t] = (g * hs[t - lo]).sum((-1, -2))
            ds[i] = g
    if dy is None:
        return y, last
    ddt = da * (A.abs() if mag else A) + (x * du).sum(-1)
    draw = ddt * torch.sigmoid(v)
    dx = dt[..., None] * du + D[:, None] * dy
    fold = lambda t: t.unflatten(2, (G, R)).sum(3)
    return (y, last, dx, draw, (dt * da).sum((0, 1)), fold(dBh), fold(dCh),
            (dy * x).sum((0, 1, 3)), draw.sum((0, 1)), ds)


# -------------------------------------------------------------------- norm ----
def norm(x, w, residual=None, gate=None, eps=1e-6, dtype=None):
    """(y, s): s rounded to `dtype`, the type in which the stream is kept."""
    x, w, residual, gate = dbl(x, w, residual, gate)
    if residual is not None:
        x = (x + residual).to(dtype).double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if gate is not None:
        y = y * gate * torch.sigmoid(gate)
    return y, x


def norm_grad(s, w, dy, gate=None, dres=None, eps=1e-6, mag=False):
    """(ds, dw, dgate); mag: the sum of the magnitudes of ds's terms instead."""
    s, w, dy, gate, dres = dbl(s, w, dy, gate, dres)
    d = s.shape[-1]
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    n = s * r
    f, slope = 1.0, None
    if gate is not None:
        sg = torch.sigmoid(gate)
        f, slope = gate * sg, sg * (1 + gate * (1 - sg))
    dn = dy * w * f
    dgate = None if gate is None else dy * n * w * slope
    rows = tuple(range(s.dim() - 1))
    if mag:
        ds = r * (dn.abs() + n.abs() * (dn.abs() * n.abs()).sum(-1, keepdim=True) / d)
        ds = ds if dres is None else ds + dres.abs()
        return ds, (dy * f * n).abs().sum(rows), None if dgate is None else dgate.abs()
    ds = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    ds = ds if dres is None else ds + dres
    return ds, (dy * f * n).sum(rows), dgate


# ------------------------------------------------------------------ codecs ----
def e4m3(v):
    """Nearest E4M3 value in 64 bits: 3 mantissa bits down to 2^-6, a fixed
    step of 2^-9 below, ties to even, saturating at 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=-5) - 4)
    return torch.clamp(torch.round(v / step) * step, -448, 448)


# -------------------------------------------------------------- comparison ----
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, mag, terms, name, extra=0.0, floor=0.0):
    """Every element within one rounding to its type plus `terms` fp32
    roundings (and `extra`, relative) of the magnitudes that were added.
    Values below the type's normal range carry half its smallest step, and
    `floor` stands for one that the call's own arithmetic has."""
    dtype = got.dtype
    g, ref, mag = got.detach().double().cpu(), ref, mag
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    tiny = torch.finfo(dtype).tiny
    tol = half_step(dtype) * (ref.abs() + tiny) + (terms * U + extra) * (mag + tiny) + floor
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        name, int(bad.sum()), bad.numel(), float(((g - ref).abs() / tol).max()))
