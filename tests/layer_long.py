"""64-bit scan in chunks of matrix products, for sequences and head counts that
the token-by-token reference is too slow for.  Differentiable, so that its
gradients are autograd's, and on any device.  Pinned to the token-by-token
reference by ``test_layer_long.py``."""

import math

import torch

CHUNK = 64


def _one(x, dt, A, B, C, h):
    """One sequence: x [T, H, P], dt [T, H], B, C [T, H, N] (a row a head),
    h [H, N, P].  Returns y without the skip term, and the last state."""
    ys = [x.new_zeros((0,) + x.shape[1:])]
    for t in range(0, x.shape[0], CHUNK):
        s = slice(t, t + CHUNK)
        c = (dt[s] * A).cumsum(0).t()                                   # H L
        gap = c[:, :, None] - c[:, None, :]
        keep = torch.ones(gap.shape[1:], dtype=torch.bool, device=x.device).tril()
        decay = torch.exp(gap.masked_fill(~keep, -math.inf))
        u = (x[s] * dt[s][..., None]).transpose(0, 1)                   # H L P
        b, k = B[s].transpose(0, 1), C[s].transpose(0, 1)               # H L N
        ys.append((((k @ b.transpose(1, 2)) * decay) @ u
                   + torch.exp(c)[..., None] * (k @ h)).transpose(0, 1))
        h = torch.exp(c[:, -1])[:, None, None] * h \
            + (b * torch.exp(c[:, -1:] - c)[..., None]).transpose(1, 2) @ u
    return torch.cat(ys), h


def scan(x, raw, A, B, C, D, bias, state, cu):
    """(y, last) of gdn_scan_prefill's arguments, all in 64 bits."""
    G, N = B.shape[2:]
    H, P = x.shape[2:]
    n = x.shape[0] if cu is None else len(cu) - 1
    v = raw if bias is None else raw + bias
    dt = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    Bh, Ch = B.repeat_interleave(H // G, 2), C.repeat_interleave(H // G, 2)
    first = x.new_zeros((n, H, N, P)) if state is None else state
    ys, last = [], []
    for i in range(n):
        at = (i, slice(None)) if cu is None else (0, slice(int(cu[i]), int(cu[i + 1])))
        y, h = _one(x[at], dt[at], A, Bh[at], Ch[at], first[i])
        ys.append(y)
        last.append(h)
    y = torch.stack(ys) if cu is None else torch.cat(ys)[None]
    return y + (0 if D is None else D[:, None] * x), torch.stack(last)


def scan_grad(x, raw, A, B, C, D, bias, state, cu, dy, dlast):
    """(y, last, dx, draw, dA, dB, dC, dD, dbias, dstate); every input given."""
    ins = [t.detach().double().requires_grad_(True) for t in (x, raw, A, B, C, D, bias, state)]
    y, last = scan(*ins, cu)
    grads = torch.autograd.grad([y, last], ins, [dy.double(), dlast.double()])
    return (y.detach(), last.detach()) + tuple(grads)


def off(got, want):
    """2-norm of the difference over the 2-norm of what is wanted."""
    want = want.double()
    return float((got.double() - want).norm() / want.norm())
