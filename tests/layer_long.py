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


# ------------------------------------------------------- pieces of operands ----
# One sequence whose states tell operands of two bf16 pieces from ones of three,
# and whose gradients of A tell one from three.  fp32 arithmetic on three pieces: a chunk adds
# twelve sums in the tensor pipe, which truncates, 2^-24 of a partial sum each
# on average, which is half of the whole on average; a rounding of the state and
# one of its decay, and the exponentials of a token (2^-24 on average): 6e-7.
# Where a state meets an adjoint, the two errors' squares add up, and the sums
# over the chunk's tokens are twelve truncations more: 1.1e-6.
STATE_BOUND, DA_BOUND = 1e-6, 1.5e-6


def pieces_case():
    """(x, raw, A, B, C, D, bias, state, dy, dlast); bf16 values where the call's
    inputs are bf16."""
    T, H, P, G, N = 1024, 4, 64, 1, 128
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g)
    b = lambda *s: r(*s).to(torch.bfloat16)
    return (b(1, T, H, P), b(1, T, H), -(torch.rand(H, generator=g) * 15 + 1), b(1, T, G, N),
            b(1, T, G, N), r(H), torch.full((H,), math.log(math.expm1(0.01))), r(1, H, N, P),
            b(1, T, H, P), r(1, H, N, P))


def pieces(t, k):
    """t as the sum of k bf16 values, each the rounding of what is left."""
    out, rest = torch.zeros_like(t), t.clone()
    for _ in range(k):
        p = rest.float().to(torch.bfloat16).double()
        out, rest = out + p, rest - p
    return out


def with_pieces(case, k):
    """(last state, dA) in 64 bits but for operands in k bf16 pieces: w x as it
    enters the state, states and adjoints as they enter the gradient."""
    x, raw, A, B, C, _, bias, h, dy, dlast = (t.double() for t in case)
    v = raw[0] + bias
    dt = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    H = x.shape[2]
    x, dy, h = x[0], dy[0], h[0]
    B, C = (t[0].repeat_interleave(H // t.shape[2], 1) for t in (B, C))
    cuts = [slice(t, t + CHUNK) for t in range(0, x.shape[0], CHUNK)]
    starts, state = [], h
    for s in cuts:
        starts.append(h)
        h = _one(x[s], dt[s], A, B[s], C[s], h)[1]
        c = (dt[s] * A).cumsum(0)
        wx = pieces(x[s] * (torch.exp(c[-1] - c) * dt[s])[..., None], k)
        state = torch.exp(c[-1])[:, None, None] * state + B[s].permute(1, 2, 0) @ wx.transpose(0, 1)
    g, dA = dlast[0], 0.0
    for s, h0 in zip(reversed(cuts), reversed(starts)):
        a = A.clone().requires_grad_(True)
        out = _one(x[s], dt[s], a, B[s], C[s], pieces(h0, k))
        dA = dA + torch.autograd.grad(out, a, [dy[s], pieces(g, k)])[0]
        h0 = h0.clone().requires_grad_(True)
        g = torch.autograd.grad(_one(x[s], dt[s], A, B[s], C[s], h0), h0, [dy[s], g])[0]
    return state[None], dA
