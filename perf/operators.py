"""The operators of a recurrent layer around and beside the gated delta rule,
as a user's program calls them: the short causal convolution in front of the
recurrence, the selective state space scan, and the root-mean-square norm
(with the residual's addition, the output gate, or an 8-bit output).

``own = False`` computes each operator in its plain form (elementary torch
operations, 32 bits, decays and their sums in 64); ``own = True`` calls the
library.  ``exact`` gives the same outputs from the definitions, token by
token, in 64 bits.

    scan   dt_t = softplus(raw_t + bias);  S_t = exp(dt_t A) S_{t-1} + B_t (dt_t x_t)^T
           y_t = S_t^T C_t + D x_t          (S: [N, P] a head, B and C shared by H / G heads)
    conv   y_t = silu(bias + sum_j w_j x_{t-W+1+j}), a channel at a time
    norm   s = x + residual;  y = s / sqrt(mean(s^2) + eps) * w * silu(gate)
"""

import math
import random

import torch

own = False

CHUNK = 64
EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # a batch of equal prompts through one layer's scan
        dict(name="scan-prompts", op="scan_prefill", dtype="bf16", n_seq=4, T=4096, lens=0,
             H=16, P=128, G=1, N=128, state=False),
        # continued prompts of very different lengths, packed one behind the other
        dict(name="scan-packed", op="scan_prefill", dtype="bf16", n_seq=64, T=4096, lens=11,
             H=16, P=64, G=2, N=128, state=True),
        # one user's long prompt: few heads, one odd length, nothing to batch
        dict(name="scan-one-long", op="scan_prefill", dtype="bf16", n_seq=1, T=8191, lens=0,
             H=8, P=64, G=1, N=128, state=False),
        # a training step's gradient of the scan
        dict(name="scan-train", op="scan_backward", dtype="bf16", n_seq=2, T=4096, lens=0,
             H=16, P=64, G=1, N=128, state=False),
        # a small check of a training program in full precision, packed documents
        dict(name="scan-train-f32", op="scan_backward", dtype="f32", n_seq=7, T=300, lens=5,
             H=6, P=128, G=2, N=64, state=True),
        # one token for every sequence of a serving batch
        dict(name="scan-token", op="scan_decode", dtype="bf16", n_seq=256, H=32, P=128, G=1,
             N=128),
        # the convolution of the same batch of prompts (x, B and C side by side)
        dict(name="conv-prompts", op="conv_prefill", dtype="bf16", n_seq=4, T=4096, lens=0,
             C=4352, W=4, state=False),
        # its gradient over packed documents
        dict(name="conv-train", op="conv_backward", dtype="bf16", n_seq=16, T=1500, lens=3,
             C=2304, W=4, state=True),
        # one token for every sequence: latency counts
        dict(name="conv-token", op="conv_decode", dtype="bf16", n_seq=256, C=4352, W=4),
        # the block's entry: residual stream, norm, 8-bit rows for the projection
        dict(name="norm-residual-fp8", op="norm", dtype="bf16", rows=16384, d=2048,
             residual=True, gate=False, out="fp8_row"),
        # the gated norm of every head's output, one token of a serving batch
        dict(name="norm-heads-token", op="norm", dtype="bf16", rows=8192, d=128,
             residual=False, gate=True, out="none"),
        # the gradient of the block's norm in training
        dict(name="norm-train", op="norm_backward", dtype="bf16", rows=16384, d=2048,
             residual=True, gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_prefill", "scan_prefill", "scan_backward", "scan_decode",
                     "conv_prefill", "conv_backward", "conv_decode", "norm", "norm_backward"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op.startswith("scan"):
        G = rng.choice([1, 1, 2, 4])
        c.update(G=G, H=G * rng.choice([1, 2, 3, 4, 8]), P=rng.choice([64, 128]),
                 N=rng.choice([64, 128]))
        if op == "scan_decode":
            c["n_seq"] = _log(rng, 1, 256)
            return c
        most = 5e5 if op == "scan_backward" else 2e6    # tokens x heads x (P / 64)
    elif op.startswith("conv"):
        c.update(C=rng.choice([8, 1]) * _log(rng, 5, 500), W=rng.choice([2, 3, 4, 4]))
        if op == "conv_decode":
            c["n_seq"] = _log(rng, 1, 256)
            return c
        most = 3e7
    else:
        d = rng.choice([64, 128, 256, 1024, 2048, 4096, 8 * _log(rng, 2, 600), _log(rng, 5, 5000)])
        c.update(rows=max(1, min(_log(rng, 1, 30000), int(2.5e7 / d))), d=d,
                 residual=rng.random() < 0.5, gate=rng.random() < 0.5)
        if op == "norm":
            c["out"] = "fp8_row" if c["dtype"] == "bf16" and rng.random() < 0.5 else "none"
        return c
    width = c["H"] * (c["P"] // 64) if "H" in c else c["C"]
    n = _log(rng, 1, 32)
    c.update(n_seq=n, T=max(1, min(_log(rng, 1, 8000), int(most / width / n))),
             lens=rng.choice([0, rng.randint(1, 1 << 20)]), state=rng.random() < 0.5)
    return c


def _lengths(c):
    """Lengths of the packed sequences (one of them may be empty), or None."""
    if not c.get("lens"):
        return None
    r = random.Random(c["lens"])
    n = [r.randint(0, c["T"]) for _ in range(c["n_seq"])]
    n[r.randrange(len(n))] = c["T"]
    return n


def _tokens(c):
    n = _lengths(c)
    return c["n_seq"] * c["T"] if n is None else sum(n)


# ---------------------------------------------------------------- prepare ----
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(int(seed))
    dt = DTYPE[c["dtype"]]

    def randn(*shape, scale=1.0, to=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(to)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=c)
    op = c["op"]
    if op in ("scan_prefill", "scan_backward", "conv_prefill", "conv_backward"):
        n = _lengths(c)
        lead = (c["n_seq"], c["T"]) if n is None else (1, sum(n))
        ends = [0]
        for v in n or []:
            ends.append(ends[-1] + v)
        s["cu_seqlens"] = None if n is None else torch.tensor(ends, dtype=torch.int32,
                                                              device="cuda")
    else:
        lead = (c.get("n_seq"),)
    if op.startswith("scan"):
        H, P, G, N = c["H"], c["P"], c["G"], c["N"]
        # x, B and C are slices of the convolution's output, dt of the projection's
        xbc = randn(*lead, H * P + 2 * G * N)
        s["x"] = xbc[..., : H * P].unflatten(-1, (H, P))
        s["B"] = xbc[..., H * P: H * P + G * N].unflatten(-1, (G, N))
        s["C"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
        s["dt"] = randn(*lead, H + 8)[..., 8:]
        s["A"] = -uniform(1.0, 16.0, H)
        s["D"] = uniform(0.5, 1.5, H)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        s["dt_bias"] = torch.log(torch.expm1(step))     # softplus(dt_bias) = step
        if op == "scan_decode":
            s["state"] = randn(*lead, H, N, P, scale=0.5, to=torch.float32)
        else:
            s["state_in"] = randn(c["n_seq"], H, N, P, scale=0.5, to=torch.float32) \
                if c["state"] else None
        if op == "scan_backward":
            s["dy"] = randn(*lead, H, P)
            s["dstate_out"] = randn(c["n_seq"], H, N, P, scale=0.1, to=torch.float32) \
                if c["state"] else None
    elif op.startswith("conv"):
        C, W = c["C"], c["W"]
        # the channels are a slice of the projection's output
        s["x"] = randn(*lead, C + 64)[..., 64:]
        s["weight"] = randn(C, W, scale=0.5, to=torch.float32)
        s["bias"] = randn(C, scale=0.1, to=torch.float32)
        if op == "conv_decode":
            s["state"] = randn(*lead, W - 1, C)
        else:
            s["state_in"] = randn(c["n_seq"], W - 1, C) if c["state"] else None
        if op == "conv_backward":
            s["dy"] = randn(*lead, C)
            s["dstate_out"] = randn(c["n_seq"], W - 1, C) if c["state"] else None
    else:
        rows, d = c["rows"], c["d"]
        s["x"] = randn(rows, d)
        s["weight"] = uniform(0.5, 1.5, d)
        s["gate"] = randn(rows, d) if c["gate"] else None
        if op == "norm":
            s["residual"] = randn(rows, d, scale=2.0) if c["residual"] else None
        else:
            s["dy"] = randn(rows, d)
            s["dresidual"] = randn(rows, d) if c["residual"] else None
    return s


# -------------------------------------------------------------------- run ----
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import state_quantized_recurrence_b200 as sqr
        if op == "scan_prefill":
            return sqr.gdn_scan_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                                        dt_bias=s["dt_bias"], state_in=s["state_in"],
                                        cu_seqlens=s["cu_seqlens"])
        if op == "scan_backward":
            return sqr.gdn_scan_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"],
                                         D=s["D"], dt_bias=s["dt_bias"],
                                         state_in=s["state_in"], cu_seqlens=s["cu_seqlens"],
                                         dstate_out=s["dstate_out"])
        if op == "scan_decode":
            y = sqr.gdn_scan_decode(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"],
                                    D=s["D"], dt_bias=s["dt_bias"])
            return y, s["state"]
        if op == "conv_prefill":
            return sqr.gdn_conv_prefill(s["x"], s["weight"], s["bias"], s["state_in"],
                                        s["cu_seqlens"])
        if op == "conv_backward":
            return sqr.gdn_conv_backward(s["x"], s["weight"], s["dy"], s["bias"],
                                         s["state_in"], s["cu_seqlens"], s["dstate_out"])
        if op == "conv_decode":
            y = sqr.gdn_conv_decode(s["x"], s["weight"], s["bias"], s["state"])
            return y, s["state"]
        if op == "norm":
            y, res = sqr.gdn_norm(s["x"], s["weight"], residual=s["residual"], gate=s["gate"],
                                  eps=EPS, qdq=c["out"])
            y = (y,) if c["out"] == "none" else (y.codes, y.scales)
            return y if res is None else y + (res,)
        dx, dw, dgate = sqr.gdn_norm_backward(s["x"], s["weight"], s["dy"], gate=s["gate"],
                                              dresidual=s["dresidual"], eps=EPS)
        return (dx, dw) if dgate is None else (dx, dw, dgate)
    if op == "scan_prefill":
        return _plain_scan(c, *_floats(s, "x dt A B C D dt_bias state_in"), s["cu_seqlens"])
    if op == "scan_backward":
        return _plain_scan_backward(s)
    if op == "scan_decode":
        return _plain_scan_decode(s)
    if op == "conv_prefill":
        return _plain_conv(c, *_floats(s, "x weight bias state_in"), s["cu_seqlens"])
    if op == "conv_backward":
        return _plain_conv_backward(s)
    if op == "conv_decode":
        return _plain_conv_decode(s)
    if op == "norm":
        return _plain_norm(s)
    return _plain_norm_backward(s)


def _floats(s, names):
    return [None if s[k] is None else s[k].float() for k in names.split()]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


# ------------------------------------------------------------ plain: scan ----
def _place(cu):
    """(sequence, position in it) of every packed token."""
    t = torch.arange(int(cu[-1]), device=cu.device)
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    return seq, t - cu.long()[seq]


def _pad(c, t, cu):
    """[n_seq, T', ...] with T' a multiple of the chunk, zeros behind each sequence."""
    T = -(-c["T"] // CHUNK) * CHUNK
    out = torch.zeros((c["n_seq"], T) + t.shape[2:], dtype=t.dtype, device=t.device)
    if cu is None:
        out[:, : c["T"]] = t
    else:
        out[_place(cu)] = t[0]
    return out


def _unpad(c, t, cu):
    return t[:, : c["T"]] if cu is None else t[_place(cu)][None]


def _scan_chunks(x, dt, A, B, C, h0):
    """y without the skip term and the last state, chunk by chunk in matrix form."""
    b, T, H, P = x.shape
    G, N = B.shape[2:]
    L, nc, R = CHUNK, T // CHUNK, H // G
    cum = (dt.double() * A.double()).view(b, nc, L, H).permute(0, 3, 1, 2).cumsum(-1)
    below = torch.ones(L, L, dtype=torch.bool, device=x.device).tril()
    gap = (cum[..., :, None] - cum[..., None, :]).masked_fill(~below, -math.inf)
    decay = torch.exp(gap).float()                                        # b H nc i j
    Bc = B.view(b, nc, L, G, N).permute(0, 3, 1, 2, 4)
    Cc = C.view(b, nc, L, G, N).permute(0, 3, 1, 2, 4)                    # b G nc L N
    u = (x * dt[..., None]).view(b, nc, L, H, P).permute(0, 3, 1, 2, 4)   # b H nc L P
    CB = (Cc @ Bc.transpose(-1, -2)).repeat_interleave(R, 1)
    y = (CB * decay) @ u
    Bh, Ch = Bc.repeat_interleave(R, 1), Cc.repeat_interleave(R, 1)
    to_end = torch.exp(cum[..., -1:] - cum).float()
    part = (Bh * to_end[..., None]).transpose(-1, -2) @ u                 # b H nc N P
    far = torch.cat([torch.zeros_like(cum[..., 0, -1:]), cum[..., -1].cumsum(-1)], -1)
    span = far[..., :, None] - far[..., None, :]                          # nc+1 x nc+1
    before = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp(span.masked_fill(~before, -math.inf)).float()
    first = torch.zeros_like(part[:, :, 0]) if h0 is None else h0
    parts = torch.cat([first[:, :, None], part], 2).flatten(3)            # b H nc+1 NP
    states = (carry @ parts).view(b, H, nc + 1, N, P)
    y = y + torch.exp(cum).float()[..., None] * (Ch @ states[:, :, :-1])
    return y.permute(0, 2, 3, 1, 4).reshape(b, T, H, P), states[:, :, -1]


def _scan_all(c, x, dt, A, B, C, D, dt_bias, h0, cu):
    step = _softplus(dt + dt_bias)
    y, last = _scan_chunks(_pad(c, x, cu), _pad(c, step, cu), A, _pad(c, B, cu),
                           _pad(c, C, cu), h0)
    return _unpad(c, y, cu) + D[:, None] * x, last


def _plain_scan(c, x, dt, A, B, C, D, dt_bias, h0, cu):
    y, last = _scan_all(c, x, dt, A, B, C, D, dt_bias, h0, cu)
    return y.to(DTYPE[c["dtype"]]), last


def _plain_scan_backward(s):
    c = s["case"]
    ins = _floats(s, "x dt A B C D dt_bias state_in")
    if ins[-1] is None:
        ins[-1] = torch.zeros((c["n_seq"], c["H"], c["N"], c["P"]), device="cuda")
    ins = [t.detach().requires_grad_(True) for t in ins]
    with torch.enable_grad():
        y, last = _scan_all(c, *ins, s["cu_seqlens"])
    d_last = torch.zeros_like(last) if s["dstate_out"] is None else s["dstate_out"]
    dx, ddt, dA, dB, dC, dD, dbias, dh0 = torch.autograd.grad([y, last], ins,
                                                             [s["dy"].float(), d_last])
    to = DTYPE[c["dtype"]]
    return dx.to(to), ddt.to(to), dA, dB.to(to), dC.to(to), dD, dbias, dh0


def _plain_scan_decode(s):
    x, dt, A, B, C, D, dt_bias = _floats(s, "x dt A B C D dt_bias")
    R = x.shape[1] // B.shape[1]
    B, C = B.repeat_interleave(R, 1), C.repeat_interleave(R, 1)
    step = _softplus(dt + dt_bias)
    h = s["state"] * torch.exp(step * A)[..., None, None] \
        + B[..., None] * (step[..., None] * x)[..., None, :]
    y = (C[..., None] * h).sum(2) + D[:, None] * x
    s["state"].copy_(h)
    return y.to(s["x"].dtype), s["state"]


# ------------------------------------------------------------ plain: conv ----
def _conv_all(c, x, weight, bias, state, cu):
    """Every sequence's rows behind the W - 1 rows of its state, in one buffer."""
    n, W, C = c["n_seq"], c["W"], c["C"]
    x = x.reshape(-1, C)
    if cu is None:
        cu = torch.arange(n + 1, device=x.device) * c["T"]
    seq, _ = _place(cu)
    at = torch.arange(x.shape[0], device=x.device) + (seq + 1) * (W - 1)
    head = (cu[:-1].long() + torch.arange(n, device=x.device) * (W - 1))[:, None] \
        + torch.arange(W - 1, device=x.device)
    tail = (cu[1:].long() + torch.arange(n, device=x.device) * (W - 1))[:, None] \
        + torch.arange(W - 1, device=x.device)
    rows = torch.zeros((x.shape[0] + n * (W - 1), C), device=x.device)
    rows = rows.index_copy(0, at, x)
    if state is not None:
        rows = rows.index_copy(0, head.reshape(-1), state.reshape(-1, C))
    m = rows.shape[0] - W + 1
    pre = sum((rows[j: j + m] * weight[:, j] for j in range(W)), bias)
    return _silu(pre)[at - (W - 1)], rows[tail.reshape(-1)].view(n, W - 1, C)


def _plain_conv(c, x, weight, bias, state, cu):
    y, last = _conv_all(c, x, weight, bias, state, cu)
    to = DTYPE[c["dtype"]]
    return y.reshape(x.shape).to(to), last.to(to)


def _plain_conv_backward(s):
    c = s["case"]
    x, weight, bias, state = _floats(s, "x weight bias state_in")
    if state is None:
        state = torch.zeros((c["n_seq"], c["W"] - 1, c["C"]), device="cuda")
    ins = [t.detach().requires_grad_(True) for t in (x, weight, bias, state)]
    with torch.enable_grad():
        y, last = _conv_all(c, *ins, s["cu_seqlens"])
    d_last = torch.zeros_like(last) if s["dstate_out"] is None else s["dstate_out"].float()
    dx, dw, db, ds = torch.autograd.grad([y, last], ins,
                                         [s["dy"].float().reshape(y.shape), d_last])
    to = DTYPE[c["dtype"]]
    return dx.to(to), dw, db, ds.to(to)


def _plain_conv_decode(s):
    x, weight, bias, state = _floats(s, "x weight bias state")
    rows = torch.cat([state, x[:, None]], 1)
    y = _silu((rows * weight.t()).sum(1) + bias)
    s["state"].copy_(rows[:, 1:])
    return y.to(s["x"].dtype), s["state"]


# ------------------------------------------------------------ plain: norm ----
def _plain_norm(s):
    x, w, gate = _floats(s, "x weight gate")
    to = s["x"].dtype
    res = None
    if s["residual"] is not None:
        res = (x + s["residual"].float()).to(to)
        x = res.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if gate is not None:
        y = y * _silu(gate)
    if s["case"]["out"] == "none":
        out = (y.to(to),)
    else:
        scale = y.abs().amax(-1) / 448
        code = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y))
        out = (code.to(torch.float8_e4m3fn), scale)
    return out if res is None else out + (res,)


def _plain_norm_backward(s):
    x, w, dy, gate, dres = _floats(s, "x weight dy gate dresidual")
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    to = s["x"].dtype
    dgate = None
    if gate is not None:
        sig = 1 / (1 + torch.exp(-gate))
        dgate = (dy * n * w * sig * (1 + gate * (1 - sig))).to(to)
        dy = dy * gate * sig
    dw = (dy * n).sum(0)
    g = dy * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if dres is not None:
        dx = dx + dres
    return (dx.to(to), dw) if dgate is None else (dx.to(to), dw, dgate)


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op.startswith("scan"):
        H, P, G, N = c["H"], c["P"], c["G"], c["N"]
        state = 4.0 * c["n_seq"] * H * N * P
        if op == "scan_decode":
            t = c["n_seq"]
            return dict(bytes=e * t * (2 * H * P + 2 * G * N + H) + 2 * state,
                        flops=5.0 * t * H * N * P)
        t = _tokens(c)
        if op == "scan_prefill":
            return dict(bytes=e * t * (2 * H * P + 2 * G * N + H)
                        + state * (2 if c["state"] else 1),
                        flops=4.0 * t * H * N * P)
        return dict(bytes=e * t * (3 * H * P + 4 * G * N + 2 * H)
                    + state * (3 if c["state"] else 1),
                    flops=10.0 * t * H * N * P)
    if op.startswith("conv"):
        C, W = c["C"], c["W"]
        state = float(e) * c["n_seq"] * (W - 1) * C
        if op == "conv_decode":
            return dict(bytes=2.0 * e * c["n_seq"] * C + 2 * state + 4 * C * (W + 1),
                        flops=(2.0 * W + 4) * c["n_seq"] * C)
        t = _tokens(c)
        if op == "conv_prefill":
            return dict(bytes=2.0 * e * t * C + state * (2 if c["state"] else 1)
                        + 4 * C * (W + 1), flops=(2.0 * W + 4) * t * C)
        return dict(bytes=3.0 * e * t * C + state * (3 if c["state"] else 1)
                    + 8 * C * (W + 1), flops=(6.0 * W + 8) * t * C)
    n = float(c["rows"]) * c["d"]
    if op == "norm":
        planes = 1 + 2 * c["residual"] + c["gate"]
        out = n + 4 * c["rows"] if c["out"] == "fp8_row" else e * n
        return dict(bytes=e * n * planes + out + 4 * c["d"], flops=6.0 * n)
    return dict(bytes=e * n * (3 + c["residual"] + 2 * c["gate"]) + 8 * c["d"], flops=12.0 * n)


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in s.items()}
    op = c["op"]
    if op == "scan_prefill":
        return _exact_scan(c, d)
    if op == "scan_backward":
        return _exact_scan_backward(c, d)
    if op == "scan_decode":
        R = c["H"] // c["G"]
        dt = torch.logaddexp(d["dt"] + d["dt_bias"], torch.zeros_like(d["dt"]))
        h = torch.exp(dt * d["A"])[:, :, None, None] * d["state"] + torch.einsum(
            "bhn,bhp,bh->bhnp", d["B"].repeat_interleave(R, 1), d["x"], dt)
        y = torch.einsum("bhnp,bhn->bhp", h, d["C"].repeat_interleave(R, 1))
        return y + d["D"][None, :, None] * d["x"], h
    if op == "conv_prefill":
        return _exact_conv(c, d)
    if op == "conv_backward":
        return _exact_conv_backward(c, d)
    if op == "conv_decode":
        h = torch.cat([d["state"], d["x"][:, None]], 1)
        pre = torch.einsum("bwc,cw->bc", h, d["weight"]) + d["bias"]
        return pre * torch.sigmoid(pre), h[:, 1:]
    return _exact_norm(c, s, d) if op == "norm" else _exact_norm_backward(d)


def _ranges(c):
    """[(batch row, first token, one past the last)] of every sequence."""
    n = _lengths(c)
    if n is None:
        return [(b, 0, c["T"]) for b in range(c["n_seq"])]
    out, at = [], 0
    for v in n:
        out.append((0, at, at + v))
        at += v
    return out


def _side_by_side(c, t):
    """Sequences as rows of [n_seq, T, ...], zeros behind their ends."""
    out = t.new_zeros((c["n_seq"], c["T"]) + t.shape[2:])
    for i, (b, lo, hi) in enumerate(_ranges(c)):
        out[i, : hi - lo] = t[b, lo:hi]
    return out


def _one_behind_the_other(c, t):
    n = _lengths(c)
    return t if n is None else torch.cat([t[i, :v] for i, v in enumerate(n)])[None]


def _scan_steps(c, d):
    raw = d["dt"] + d["dt_bias"]
    dt = _side_by_side(c, torch.logaddexp(raw, torch.zeros_like(raw)))
    x, B, C = (_side_by_side(c, d[k]) for k in ("x", "B", "C"))
    R = c["H"] // c["G"]
    h = d["state_in"]
    if h is None:
        h = x.new_zeros((c["n_seq"], c["H"], c["N"], c["P"]))
    return raw, dt, x, B.repeat_interleave(R, 2), C.repeat_interleave(R, 2), h


def _exact_scan(c, d):
    raw, dt, x, B, C, h = _scan_steps(c, d)
    y = torch.empty_like(x)
    a, u = torch.exp(dt * d["A"]), dt[..., None] * x
    h = h.clone()
    for t in range(c["T"]):
        h.mul_(a[:, t, :, None, None]).addcmul_(B[:, t, :, :, None], u[:, t, :, None, :])
        y[:, t] = (C[:, t, :, None, :] @ h)[:, :, 0]
    return _one_behind_the_other(c, y) + d["D"][:, None] * d["x"], h


def _exact_scan_backward(c, d):
    raw, dt, x, B, C, h = _scan_steps(c, d)
    dy = _side_by_side(c, d["dy"])
    a, u = torch.exp(dt * d["A"]), dt[..., None] * x
    T, K = c["T"], 32

    def step(h, t):
        return h * a[:, t, :, None, None] + B[:, t, :, :, None] * u[:, t, :, None, :]

    marks = []
    for t in range(T):
        if t % K == 0:
            marks.append(h)
        h = step(h, t)
    g = torch.zeros_like(h) if d["dstate_out"] is None else d["dstate_out"]
    du, dB, dC = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C)
    da = torch.empty_like(dt)
    for k in reversed(range(len(marks))):
        hs = [marks[k]]
        for t in range(k * K, min(T, k * K + K)):
            hs.append(step(hs[-1], t))
        for t in reversed(range(k * K, min(T, k * K + K))):
            now, was = hs[t - k * K + 1], hs[t - k * K]
            g = g + C[:, t, :, :, None] * dy[:, t, :, None, :]
            dC[:, t] = (now @ dy[:, t, :, :, None])[..., 0]
            dB[:, t] = (g @ u[:, t, :, :, None])[..., 0]
            du[:, t] = (B[:, t, :, None, :] @ g)[:, :, 0]
            g = g * a[:, t, :, None, None]
            da[:, t] = (g * was).sum((-1, -2))
    ddt = da * d["A"] + (du * x).sum(-1)
    dx = du * dt[..., None] + d["D"][:, None] * dy
    shared = (c["G"], c["H"] // c["G"])
    back = [_one_behind_the_other(c, v) for v in
            (dx, ddt, dB.unflatten(2, shared).sum(3), dC.unflatten(2, shared).sum(3))]
    draw_dt = back[1] * torch.sigmoid(raw)
    return (back[0], draw_dt, (da * dt).sum((0, 1)), back[2], back[3],
            (d["dy"] * d["x"]).sum((0, 1, 3)), draw_dt.sum((0, 1)), g)


def _exact_conv(c, d):
    y = torch.empty_like(d["x"])
    last = d["x"].new_zeros((c["n_seq"], c["W"] - 1, c["C"]))
    for i, (b, lo, hi) in enumerate(_ranges(c)):
        h = last[i] if d["state_in"] is None else d["state_in"][i]
        h = torch.cat([h, d["x"][b, lo:hi]])
        if hi > lo:
            y[b, lo:hi] = torch.einsum("tcw,cw->tc", h.unfold(0, c["W"], 1), d["weight"])
        last[i] = h[hi - lo:]
    y = y + d["bias"]
    return y * torch.sigmoid(y), last


def _exact_conv_backward(c, d):
    W = c["W"]
    dx = torch.zeros_like(d["x"])
    dw = torch.zeros_like(d["weight"])
    db = torch.zeros_like(d["bias"])
    ds = d["x"].new_zeros((c["n_seq"], W - 1, c["C"]))
    for i, (b, lo, hi) in enumerate(_ranges(c)):
        n = hi - lo
        h = torch.cat([ds[i] if d["state_in"] is None else d["state_in"][i], d["x"][b, lo:hi]])
        dh = torch.zeros_like(h)
        if d["dstate_out"] is not None:
            dh[n:] += d["dstate_out"][i]
        if n:
            pre = torch.einsum("tcw,cw->tc", h.unfold(0, W, 1), d["weight"]) + d["bias"]
            sig = torch.sigmoid(pre)
            dp = d["dy"][b, lo:hi] * sig * (1 + pre * (1 - sig))
            dw += torch.einsum("tcw,tc->cw", h.unfold(0, W, 1), dp)
            db += dp.sum(0)
            for j in range(W):
                dh[j: j + n] += dp * d["weight"][:, j]
        ds[i] = dh[: W - 1]
        dx[b, lo:hi] = dh[W - 1:]
    return dx, dw, db, ds


def _e4m3(v):
    """Nearest E4M3 value, ties to the even one, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=-5) - 4)
    return torch.clamp(torch.round(v / step) * step, -448, 448)


def _exact_norm(c, s, d):
    x, res = d["x"], None
    if d["residual"] is not None:
        res = (x + d["residual"]).to(DTYPE[c["dtype"]]).double()   # the stream as it is kept
        x = res
    y = x / torch.sqrt((x ** 2).mean(1, keepdim=True) + EPS) * d["weight"]
    if d["gate"] is not None:
        y = y * d["gate"] * torch.sigmoid(d["gate"])
    out = (y,)
    if c["out"] == "fp8_row":
        scale = y.abs().amax(1) / 448
        out = (_e4m3(y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]), scale)
    return out if res is None else out + (res,)


def _exact_norm_backward(d):
    x, w, dy = d["x"], d["weight"], d["dy"]
    v = (x ** 2).mean(1, keepdim=True) + EPS
    dgate = None
    if d["gate"] is not None:
        sig = torch.sigmoid(d["gate"])
        dgate = dy * (x / v.sqrt() * w) * (sig + d["gate"] * sig * (1 - sig))
        dy = dy * d["gate"] * sig
    dw = (dy * x / v.sqrt()).sum(0)
    dx = dy * w / v.sqrt() - x * (dy * w * x).mean(1, keepdim=True) / v ** 1.5
    if d["dresidual"] is not None:
        dx = dx + d["dresidual"]
    return (dx, dw) if dgate is None else (dx, dw, dgate)
