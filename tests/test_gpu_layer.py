"""The operators run one behind the other, as a recurrent layer uses them:
residual and norm in 8 bits, projection, convolution, scan (or the gated delta
rule), gated norm.  Every stage is compared with the 64-bit reference on the
inputs that it was given, so that each bound is the stage's own."""

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
D, H, P, G, N, W = 96, 2, 64, 1, 64, 4
XBC = H * P + 2 * G * N


class Layer:
    def __init__(self, dtype, seed=1):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).cuda()
        self.dtype = dtype
        self.w_in = r(D, k=0.1) + 1
        self.proj = r(D, H * P + XBC + H, k=D ** -0.5).to(dtype)     # z, x|B|C, dt
        self.conv_w, self.conv_b = r(XBC, W, k=0.5), r(XBC, k=0.1)
        self.A = -(torch.rand(H, generator=g) * 3 + 1).cuda()
        self.D, self.dt_bias = r(H), r(H) - 2
        self.w_out = r(P, k=0.1) + 1

    def split(self, h):
        p = h @ self.proj
        return p[..., :H * P], p[..., H * P:H * P + XBC], p[..., H * P + XBC:]

    def xbc(self, c):
        return (c[..., :H * P].unflatten(-1, (H, P)),
                c[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
                c[..., H * P + G * N:].unflatten(-1, (G, N)))


def prompt(lib, L, x, res, cu=None, conv_state=None, scan_state=None):
    q, s = lib.gdn_norm(x, L.w_in, residual=res, qdq="fp8_row")
    z, xbc, dt = L.split(q.dequantize().to(L.dtype))
    c, cs = lib.gdn_conv_prefill(xbc, L.conv_w, L.conv_b, conv_state, cu)
    u, B, C = L.xbc(c)
    y, ss = lib.gdn_scan_prefill(u, dt, L.A, B, C, D=L.D, dt_bias=L.dt_bias, state_in=scan_state,
                                 cu_seqlens=cu)
    o, _ = lib.gdn_norm(y, L.w_out, gate=z.unflatten(-1, (H, P)))
    return dict(q=q, s=s, z=z, xbc=xbc, dt=dt, c=c, cs=cs, u=u, B=B, C=C, y=y, ss=ss, o=o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [None, (5, 0, 66, 1, 130)])
def test_prompt_stage_by_stage(cuda_lib, lens, dtype):
    L = Layer(dtype)
    g = torch.Generator().manual_seed(2)
    cu, lead = None, (2, 70)
    if lens:
        cu, lead = [0], (1, sum(lens))
        for n in lens:
            cu.append(cu[-1] + n)
    x, res = (torch.randn(*lead, D, generator=g).to(dtype).cuda() for _ in range(2))
    n = 2 if cu is None else len(lens)
    cs0 = torch.randn(n, W - 1, XBC, generator=g).to(dtype).cuda()
    ss0 = torch.randn(n, H, N, P, generator=g).cuda()
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = prompt(cuda_lib, L, x, res, cud, cs0, ss0)
    cuda_lib.check_last_error()
    y, s = ref.norm(x, L.w_in, res, dtype=dtype)
    assert torch.equal(r["s"].double().cpu(), s)
    scale = r["q"].scales.double().cpu()[..., None]
    val = r["q"].codes.double().cpu() * scale
    assert ((val - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10)
            * (1 + 1e-5) + y.abs() * 1e-5).all()
    want = ref.conv(r["xbc"], L.conv_w, L.conv_b, cs0, cu)
    mag = ref.conv(r["xbc"], L.conv_w, L.conv_b, cs0, cu, mag=True)
    ref.within(r["c"], want[0], mag[0], 45, "conv")
    assert torch.equal(r["cs"].double().cpu(), want[1])
    args = (r["u"], r["dt"], L.A, r["B"], r["C"], L.D, L.dt_bias, ss0, cu)
    want, mag = ref.scan(*args), ref.scan(*args, mag=True)
    k = 3 * max(lens or (70,)) + N + P + 64
    ref.within(r["y"], want[0], mag[0], k, "scan", 2.0 ** -15 if dtype == BF16 else 0.0)
    ref.within(r["ss"], want[1], mag[1], k, "state")
    want, _ = ref.norm(r["y"], L.w_out, gate=r["z"].unflatten(-1, (H, P)))
    ref.within(r["o"], want, want.abs(), 90, "out")


def test_tokens_after_a_prompt(cuda_lib):
    """A prompt and then single tokens: the convolution's state and outputs
    are the whole sequence's bit for bit, the scan's within the sum of the two
    forms' bounds, also when the token step is a replayed graph."""
    L = Layer(BF16)
    g = torch.Generator().manual_seed(3)
    T, cut, n = 90, 80, 3
    x, res = (torch.randn(n, T, D, generator=g).to(BF16).cuda() for _ in range(2))
    whole = prompt(cuda_lib, L, x, res)
    head = prompt(cuda_lib, L, x[:, :cut].contiguous(), res[:, :cut].contiguous())
    cs, ss = head["cs"], head["ss"]
    xbc, dt = torch.empty_like(whole["xbc"][:, 0]), torch.empty_like(whole["dt"][:, 0])

    def token():
        c = cuda_lib.gdn_conv_decode(xbc, L.conv_w, L.conv_b, cs)
        u, B, C = L.xbc(c)
        return c, cuda_lib.gdn_scan_decode(u, dt, L.A, B, C, ss, D=L.D, dt_bias=L.dt_bias)

    keep = cs.clone(), ss.clone()
    xbc.copy_(whole["xbc"][:, cut])
    dt.copy_(whole["dt"][:, cut])
    token()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    cs.copy_(keep[0])
    ss.copy_(keep[1])
    args = (whole["u"], whole["dt"], L.A, whole["B"], whole["C"], L.D, L.dt_bias, None, None)
    want, mag = ref.scan(*args), ref.scan(*args, mag=True)
    k = 3 * T + N + P + 64
    for t in range(cut, T):
        xbc.copy_(whole["xbc"][:, t])
        dt.copy_(whole["dt"][:, t])
        graph.replay()
        assert torch.equal(out[0], whole["c"][:, t])
        ref.within(out[1], want[0][:, t], mag[0][:, t], k, "token", 2.0 ** -15)
    assert torch.equal(cs, whole["cs"])
    ref.within(ss, want[1], mag[1], k, "state")


def test_gradient_chain(cuda_lib):
    """The layer's gradient from the entry points' gradients, fp32: its
    product with a direction equals the difference quotient of the 64-bit
    reference chain along that direction.  fp32: a few hundred roundings a
    stage, 3 stages, against the sum of the products' magnitudes: 1e-4; the
    quotient's own error is 1e-6 of the third derivative and below."""
    L = Layer(F32)
    g = torch.Generator().manual_seed(4)
    n, T = 2, 70
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    xbc, dt, z = rnd(n, T, XBC), rnd(n, T, H), rnd(n, T, H, P)
    do = rnd(n, T, H, P)
    c, _ = cuda_lib.gdn_conv_prefill(xbc, L.conv_w, L.conv_b)
    u, B, C = L.xbc(c)
    y, _ = cuda_lib.gdn_scan_prefill(u, dt, L.A, B, C, D=L.D, dt_bias=L.dt_bias)
    dy, dw_out, dz = cuda_lib.gdn_norm_backward(y, L.w_out, do, gate=z)
    du, ddt, dA, dB, dC, dD, db, _ = cuda_lib.gdn_scan_backward(
        u, dt, L.A, B, C, dy, D=L.D, dt_bias=L.dt_bias)
    dc = torch.cat([du.flatten(2), dB.flatten(2), dC.flatten(2)], -1)
    dxbc, dcw, dcb, _ = cuda_lib.gdn_conv_backward(xbc, L.conv_w, dc, L.conv_b)
    params = [xbc, dt, z, L.conv_w, L.conv_b, L.A, L.D, L.dt_bias, L.w_out]
    grads = [dxbc, ddt, dz, dcw, dcb, dA, dD, db, dw_out]

    def loss(p):
        xbc, dt, z, cw, cb, A, Dk, b, w = p
        c, _ = ref.conv(xbc, cw, cb, None, None)
        u, B, C = L.xbc(c)
        y, _ = ref.scan(u, dt, A, B, C, Dk, b, None, None)
        o, _ = ref.norm(y, w, gate=z)
        return float((o * do.double().cpu()).sum())

    base = [p.double().cpu() for p in params]
    for i in range(len(params)):
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        e = 1e-4
        hi = loss([p + e * d if j == i else p for j, p in enumerate(base)])
        lo = loss([p - e * d if j == i else p for j, p in enumerate(base)])
        prod = grads[i].double().cpu() * d
        assert abs(float(prod.sum()) - (hi - lo) / (2 * e)) <= 1e-4 * float(prod.abs().sum()), i


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_around_the_delta_rule(cuda_lib, dtype):
    """Convolution in front of gdn_prefill's q, k and v, the gated norm of
    every head behind it."""
    g = torch.Generator().manual_seed(5)
    n, T, h, d = 2, 70, 2, 128
    qkv = torch.randn(n, T, 3 * h * d, generator=g).to(dtype).cuda()
    z = torch.randn(n, T, h * d + 8, generator=g).to(dtype).cuda()[..., 8:].unflatten(-1, (h, d))
    w, b = (torch.randn(3 * h * d, W, generator=g) * 0.5).cuda(), None
    c, _ = cuda_lib.gdn_conv_prefill(qkv, w, b)
    q, k, v = (t.unflatten(-1, (h, d)).contiguous() for t in c.chunk(3, -1))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(dtype) for t in (q, k))
    gate = -torch.rand(n, T, h, generator=g).cuda() * 0.1
    beta = torch.rand(n, T, h, generator=g).cuda()
    o, _ = cuda_lib.gdn_prefill(q, k, v, gate, beta)
    out, _ = cuda_lib.gdn_norm(o, torch.ones(d, device="cuda"), gate=z)
    cuda_lib.check_last_error()
    want, _ = ref.norm(o, torch.ones(d), gate=z)
    ref.within(out, want, want.abs(), 90, "out")
    codes, _ = cuda_lib.gdn_norm(o, torch.ones(d, device="cuda"), gate=z, qdq="int8_g32")
    sc = codes.scales.double().cpu().repeat_interleave(32, -1)
    val = codes.dequantize().double().cpu()
    assert ((val - want).abs() <= sc * 0.5 * (1 + 1e-5) + want.abs() * 1e-5).all()


def test_calls_at_once_on_two_streams(cuda_lib):
    """Each call has its own workspace: two gradients and two prompts in
    flight on two streams give the same bits as one behind the other."""
    L = Layer(BF16)
    g = torch.Generator().manual_seed(6)
    sets = []
    for _ in range(2):
        x = torch.randn(1, 700, H, P, generator=g).to(BF16).cuda()
        dt = torch.randn(1, 700, H, generator=g).to(BF16).cuda()
        B, C = (torch.randn(1, 700, G, N, generator=g).to(BF16).cuda() for _ in range(2))
        dy = torch.randn(1, 700, H, P, generator=g).to(BF16).cuda()
        sets.append((x, dt, L.A, B, C, dy))

    def run(s):
        return cuda_lib.gdn_scan_prefill(*s[:5], D=L.D, dt_bias=L.dt_bias) + \
            cuda_lib.gdn_scan_backward(*s, D=L.D, dt_bias=L.dt_bias)

    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(run(s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_given_stream(cuda_lib):
    """``stream=`` and the current stream give the same bits, with outputs and
    workspaces that belong to the stream that writes them."""
    L = Layer(BF16)
    g = torch.Generator().manual_seed(7)
    x, res = (torch.randn(1, 700, D, generator=g).to(BF16).cuda() for _ in range(2))
    r = prompt(cuda_lib, L, x, res)
    dy = torch.randn(1, 700, H, P, generator=g).to(BF16).cuda()
    dc = torch.randn(1, 700, XBC, generator=g).to(BF16).cuda()
    scan = (r["u"], r["dt"], L.A, r["B"], r["C"])

    def run(**kw):
        return (cuda_lib.gdn_scan_prefill(*scan, D=L.D, **kw)
                + cuda_lib.gdn_scan_backward(*scan, dy, D=L.D, **kw)
                + cuda_lib.gdn_conv_prefill(r["xbc"], L.conv_w, L.conv_b, **kw)
                + cuda_lib.gdn_conv_backward(r["xbc"], L.conv_w, dc, L.conv_b, **kw)
                + cuda_lib.gdn_norm(x, L.w_in, residual=res, **kw)
                + cuda_lib.gdn_norm_backward(x, L.w_in, res, **kw)[:2])

    want = run()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = run(stream=side)
        junk = [torch.zeros(1 << 20, device="cuda") for _ in range(8)]   # the current stream's own
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del junk


def _far_apart(rows, width, stride, dtype, gen):
    """[1, rows, width] whose tokens lie `stride` elements apart: the last
    one's offset passes 2^31 elements (and 32 bits of bytes)."""
    base = torch.empty((rows - 1) * stride + width, dtype=dtype, device="cuda")
    x = base.as_strided((1, rows, width), (rows * stride, stride, 1))
    x.copy_(torch.randn(1, rows, width, generator=gen))
    return x


def test_offsets_past_32_bits(cuda_lib):
    g = torch.Generator().manual_seed(8)
    T, stride = 70, 1 << 25
    x = _far_apart(T, 256, stride, BF16, g)
    assert (T - 1) * stride > 1 << 31
    near = x.contiguous()
    w = torch.randn(256, W, generator=g).cuda()
    dy = torch.randn(1, T, 256, generator=g).to(BF16).cuda()
    for far, close in zip(cuda_lib.gdn_conv_prefill(x, w) + cuda_lib.gdn_conv_backward(x, w, dy),
                          cuda_lib.gdn_conv_prefill(near, w)
                          + cuda_lib.gdn_conv_backward(near, w, dy)):
        assert torch.equal(far, close)
    one = torch.ones(256, device="cuda")
    assert torch.equal(cuda_lib.gdn_norm(x, one)[0], cuda_lib.gdn_norm(near, one)[0])
    for far, close in zip(cuda_lib.gdn_norm_backward(x, one, dy)[:2],
                          cuda_lib.gdn_norm_backward(near, one, dy)[:2]):
        assert torch.equal(far, close)
    A = -torch.rand(2, generator=g).cuda() - 0.5
    dt = torch.randn(1, T, 2, generator=g).to(BF16).cuda()

    def scan(t, d):
        a = (t[..., :128].unflatten(-1, (2, 64)), d, A, t[..., 128:192].unflatten(-1, (1, 64)),
             t[..., 192:].unflatten(-1, (1, 64)))
        return cuda_lib.gdn_scan_prefill(*a) + cuda_lib.gdn_scan_backward(
            *a, dy[..., :128].unflatten(-1, (2, 64)).contiguous())

    for far, close in zip(scan(x, dt), scan(near, dt)):
        assert torch.equal(far, close)


def test_packed_call_replayed_with_other_lengths(cuda_lib):
    """A captured packed call reads cu_seqlens when it is replayed."""
    L = Layer(BF16)
    g = torch.Generator().manual_seed(9)
    T = 300
    xbc = torch.randn(1, T, XBC, generator=g).to(BF16).cuda()
    dt = torch.randn(1, T, H, generator=g).to(BF16).cuda()
    cus = [torch.tensor(c, dtype=torch.int32, device="cuda")
           for c in ([0, 100, 200, 300], [0, 0, 299, 300], [0, 300, 300, 300])]

    def run(cu):
        c, cs = cuda_lib.gdn_conv_prefill(xbc, L.conv_w, L.conv_b, None, cu)
        u, B, C = L.xbc(c)
        return (c, cs) + cuda_lib.gdn_scan_prefill(u, dt, L.A, B, C, D=L.D, cu_seqlens=cu)

    want = [run(cu) for cu in cus]
    cu = cus[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(cu)
    for c, w in zip(cus, want):
        cu.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    cuda_lib.check_last_error()
