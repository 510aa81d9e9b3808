"""ecc_gated_linear and ecc_gated_linear_grad against a plain 64-bit
computation.

Tolerances, those of the linear layer's tests: u is half a unit in the last
place of a stored type, `tiny` half its smallest step; a sum of K products in
float32, each addition truncated, is off by (K + 8) 2^-23 sum |x||w|; the
activations have slopes of at most 1.13 and are computed to a relative 2^-20
and an absolute 2^-22 of their argument.  A product of two such values is off
by each one's error times the other's magnitude (with its error) and 2^-24 of
itself.  In the backward pass tg = dy u act'(g) and tu = dy act(g), each times
its share of the larger scale, are rounded to the operands' type.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
U = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11, E4M3: 2.0**-4}
TINY = {F32: 2.0**-149, BF16: 2.0**-133, F16: 2.0**-25, E4M3: 2.0**-10}
F = torch.nn.functional
ACTS = {"none": lambda a: a, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
        "gelu_tanh": lambda a: F.gelu(a, approximate="tanh")}


def rows_of(gen, rows, cols, dtype, pad=0, off=0, std=1.0):
    base = torch.randn(rows * (cols + pad) + off, generator=gen, device="cuda") * std
    return base.to(dtype)[off:].view(rows, cols + pad)[:, :cols]


def projection(x, w, bias, scale):
    a = scale * (x.double() @ w.double().T)
    e = abs(scale) * (x.shape[1] + 8) * 2.0**-23 * (x.double().abs() @ w.double().abs().T)
    if bias is not None:
        a = a + bias.double()
    return a, e + 2.0**-22 * a.abs()


def check(x, wg, wu, bg=None, bu=None, act="silu", scale=1.0, up_scale=None, out_dtype=None, out_scale=1.0, pre_dtype=None,
          pre_pad=0, **kw):
    M, N = x.shape[0], wg.shape[0]
    pre = [None, None]
    if pre_dtype is not None:
        pre = [torch.full((M, N + pre_pad * i), float("nan"), dtype=pre_dtype, device="cuda")[:, :N] for i in range(2)]
    y, st = ecc.ecc_gated_linear(x, wg, wu, bg, bu, act=act, scale=scale, up_scale=up_scale, out_dtype=out_dtype,
                                 out_scale=out_scale, pre_gate=pre[0], pre_up=pre[1], **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == ecc.OK
    g, eg = projection(x, wg, bg, scale)
    u, eu = projection(x, wu, bu, scale if up_scale is None else up_scale)
    h = ACTS[act](g)
    eh = eg if act == "none" else 1.13 * eg + 2.0**-20 * h.abs() + 2.0**-22 * g.abs()
    ref = h * u * out_scale
    e = (eh * (u.abs() + eu) + h.abs() * eu + 2.0**-23 * (h * u).abs()) * abs(out_scale)
    if y.dtype == E4M3:
        ref = ref.clamp(-448, 448)
    assert bool(((y.double() - ref).abs() <= 1.01 * U[y.dtype] * ref.abs() + TINY[y.dtype] + e).all())
    for p, a, ea in ((pre[0], g, eg), (pre[1], u, eu)):
        if p is not None:
            assert bool(((p.double() - a).abs() <= 1.01 * U[pre_dtype] * a.abs() + TINY[pre_dtype] + ea).all())
    return y


SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (1, 1000, 512), (2, 64, 4096), (5, 4096, 64), (16, 2048, 2048), (17, 129, 65),
          (64, 512, 1000), (65, 1000, 129), (128, 128, 64), (128, 256, 8192), (129, 257, 192), (200, 333, 1001),
          (256, 256, 256), (511, 768, 520), (1000, 1024, 96), (2048, 640, 320), (33, 16384, 72), (6, 24, 16384), (8, 63, 640),
          (300, 65, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_shapes(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 3 * N + 7 * K)
    s = 1 / math.sqrt(K)
    for pad, off in ((0, 0), (16, 0), (5, 3)):
        x = rows_of(gen, M, K, dtype, pad, off)
        wg, wu = rows_of(gen, N, K, dtype, pad), rows_of(gen, N, K, dtype, 2 * pad)
        check(x, wg, wu, scale=s)
    for pads in ((3, 0, 0), (0, 3, 0), (0, 0, 3)):          # one operand's rows on any boundary
        check(*(rows_of(gen, r, K, dtype, p) for r, p in zip((M, N, N), pads)), scale=s, up_scale=-s)
    p_dtype = BF16 if dtype == E4M3 else dtype
    bg, bu = rows_of(gen, 2, N, p_dtype)
    check(x, wg, wu, bg, bu, "gelu", s, pre_dtype=p_dtype, pre_pad=3)
    check(x, wg, wu, bg.float(), None, "gelu_tanh", s, 2 * s, out_dtype=E4M3, out_scale=8.0)
    check(x, wg, wu, None, bu.float(), "relu", s, out_dtype=F32, pre_dtype=F32)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out_dtype", [BF16, F16, F32, E4M3])
@pytest.mark.parametrize("M", [1, 5, 300])
def test_gated_epilogues(M, act, out_dtype):
    gen = torch.Generator("cuda").manual_seed(2)
    x, wg, wu = rows_of(gen, M, 256, BF16), rows_of(gen, 424, 256, BF16, std=0.25), rows_of(gen, 424, 256, BF16, std=0.1)
    bg, bu = rows_of(gen, 2, 424, F32)
    check(x, wg, wu, bg, bu, act, 1.0, 0.5, out_dtype, 3.0 if out_dtype == E4M3 else 1.0, pre_dtype=BF16)
    check(x, wg, wu, None, None, act, -0.5, None, out_dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 15), (7, 131), (130, 2049), (8197, 255), (1024, 2048), (1025, 4095), (70001, 17)])
def test_gated_few_rows(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M * 31 + N + K)
    outs = [BF16, F16, F32, E4M3]
    for i, (pad, off) in enumerate(((0, 0), (8, 0), (5, 3), (1, 1))):
        x = rows_of(gen, M, K, dtype, pad, off)
        wg, wu = rows_of(gen, N, K, dtype, 2 * pad, off, std=K**-0.5), rows_of(gen, N, K, dtype, pad, std=K**-0.5)
        bg, bu = rows_of(gen, 2, N, F32)
        args = dict(act=list(ACTS)[(M + i) % 5], scale=0.75, up_scale=1.5, out_dtype=outs[(M + i) % 4],
                    pre_dtype=F16 if i > 1 else None)
        first = check(x, wg, wu, bg if i else None, bu if i % 2 else None, **args)
        again = check(x, wg, wu, bg if i else None, bu if i % 2 else None, **args)
        assert torch.equal(first.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("M", [20, 700])
def test_gated_weights_wherever_they_lie(M, dtype):
    """Gates above ups and below them, rows of one matrix in turns, the same matrix twice, other strides, far apart."""
    gen = torch.Generator("cuda").manual_seed(17)
    N, K = 160, 256
    x, both = rows_of(gen, M, K, dtype), rows_of(gen, 2 * N, K, dtype, std=0.1)
    far = torch.empty(3 << 30, dtype=torch.uint8, device="cuda")[-N * K * both.element_size():].view(dtype).view(N, K)
    far.copy_(both[N:])
    a, b = both[:N], both[N:]
    bias = rows_of(gen, 2, N, F32)
    for wg, wu in ((a, b), (b, a), (both[::2], both[1::2]), (both[1::2], both[::2]), (a, a), (a, both[::2]), (a, far), (far, a),
                   (both[1:N + 1], both[:N])):
        check(x, wg, wu, *bias, pre_dtype=BF16, up_scale=0.5)


def test_gated_large_offsets_and_rows_beside_the_output():
    gen = torch.Generator("cuda").manual_seed(3)
    buf = torch.zeros((1 << 32) + 4096, dtype=BF16, device="cuda")       # rows 2^31 elements apart
    far = buf.as_strided((3, 512), ((1 << 31) + 8, 1))
    far.copy_(torch.randn(3, 512, device="cuda"))
    for M in (1, 3, 150):
        near = rows_of(gen, M, 512, BF16)
        check(far, near, near, scale=0.1)
        check(near, far, rows_of(gen, 3, 512, BF16), scale=0.1)
        check(near, rows_of(gen, 3, 512, BF16), far, scale=0.1)
    del buf, far
    for M, N in ((3, 100), (200, 131)):
        x, wg, wu = rows_of(gen, M, 128, BF16), rows_of(gen, N, 128, BF16), rows_of(gen, N, 128, BF16)
        whole = torch.full((M + 2, N + 9), 7.0, dtype=BF16, device="cuda")
        out = whole[1:M + 1, 4:N + 4]
        ecc.ecc_gated_linear(x, wg, wu, scale=0.1, out=out)
        assert torch.equal(out, check(x, wg, wu, scale=0.1))
        out.fill_(7)
        assert bool((whole == 7).all())


def test_gated_zero_lengths():
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    for M, N in ((0, 8), (8, 0), (0, 0)):
        y, st = ecc.ecc_gated_linear(e(M, 16), e(N, 16), e(N, 16))
        assert y.shape == (M, N) and int(st.item()) == 0
    bg, bu = torch.randn(2, 40, device="cuda")
    for M in (3, 200):
        y, st = ecc.ecc_gated_linear(e(M, 0), e(40, 0), e(40, 0), bg, bu, act="relu", out_dtype=F32)
        assert torch.equal(y, (bg.relu() * bu).expand(M, 40)) and int(st.item()) == 0
    r = ecc.ecc_gated_linear_grad(e(0, 24), e(0, 16), e(24, 16), e(24, 16), e(0, 24), e(0, 24))
    assert r[0].shape == (0, 16) and not any(t.any() for t in r[1:])
    r = ecc.ecc_gated_linear_grad(e(5, 0), e(5, 16), e(0, 16), e(0, 16), e(5, 0), e(5, 0))
    assert not r[0].any() and r[1].shape == r[2].shape == (0, 16) and int(r[5].item()) == 0


def test_gated_non_finite_values_stay_in_place():
    gen = torch.Generator("cuda").manual_seed(4)
    for M, N, K in ((1, 300, 200), (4, 300, 3000), (300, 400, 264)):
        x, wg, wu = rows_of(gen, M, K, BF16), rows_of(gen, N, K, BF16), rows_of(gen, N, K, BF16)
        clean = check(x, wg, wu, scale=0.05)
        for w in (wg, wu):
            keep = w[5].clone()
            w[5, 7] = float("nan")
            y = ecc.ecc_gated_linear(x, wg, wu, scale=0.05)[0]
            assert bool(y[:, 5].isnan().all()) and torch.equal(y[:, :5], clean[:, :5]) and torch.equal(y[:, 6:], clean[:, 6:])
            w[5] = keep
        x[0, 3] = float("inf")
        y = ecc.ecc_gated_linear(x, wg, wu, scale=0.05)[0]
        assert not bool(y[0].isfinite().all()) and torch.equal(y[1:], clean[1:])


def check_grad(dy, x, wg, wu, g, u, act="silu", scale=1.0, up_scale=None, **kw):
    r = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, act=act, scale=scale, up_scale=up_scale, **kw)
    torch.cuda.synchronize()
    assert int(r[5].item()) == ecc.OK
    (M, N), up = dy.shape, scale if up_scale is None else up_scale
    a, d, ud = g.double().requires_grad_(), dy.double(), u.double()
    h = ACTS[act](a)
    slope, = torch.autograd.grad(h.sum(), a)
    a, h = a.detach(), h.detach()
    near = (1 + a.abs()) * (a.abs() < 20)
    es, eh = 2.0**-19 * slope.abs() + 2.0**-20 * near, 2.0**-19 * h.abs() + 2.0**-20 * near
    if act == "none":
        es = eh = torch.zeros_like(a)
    tg, tu = d * ud * slope, d * h
    eg, eu = (d * ud).abs() * es + 2.0**-22 * tg.abs(), d.abs() * eh + 2.0**-22 * tu.abs()
    big = max(abs(scale), abs(up))
    rg = eg + U[dy.dtype] * tg.abs() + (TINY[dy.dtype] * big / abs(scale) if scale else 0)
    ru = eu + U[dy.dtype] * tu.abs() + (TINY[dy.dtype] * big / abs(up) if up else 0)

    def near_to(got, ref, e):
        assert bool(((got.double() - ref).abs() <= 1.01 * U[got.dtype] * ref.abs() + TINY[got.dtype] + 1.01 * e).all())

    gd, wd = wg.double(), wu.double()
    if r[0] is not None:
        sums = abs(scale) * (tg.abs() @ gd.abs()) + abs(up) * (tu.abs() @ wd.abs())
        near_to(r[0], scale * (tg @ gd) + up * (tu @ wd),
                abs(scale) * (rg @ gd.abs()) + abs(up) * (ru @ wd.abs()) + (2 * N + 136) * 2.0**-23 * sums)
    xd = x.double()
    for got, t, e, s in ((r[1], tg, rg, scale), (r[2], tu, ru, up)):
        if got is not None:
            near_to(got, s * (t.T @ xd), abs(s) * (e.T @ xd.abs() + (M + 8) * 2.0**-23 * (t.T.abs() @ xd.abs())))
    for got, t, e in ((r[3], tg, eg), (r[4], tu, eu)):
        if got is not None:
            assert bool(((got.double() - t.sum(0)).abs() <= e.sum(0) + (M + 16) * 2.0**-24 * t.abs().sum(0)).all())
    return r


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_grad_shapes(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 5 * N + 11 * K)
    s = 1 / math.sqrt(N)
    for pad, off, act in ((0, 0, "silu"), (16, 0, "none"), (5, 3, "gelu"), (3, 0, "gelu_tanh")):
        x = rows_of(gen, M, K, dtype, pad, off)
        wg, wu = rows_of(gen, N, K, dtype, pad, std=s), rows_of(gen, N, K, dtype, 2 * pad, std=s)
        dy, g, u = rows_of(gen, M, N, dtype, pad), rows_of(gen, M, N, dtype, 2 * pad), rows_of(gen, M, N, dtype)
        check_grad(dy, x, wg, wu, g, u, act)
    check_grad(dy, x, wg, wu, g.float(), u.float(), "relu", 0.5, -0.125, dw_dtype=F32)


@pytest.mark.parametrize("act", list(ACTS))
def test_gated_grad_wanted_outputs_and_repeats(act):
    gen = torch.Generator("cuda").manual_seed(12)
    x, wg, wu = rows_of(gen, 130, 200, BF16), rows_of(gen, 300, 200, BF16, std=0.05), rows_of(gen, 300, 200, BF16, std=0.05)
    dy, g, u = rows_of(gen, 130, 300, BF16), rows_of(gen, 130, 300, BF16, std=3.0), rows_of(gen, 130, 300, BF16)
    for scales in ((-2.0, None), (1.0, 0.0), (0.0, 3.0), (0.0, 0.0)):
        first = check_grad(dy, x, wg, wu, g, u, act, *scales)
        for want in (("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ()):
            got = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, act=act, scale=scales[0], up_scale=scales[1], want=want)
            for name, t, f in zip(("dx", "dw", "dw", "dbias", "dbias"), got, first):
                assert (t is None) if name not in want else torch.equal(t, f)


def test_gated_grad_into_given_tensors():
    gen = torch.Generator("cuda").manual_seed(14)
    for M, N, K in ((40, 100, 72), (600, 257, 320)):
        x, wg, wu = rows_of(gen, M, K, BF16), rows_of(gen, N, K, BF16), rows_of(gen, N, K, BF16)
        dy, g, u = rows_of(gen, M, N, BF16), rows_of(gen, M, N, BF16), rows_of(gen, M, N, BF16)
        ref = check_grad(dy, x, wg, wu, g, u, scale=0.1, dw_dtype=F32)
        whole = [torch.full((r + 2, c + 9), 7.0, dtype=t, device="cuda") for r, c, t in ((M, K, BF16), (N, K, F32), (N, K, F32))]
        views = [w[1:-1, 4:-5] for w in whole]
        got = check_grad(dy, x, wg, wu, g, u, scale=0.1, dx=views[0], dw_gate=views[1], dw_up=views[2])
        assert all(torch.equal(a, b) for a, b in zip(got[:5], ref[:5]))
        for w, v in zip(whole, views):
            v.fill_(7)
            assert bool((w == 7).all())


def test_gated_grad_against_differences():
    gen = torch.Generator("cuda").manual_seed(13)
    x, wg, wu = rows_of(gen, 6, 24, BF16), rows_of(gen, 16, 24, BF16, std=0.3), rows_of(gen, 16, 24, BF16, std=0.3)
    bg, bu = rows_of(gen, 2, 16, F32)
    dy = rows_of(gen, 6, 16, BF16)
    for act in ("gelu", "gelu_tanh", "silu", "none"):
        g, u = torch.empty(2, 6, 16, dtype=F32, device="cuda")
        ecc.ecc_gated_linear(x, wg, wu, bg, bu, act=act, pre_gate=g, pre_up=u, scale=0.7, up_scale=0.4)
        grads = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, act=act, scale=0.7, up_scale=0.4, dw_dtype=F32)

        def loss(x, wg, wu, bg, bu):
            return float((ACTS[act](0.7 * x @ wg.T + bg) * (0.4 * x @ wu.T + bu) * dy.double()).sum())

        args = [t.double() for t in (x, wg, wu, bg, bu)]
        h = 1e-4
        for k in range(12):
            for at, grad in enumerate(grads[:5]):
                t = args[at]
                i = (k % t.shape[0], (5 * k) % t.shape[1]) if t.dim() == 2 else (k,)
                e = torch.zeros_like(t)
                e[i] = h
                up, down = list(args), list(args)
                up[at], down[at] = t + e, t - e
                diff = (loss(*up) - loss(*down)) / (2 * h)
                # t is rounded to bfloat16 (2^-8 of at most 32 terms, of 6 for the weights), dx too
                assert abs(diff - float(grad[i])) < 2.0**-8 * (abs(diff) + 8)


def test_gated_captured_on_another_stream_and_replayed():
    gen = torch.Generator("cuda").manual_seed(15)
    for M, N, K in ((1, 256, 512), (70, 200, 321), (400, 600, 512)):
        x, wg, wu = rows_of(gen, M, K, BF16), rows_of(gen, N, K, BF16), rows_of(gen, N, K, BF16)
        dy, g, u = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(3))
        dy.normal_()
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            y, s1 = ecc.ecc_gated_linear(x, wg, wu, scale=0.1, pre_gate=g, pre_up=u)
            r = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, scale=0.1)
        for _ in range(3):
            x.copy_(torch.randn(M, K, generator=gen, device="cuda"))
            graph.replay()
            ref = check(x, wg, wu, scale=0.1)
            want = check_grad(dy, x, wg, wu, g, u, scale=0.1)
            assert torch.equal(y, ref) and all(torch.equal(a, b) for a, b in zip(r, want))
        got = [ecc.ecc_gated_linear(x, wg, wu, scale=0.1, stream=stream) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(t, ref) and int(s.item()) == 0 for t, s in got)


def test_gated_bytes_go_to_the_coder():
    gen = torch.Generator("cuda").manual_seed(16)
    x, wg, wu = (rows_of(gen, r, 256, E4M3) for r in (128, 512, 512))
    y = check(x, wg, wu, act="gelu_tanh", scale=1 / 16, out_dtype=E4M3, out_scale=16.0)
    a, _ = ecc.ecc_gated_linear(x.view(torch.uint8), wg.view(torch.uint8), wu.view(torch.uint8), act="gelu_tanh", scale=1 / 16,
                                out_dtype=torch.uint8, out_scale=16.0)
    assert torch.equal(a, y.view(torch.uint8))
    count = ecc.e4m3_histogram(a.view(-1))
    cb = ecc.to_device(ecc.qlc_build_tables(count.cpu().numpy().view("uint64")))
    enc = ecc.ecc_encode(a.view(-1), cb)
    out, st = ecc.ecc_decode(enc, cb)
    assert int(st.item()) == 0 and torch.equal(out[:a.numel()], a.view(-1))


def test_gated_refusals():
    x, w = torch.randn(4, 64, device="cuda").to(BF16), torch.randn(32, 64, device="cuda").to(BF16)
    b, r = torch.randn(32, device="cuda"), torch.randn(4, 32, device="cuda")
    g = r.to(BF16)
    f, d = ecc.ecc_gated_linear, ecc.ecc_gated_linear_grad
    bad = [lambda: f(x.float(), w.float(), w.float()), lambda: f(x, w, w.half()), lambda: f(x, w.half(), w),
           lambda: f(x, w, w[:31]), lambda: f(x, w[:, :63], w[:, :63]), lambda: f(x, w.t(), w.t()), lambda: f(x, w[0], w[0]),
           lambda: f(x, w, None), lambda: f(x, w, w, act="tanh"), lambda: f(x, w, w, b[:31]), lambda: f(x, w, w, b, b.half()),
           lambda: f(x, w, w, b.double()), lambda: f(x, w, w, out_scale=2.0), lambda: f(x, w, w, scale=float("nan")),
           lambda: f(x, w, w, up_scale=float("inf")), lambda: f(x.cpu(), w, w), lambda: f(x, w, w.cpu()),
           lambda: f(x, w, w, out=r[:, :31]), lambda: f(x, w, w, out_dtype=torch.float64), lambda: f(x, w, w, pre_gate=r),
           lambda: f(x, w, w, pre_up=r), lambda: f(x, w, w, pre_gate=r, pre_up=g), lambda: f(x, w, w, pre_gate=r[:3], pre_up=r[:3]),
           lambda: f(x[:1].expand(4, 64), w, w), lambda: f(x, w, w, status=torch.zeros(1, device="cuda")),
           lambda: f(torch.randn(40, 65, device="cuda").to(BF16)[:, :64], torch.randn(999, 64, device="cuda").to(BF16),
                     torch.randn(999, 64, device="cuda").to(BF16), ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: d(g, x, w, w, None, g), lambda: d(g, x, w, w, g, None), lambda: d(g, x, w, w, g, r), lambda: d(r, x, w, w, g, g),
           lambda: d(g, x[:3], w, w, g, g), lambda: d(g, x, w[:31], w, g, g), lambda: d(g, x, w, w[:31], g, g),
           lambda: d(g, x, w, w, g, g, dw_dtype=F16), lambda: d(g, x, w, w, g, g, act="tanh"),
           lambda: d(g, x, w, w, g, g, dw_gate=torch.empty(32, 64, device="cuda"), dw_up=torch.empty(32, 64, dtype=BF16, device="cuda")),
           lambda: d(g, x, w, w, g, g, dx=torch.empty(4, 64, device="cuda")),
           lambda: d(g.to(E4M3), x.to(E4M3), w.to(E4M3), w.to(E4M3), g, g),
           lambda: d(g, x, w, w, g, g, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for call in bad:
        with pytest.raises(ecc.EccError) as e:
            call()
        assert e.value.code == ecc.ERR_ARG
