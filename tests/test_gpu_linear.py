"""ecc_linear and ecc_linear_grad against a plain 64-bit computation.

Tolerances.  u is half a unit in the last place of a stored type (2^-24
float32, 2^-8 bfloat16, 2^-11 float16, 2^-4 e4m3; `tiny` half its smallest
step).  A sum of K products in float32, in any order and with each addition
truncated, is off by at most (K + 8) 2^-23 sum |x||w|.  The activations have
slopes of at most 1.13 and are computed to a relative 2^-20 and an absolute
2^-22 of their argument's magnitude.  In the backward pass t = dy act'(pre) is
rounded to the operands' type: u |t| + tiny for each term.
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


def check(x, w, bias=None, residual=None, act="none", scale=1.0, out_dtype=None, out_scale=1.0, pre_dtype=None, **kw):
    M, N, K = x.shape[0], w.shape[0], x.shape[1]
    pre = None if pre_dtype is None else torch.full((M, N), float("nan"), dtype=pre_dtype, device="cuda")
    y, st = ecc.ecc_linear(x, w, bias, residual, act=act, scale=scale, out_dtype=out_dtype, out_scale=out_scale,
                           pre=pre, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == ecc.OK
    xd, wd = x.double(), w.double()
    a = scale * (xd @ wd.T)
    ea = abs(scale) * (K + 8) * 2.0**-23 * (xd.abs() @ wd.abs().T)
    if bias is not None:
        a = a + bias.double()
    ea = ea + 2.0**-22 * a.abs()
    ref = ACTS[act](a)
    e = ea if act == "none" else 1.13 * ea + 2.0**-20 * ref.abs() + 2.0**-22 * a.abs()
    if residual is not None:
        ref = ref + residual.double()
        e = e + 2.0**-23 * (ref.abs() + residual.double().abs())
    ref, e = ref * out_scale, e * out_scale
    if y.dtype == E4M3:
        ref = ref.clamp(-448, 448)
    err = (y.double() - ref).abs()
    assert bool((err <= 1.01 * U[y.dtype] * ref.abs() + TINY[y.dtype] + e).all())
    if pre is not None:
        assert bool(((pre.double() - a).abs() <= 1.01 * U[pre_dtype] * a.abs() + TINY[pre_dtype] + ea).all())
    return y


SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (1, 1000, 512), (2, 64, 4096), (8, 4096, 64), (16, 2048, 2048),
          (17, 129, 65), (64, 512, 1000), (65, 1000, 129), (128, 128, 64), (128, 256, 8192), (129, 257, 192),
          (200, 333, 1001), (256, 256, 256), (511, 768, 520), (1000, 1024, 96), (2048, 640, 320), (33, 16384, 72),
          (4, 24, 16384)]


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_shapes(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 3 * N + 7 * K)
    s = 1 / math.sqrt(K)
    for pad, off in ((0, 0), (16, 0), (5, 3)):
        x, w = rows_of(gen, M, K, dtype, pad, off), rows_of(gen, N, K, dtype, pad)
        check(x, w, scale=s)
    check(rows_of(gen, M, K, dtype), rows_of(gen, N, K, dtype, 3), scale=s)   # one operand's rows aligned
    p_dtype = BF16 if dtype == E4M3 else dtype
    bias, res = rows_of(gen, 1, N, p_dtype)[0], rows_of(gen, M, N, p_dtype, 5)
    check(x, w, bias, res, "gelu", s, pre_dtype=p_dtype)
    check(x, w, bias.float(), None, "silu", s, out_dtype=E4M3, out_scale=8.0)
    check(x, w, None, res.float(), "relu", s, out_dtype=F32, pre_dtype=F32)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out_dtype", [BF16, F16, F32, E4M3])
@pytest.mark.parametrize("M", [5, 300])
def test_linear_epilogues(M, act, out_dtype):
    gen = torch.Generator("cuda").manual_seed(2)
    x, w = rows_of(gen, M, 256, BF16), rows_of(gen, 424, 256, BF16, std=0.25)
    bias, res = rows_of(gen, 1, 424, F32)[0], rows_of(gen, M, 424, F16)
    check(x, w, bias, res, act, 1.0, out_dtype, 3.0 if out_dtype == E4M3 else 1.0, pre_dtype=BF16)
    check(x, w, None, None, act, -0.5, out_dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 15), (6, 131), (130, 2049), (8197, 513), (2048, 2048), (70001, 33), (1025, 4095),
                                 (4097, 4103), (130, 40001)])
def test_linear_few_rows(M, N, K, dtype):
    """Single tokens and the next few, on and off 16-byte boundaries, odd ends, every epilogue."""
    gen = torch.Generator("cuda").manual_seed(M * 31 + N + K)
    acts, outs = list(ACTS), [BF16, F16, F32, E4M3]
    for i, (pad, off) in enumerate(((0, 0), (8, 0), (5, 3), (1, 1))):
        x, w = rows_of(gen, M, K, dtype, pad, off), rows_of(gen, N, K, dtype, 2 * pad, off, std=K**-0.5)
        bias = torch.randn(N, generator=gen, device="cuda")
        res = torch.randn(M, N + pad, generator=gen, device="cuda").to(BF16)[:, :N]
        out = outs[(M + i) % 4]
        first = check(x, w, bias if i else None, res if i % 2 else None, act=acts[(M + i) % len(acts)], scale=0.75, out_dtype=out,
                      out_scale=2.0 if out == E4M3 else 1.0, pre_dtype=F16 if i > 1 else None)
        again = check(x, w, bias if i else None, res if i % 2 else None, act=acts[(M + i) % len(acts)], scale=0.75, out_dtype=out,
                      out_scale=2.0 if out == E4M3 else 1.0, pre_dtype=F16 if i > 1 else None)
        assert torch.equal(first.view(torch.uint8), again.view(torch.uint8))


def test_linear_long_sums_and_large_offsets():
    gen = torch.Generator("cuda").manual_seed(3)
    check(rows_of(gen, 130, 60000, BF16), rows_of(gen, 140, 60000, BF16), scale=0.01, out_dtype=F32)
    check(rows_of(gen, 2, 60000, BF16), rows_of(gen, 140, 60000, BF16), scale=0.01, out_dtype=F32)
    for M in (3, 150):
        buf = torch.zeros((1 << 32) + 4096, dtype=BF16, device="cuda")   # rows 2^31 elements and more apart
        x = buf.as_strided((3, 512), ((1 << 31) + 8, 1))
        x.copy_(torch.randn(3, 512, device="cuda"))
        w = rows_of(gen, M, 512, BF16)
        check(x, w, scale=0.1)
        check(w, x, scale=0.1)
    out = torch.zeros((1 << 32) + 4096, dtype=BF16, device="cuda").as_strided((3, 150), ((1 << 31) + 8, 1))
    y, st = ecc.ecc_linear(x, w, out=out)
    assert torch.equal(out, check(x, w))


def test_linear_zero_lengths():
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    for M, N in ((0, 8), (8, 0), (0, 0)):
        y, st = ecc.ecc_linear(e(M, 16), e(N, 16))
        assert y.shape == (M, N) and int(st.item()) == 0
    bias, res = torch.randn(40, device="cuda"), torch.randn(3, 40, device="cuda")
    y, st = ecc.ecc_linear(e(3, 0), e(40, 0), bias, res, act="relu", out_dtype=F32)
    assert torch.equal(y, bias.relu() + res) and int(st.item()) == 0
    dx, dw, db, st = ecc.ecc_linear_grad(e(0, 24), e(0, 16), e(24, 16))
    assert dx.shape == (0, 16) and not dw.any() and not db.any() and int(st.item()) == 0
    dx, dw, db, st = ecc.ecc_linear_grad(e(5, 0), e(5, 16), e(0, 16))
    assert not dx.any() and dw.shape == (0, 16) and int(st.item()) == 0


def test_linear_non_finite_values_stay_in_place():
    gen = torch.Generator("cuda").manual_seed(4)
    for M, N, K in ((4, 300, 200), (300, 400, 264)):
        x, w = rows_of(gen, M, K, BF16), rows_of(gen, N, K, BF16)
        clean = check(x, w)
        x[1, 3] = float("nan")
        y = ecc.ecc_linear(x, w)[0]
        assert bool(y[1].isnan().all()) and torch.equal(y[2:], clean[2:]) and torch.equal(y[0], clean[0])
        x[1, 3] = 0
        w[5, 7] = float("inf")
        y = ecc.ecc_linear(x, w, act="relu")[0]
        assert not bool(y[:, 5].isfinite().all()) and bool(y[:, :5].isfinite().all()) and bool(y[:, 6:].isfinite().all())
    x = torch.full((2, 64), 448.0, device="cuda").to(E4M3)
    y = ecc.ecc_linear(x, x, out_dtype=E4M3)[0]
    assert bool((y.float() == 448).all())                       # saturates


def test_linear_in_place_residual_bytes_streams_and_leading_dimensions():
    gen = torch.Generator("cuda").manual_seed(5)
    for M in (6, 270):
        x, w, res = rows_of(gen, M, 320, BF16), rows_of(gen, 200, 320, BF16), rows_of(gen, M, 200, BF16)
        ref = check(x, w, None, res, scale=0.1)
        y = res.clone()
        ecc.ecc_linear(x, w, None, y, scale=0.1, out=y)
        assert torch.equal(y, ref)
        y = ecc.ecc_linear(x.view(2, M // 2, 320), w, None, res.view(2, M // 2, 200), scale=0.1)[0]
        assert torch.equal(y.view(M, 200), ref)
        x8, w8 = x.to(E4M3), w.to(E4M3)
        assert torch.equal(ecc.ecc_linear(x8.view(torch.uint8), w8.view(torch.uint8))[0], check(x8, w8))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        xo, wo = rows_of(gen, M, 321, BF16)[:, :320], rows_of(gen, 200, 321, BF16)[:, :320]   # needs scratch
        ref = check(xo, wo)
        got = [ecc.ecc_linear(xo, wo, stream=s) for _ in range(4)]
        junk = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, ref) and int(st.item()) == 0 for y, st in got) and len(junk) == 4


def test_linear_repeats_bit_for_bit():
    gen = torch.Generator("cuda").manual_seed(6)
    for M, N, K in ((1, 4096, 4096), (7, 1111, 9000), (700, 900, 3000)):
        x, w = rows_of(gen, M, K, F16), rows_of(gen, N, K, F16)
        first = ecc.ecc_linear(x, w, out_dtype=F32)[0]
        assert all(torch.equal(ecc.ecc_linear(x, w, out_dtype=F32)[0], first) for _ in range(3))


def check_grad(dy, x, w, pre=None, act="none", scale=1.0, **kw):
    dx, dw, db, st = ecc.ecc_linear_grad(dy, x, w, pre, act=act, scale=scale, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == ecc.OK
    (M, N), K = dy.shape, x.shape[1]
    t = dy.double()
    et = torch.zeros_like(t)
    if act != "none":
        a = pre.double().requires_grad_()
        slope, = torch.autograd.grad(ACTS[act](a).sum(), a)
        a = a.detach()
        es = dy.double().abs() * (2.0**-19 * slope.abs() + 2.0**-20 * (1 + a.abs()) * (a.abs() < 20))
        t = t * slope
        et = es + U[dy.dtype] * t.abs() + TINY[dy.dtype]
        edb = es
    else:
        edb = et
    s = abs(scale)
    if dx is not None:
        ref = scale * (t @ w.double())
        e = s * (et @ w.double().abs() + (N + 8) * 2.0**-23 * (t.abs() @ w.double().abs()))
        assert bool(((dx.double() - ref).abs() <= 1.01 * U[dx.dtype] * ref.abs() + TINY[dx.dtype] + 1.01 * e).all())
    if dw is not None:
        ref = scale * (t.T @ x.double())
        e = s * (et.T @ x.double().abs() + (M + 8) * 2.0**-23 * (t.T.abs() @ x.double().abs()))
        assert bool(((dw.double() - ref).abs() <= 1.01 * U[dw.dtype] * ref.abs() + TINY[dw.dtype] + 1.01 * e).all())
    if db is not None:
        assert bool(((db.double() - t.sum(0)).abs() <= edb.sum(0) + (M + 16) * 2.0**-24 * t.abs().sum(0)).all())
    return dx, dw, db


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_grad_shapes(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 5 * N + 11 * K)
    for pad, off, act in ((0, 0, "gelu"), (16, 0, "none"), (5, 3, "silu"), (3, 0, "none")):
        x, w = rows_of(gen, M, K, dtype, pad, off), rows_of(gen, N, K, dtype, pad, std=1 / math.sqrt(N))
        dy, pre = rows_of(gen, M, N, dtype, pad), rows_of(gen, M, N, dtype, 2 * pad)
        check_grad(dy, x, w, pre, act)
    check_grad(dy, x, w, pre.float(), "relu", 0.5, dw_dtype=F32)


@pytest.mark.parametrize("act", list(ACTS))
def test_linear_grad_activations_wanted_outputs_and_repeats(act):
    gen = torch.Generator("cuda").manual_seed(12)
    x, w = rows_of(gen, 130, 200, BF16), rows_of(gen, 300, 200, BF16, std=0.05)
    dy, pre = rows_of(gen, 130, 300, BF16), rows_of(gen, 130, 300, BF16, std=3.0)
    first = check_grad(dy, x, w, pre, act, -2.0)
    for want in (("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ()):
        got = ecc.ecc_linear_grad(dy, x, w, pre, act=act, scale=-2.0, want=want)
        for name, g, f in zip(("dx", "dw", "dbias"), got, first):
            assert (g is None) if name not in want else torch.equal(g, f)


def test_linear_grad_against_differences():
    gen = torch.Generator("cuda").manual_seed(13)
    x, w = rows_of(gen, 6, 24, BF16), rows_of(gen, 16, 24, BF16, std=0.3)
    b, dy = rows_of(gen, 1, 16, F32)[0], rows_of(gen, 6, 16, BF16)
    for act in ("gelu", "gelu_tanh", "silu", "none"):
        pre = torch.empty(6, 16, dtype=F32, device="cuda")
        ecc.ecc_linear(x, w, b, act=act, pre=pre, scale=0.7)
        dx, dw, db, _ = ecc.ecc_linear_grad(dy, x, w, pre, act=act, scale=0.7, dw_dtype=F32)

        def loss(x, w, b):
            return float((ACTS[act](0.7 * x @ w.T + b) * dy.double()).sum())

        args = [x.double(), w.double(), b.double()]
        h = 1e-4
        for k in range(12):
            for at, grad in ((0, dx), (1, dw), (2, db)):
                t = args[at]
                i = (k % t.shape[0], (5 * k) % t.shape[1]) if t.dim() == 2 else (k,)
                e = torch.zeros_like(t)
                e[i] = h
                up, down = list(args), list(args)
                up[at], down[at] = t + e, t - e
                diff = (loss(*up) - loss(*down)) / (2 * h)
                # t is rounded to bfloat16 (2^-8 of at most 16 or 24 terms), dx too
                assert abs(diff - float(grad[i])) < 2.0**-8 * (abs(diff) + 4)


def test_linear_refusals():
    x, w = torch.randn(4, 64, device="cuda").to(BF16), torch.randn(32, 64, device="cuda").to(BF16)
    b, r = torch.randn(32, device="cuda"), torch.randn(4, 32, device="cuda")
    g = r.to(BF16)
    bad = [lambda: ecc.ecc_linear(x.float(), w.float()), lambda: ecc.ecc_linear(x, w.half()),
           lambda: ecc.ecc_linear(x, w[:, :63]), lambda: ecc.ecc_linear(x, w.t()), lambda: ecc.ecc_linear(x, w[0]),
           lambda: ecc.ecc_linear(x, w, act="tanh"), lambda: ecc.ecc_linear(x, w, b[:31]),
           lambda: ecc.ecc_linear(x, w, b.double()), lambda: ecc.ecc_linear(x, w, b, r[:3]),
           lambda: ecc.ecc_linear(x, w, residual=r.to(E4M3)), lambda: ecc.ecc_linear(x, w, out_scale=2.0),
           lambda: ecc.ecc_linear(x, w, scale=float("nan")), lambda: ecc.ecc_linear(x.cpu(), w),
           lambda: ecc.ecc_linear(x, w.cpu()), lambda: ecc.ecc_linear(x, w, out=r[:, :31]),
           lambda: ecc.ecc_linear(x, w, out_dtype=torch.float64), lambda: ecc.ecc_linear(x, w, pre=r[:3]),
           lambda: ecc.ecc_linear(x[:1].expand(4, 64), w),
           lambda: ecc.ecc_linear_grad(g, x, w, act="gelu"), lambda: ecc.ecc_linear_grad(r, x, w),
           lambda: ecc.ecc_linear_grad(g, x[:3], w), lambda: ecc.ecc_linear_grad(g, x, w[:31]),
           lambda: ecc.ecc_linear_grad(g, x, w, dw_dtype=F16),
           lambda: ecc.ecc_linear_grad(g.to(E4M3), x.to(E4M3), w.to(E4M3)),
           lambda: ecc.ecc_linear_grad(g, x, w, g, act="gelu", ws=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for call in bad:
        with pytest.raises(ecc.EccError) as e:
            call()
        assert e.value.code == ecc.ERR_ARG
