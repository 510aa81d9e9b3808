"""ecc_layer_norm and ecc_layer_norm_grad against a plain 64-bit computation.

Tolerances.  u is half a unit in the last place of the output type (2^-24
float32, 2^-8 bfloat16, 2^-11 float16, 2^-4 e4m3).  A float32 sum of n terms
spread over at least 32 lanes is off by at most g = (n / 32 + 16) 2^-24 of the
sum of the terms' magnitudes.  The mean is then off by g avg|x|, which shifts
xh by g rstd avg|x|; rstd is off by a relative 2 g: y is off by at most
4 g (1 + rstd max|x|) max|w| besides its own rounding u |y|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float8_e4m3fn: 2.0**-4}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0**-25, torch.float8_e4m3fn: 2.0**-10}
F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 33), (7, 256), (3, 1000), (2, 1003), (37, 1024), (300, 2048), (5, 4096),
          (2, 5003), (3, 8192), (2, 16384), (1, 20000), (2, 40003), (2000, 64), (999, 129)]


def g_of(n):
    return (n / 32 + 16) * 2.0**-24


def rows_of(gen, rows, cols, dtype, pad=0, off=0, std=1.0, mean=0.0):
    """[rows, cols] values in rows of cols + pad elements that start off elements into a buffer."""
    base = torch.randn(rows * (cols + pad) + off, generator=gen, device="cuda") * std + mean
    return base.to(dtype)[off:].view(rows, cols + pad)[:, :cols]


def check_norm(x, w, b, eps, out_dtype, out_scale=1.0, **kw):
    y, mean, rstd = ecc.ecc_layer_norm(x, w, b, eps=eps, out_dtype=out_dtype, out_scale=out_scale, **kw)
    torch.cuda.synchronize()
    xd = x.double()
    m = xd.mean(-1, keepdim=True)
    r = ((xd - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    ref = (xd - m) * r
    wm = 1.0 if w is None else float(w.double().abs().max())
    ref = ref if w is None else ref * w.double()
    ref = ref if b is None else ref + b.double()
    g = g_of(x.shape[-1])
    slack = 4 * g * (1 + r * xd.abs().amax(-1, keepdim=True)) * wm + 2.0**-22 * ref.abs()
    ref, slack = ref * out_scale, slack * out_scale
    if out_dtype == E4M3:
        ref = ref.clamp(-448, 448)
    err = (y.double() - ref).abs()
    assert bool((err <= U[out_dtype] * ref.abs() * 1.01 + TINY[out_dtype] + slack).all())
    am = xd.abs().mean(-1)
    assert bool(((mean.double() - m[..., 0]).abs() <= 2 * g * am + 1e-30).all())
    assert bool(((rstd.double() / r[..., 0] - 1).abs() <= 4 * g * (1 + r[..., 0] * am)).all())
    return y


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_shapes(rows, cols, dtype):
    gen = torch.Generator("cuda").manual_seed(rows * 7 + cols)
    for pad, off in ((0, 0), (8, 0), (5, 3)):
        x = rows_of(gen, rows, cols, dtype, pad, off)
        w, b = rows_of(gen, 1, cols, dtype)[0], rows_of(gen, 1, cols, dtype)[0]
        check_norm(x, w, b, 1e-5, dtype)
        check_norm(x, w.float(), None, 1e-5, E4M3, 16.0)
    check_norm(x, None, None, 1e-5, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", [(2101, 513), (700, 1537), (300, 5003), (270, 4099), (150, 8190), (2500, 1024),
                                       (2501, 256), (2600, 97), (2437, 4096), (2433, 2040)])
def test_norm_many_rows(rows, cols, dtype):
    """Enough rows for the kernels that several rows, or rows on any boundary, go through."""
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    w, b = rows_of(gen, 1, cols + 3, dtype)[0], rows_of(gen, 1, cols + 1, dtype)[0]
    for pad, off in ((0, 0), (5, 3), (8, 1), (3, 0)):
        x = rows_of(gen, rows, cols, dtype, pad, off)
        check_norm(x, w[:cols], b[1:], 1e-5, dtype)          # parameters on any boundary too
        check_norm(x, w[3:].float(), None, 1e-5, E4M3, 16.0)
        out = torch.empty_strided((rows, cols), (cols + 7, 1), dtype=dtype, device="cuda")
        check_norm(x, None, b[:cols], 1e-5, dtype, out=out)
        # in place: the bits of a call that writes rows of the same layout elsewhere
        base = torch.empty(rows * (cols + pad) + 8, dtype=dtype, device="cuda")
        y = base[:rows * (cols + pad)].view(rows, cols + pad)[:, :cols].copy_(x)
        other = torch.empty_like(base)[:rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        ecc.ecc_layer_norm(y, out=other)
        ecc.ecc_layer_norm(y, out=y)
        assert torch.equal(y, other)


def test_norm_large_mean_constant_rows_and_eps():
    gen = torch.Generator("cuda").manual_seed(5)
    x = rows_of(gen, 64, 1536, F32, mean=1000.0)   # a one-pass variance would lose all digits here
    check_norm(x, None, None, 1e-5, F32)
    x = torch.full((3, 512), 2.5, device="cuda")
    y, mean, rstd = ecc.ecc_layer_norm(x, eps=0.25)
    torch.cuda.synchronize()
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mean, torch.full_like(mean, 2.5))
    assert torch.equal(rstd, torch.full_like(rstd, 2.0))


def test_norm_non_finite_values_stay_in_their_row():
    x = torch.randn(5, 777, device="cuda", dtype=BF16)
    clean = ecc.ecc_layer_norm(x)[0]
    x[1, 5], x[3, 700] = float("nan"), float("inf")
    y, mean, rstd = ecc.ecc_layer_norm(x)
    torch.cuda.synchronize()
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().any()) and bool(mean[1].isnan())
    for r in (0, 2, 4):
        assert torch.equal(y[r], clean[r])
    z, _, _ = ecc.ecc_layer_norm(x, out_dtype=torch.uint8)
    assert bool(((z[1] & 0x7F) == 0x7F).all())   # e4m3 keeps NaN


def test_norm_in_place_leading_dimensions_and_empty():
    gen = torch.Generator("cuda").manual_seed(6)
    for cols in (640, 40003):
        x = rows_of(gen, 12, cols, BF16).view(3, 4, cols)
        ref = check_norm(x, None, None, 1e-5, BF16)
        y = x.clone()
        ecc.ecc_layer_norm(y, out=y)
        assert torch.equal(y, ref) and ref.shape == (3, 4, cols)
    y, mean, rstd = ecc.ecc_layer_norm(torch.empty(0, 64, device="cuda"))
    assert y.shape == (0, 64) and mean.shape == (0,)
    v = torch.randn(96, device="cuda")
    assert ecc.ecc_layer_norm(v)[1].shape == ()


def test_norm_offsets_past_32_bits():
    buf = torch.zeros((1 << 32) + 4096, dtype=BF16, device="cuda")
    x = buf.as_strided((3, 1000), ((1 << 31) + 8, 1))
    x.copy_(torch.randn(3, 1000, device="cuda"))
    check_norm(x, None, None, 1e-5, BF16)
    ref = x.float()
    got = ecc.ecc_layer_norm_grad(x, x, None, ref.mean(-1), torch.ones(3, device="cuda"))
    want = (ref.double() * (ref.double() - ref.mean(-1, keepdim=True).double())).sum(0)
    assert float((got[1].double() - want).abs().max()) < 1e-4


def check_grad(dy, x, w, mean, rstd, **kw):
    dx, dw, db = ecc.ecc_layer_norm_grad(dy, x, w, mean, rstd, **kw)
    torch.cuda.synchronize()
    n, rows = x.shape[-1], x.shape[0]
    d, r = dy.double(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    gw = d if w is None else d * w.double()
    ref = r * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    g = g_of(n)
    # xh itself is off by 2^-22 (|xh| + rstd |mean|); the two averages by g of theirs
    xe = 2.0**-22 * (xh.abs() + r * mean.double().abs()[:, None])
    a1, a2 = gw.abs().mean(-1, keepdim=True), (gw * xh).abs().mean(-1, keepdim=True)
    e2 = (gw.abs() * xe).mean(-1, keepdim=True)
    slack = r * (2.0**-21 * gw.abs() + 2 * g * a1 + xh.abs() * (2 * g * a2 + e2) + xe * a2 * 2)
    err = (dx.double() - ref).abs()
    assert bool((err <= U[x.dtype] * ref.abs() * 1.01 + TINY[x.dtype] + slack).all())
    gr = (rows + 16) * 2.0**-24
    assert bool(((dw.double() - (d * xh).sum(0)).abs() <= 2 * gr * (d * xh).abs().sum(0) + (d.abs() * xe).sum(0)).all())
    assert bool(((db.double() - d.sum(0)).abs() <= gr * d.abs().sum(0)).all())
    return dx, dw, db


def stats(x, eps=1e-5):
    xd = x.double()
    m = xd.mean(-1)
    return m.float(), ((xd - m[:, None]).square().mean(-1) + eps).rsqrt().float()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_grad_shapes(rows, cols, dtype):
    gen = torch.Generator("cuda").manual_seed(rows * 5 + cols)
    for pad, off in ((0, 0), (8, 0), (5, 1)):
        x, dy = rows_of(gen, rows, cols, dtype, pad, off), rows_of(gen, rows, cols, dtype, 2 * pad)
        w = rows_of(gen, 1, cols, dtype)[0]
        m, r = stats(x)
        first = check_grad(dy, x, w, m, r)
        again = ecc.ecc_layer_norm_grad(dy, x, w, m, r)
        assert all(torch.equal(p, q) for p, q in zip(first, again))   # the sums' order is fixed
    check_grad(dy, x, None, m, r)
    check_grad(dy, x, w.float(), m, r)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols", [(2501, 513), (3001, 7), (2900, 256), (1301, 1537), (1503, 4099), (1100, 4096), (801, 8190),
                                       (700, 9001), (650, 16000)])
def test_norm_grad_many_rows(rows, cols, dtype):
    """Several steps of every ring, rows on and off 16-byte boundaries, each
    of the arrays on its own; dx in place, next to other rows' bytes."""
    gen = torch.Generator("cuda").manual_seed(rows * 9 + cols)
    for pad, off, dpad, doff in ((0, 0, 0, 0), (0, 0, 8, 0), (3, 1, 0, 0), (1, 3, 6, 5)):
        x, dy = rows_of(gen, rows, cols, dtype, pad, off), rows_of(gen, rows, cols, dtype, dpad, doff)
        w = rows_of(gen, 1, cols, dtype, 0, off)[0]
        m, r = stats(x)
        dx, dw, db = check_grad(dy, x, w, m, r)
        rest = ecc.ecc_layer_norm_grad(dy, x, w, m, r)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), rest))
        # in place: the padding stays, the rest are the bits of a call on the same layout
        for into, ld in ((x, cols + pad), (dy, cols + dpad)):
            base = torch.full((rows * ld + 8,), 7.0, dtype=dtype, device="cuda")
            y = base[off if into is x else doff:][:rows * ld].view(rows, ld)[:, :cols].copy_(into)
            args = (dy, y, w, m, r) if into is x else (y, x, w, m, r)
            kept = ecc.ecc_layer_norm_grad(*args, dx=torch.empty_like(base)[off if into is x else doff:][:rows * ld]
                                           .view(rows, ld)[:, :cols])
            got = ecc.ecc_layer_norm_grad(*args, dx=y)
            assert all(torch.equal(p, q) for p, q in zip(kept, got))
            whole = base[off if into is x else doff:][:rows * ld].view(rows, ld)
            assert bool((whole[:, cols:] == 7).all()) and bool((base[:off if into is x else doff] == 7).all())


def test_norm_grad_in_place_and_empty():
    gen = torch.Generator("cuda").manual_seed(9)
    for cols in (1024, 40003):
        x, dy = rows_of(gen, 50, cols, BF16), rows_of(gen, 50, cols, BF16)
        m, r = stats(x)
        ref = check_grad(dy, x, None, m, r)
        for target in (0, 1):
            args = [dy.clone(), x.clone()]
            got = ecc.ecc_layer_norm_grad(args[0], args[1], None, m, r, dx=args[target])
            assert all(torch.equal(p, q) for p, q in zip(got, ref))
    e = torch.empty(0, 48, device="cuda")
    _, dw, db = ecc.ecc_layer_norm_grad(e, e, None, e[:, 0].contiguous(), e[:, 0].contiguous())
    assert not dw.any() and not db.any()


def test_norm_grad_against_differences():
    gen = torch.Generator("cuda").manual_seed(11)
    x, w, b = (rows_of(gen, r, 24, F32) for r in (6, 1, 1))
    dy = rows_of(gen, 6, 24, F32)
    y, m, r = ecc.ecc_layer_norm(x, w[0], b[0])
    dx, dw, db = ecc.ecc_layer_norm_grad(dy, x, w[0], m, r)

    def loss(x, w, b):
        x = x.double()
        d = x - x.mean(-1, keepdim=True)
        return float(((d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w.double() + b.double())
                      * dy.double()).sum())

    h = 1e-4   # central differences in 64 bits: error O(h^2) = 1e-8 against float32's 1e-6
    for k in range(12):
        for t, grad in ((x, dx), (w, dw[None]), (b, db[None])):
            i, j = k % t.shape[0], (5 * k) % 24
            e = torch.zeros_like(t, dtype=torch.float64)
            e[i, j] = h
            args = [a.double() for a in (x, w, b)]
            at = [x is t, w is t, b is t].index(True)
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + e, args[at] - e
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - float(grad[i, j])) < 2e-5 * (1 + abs(diff)) * 4


def test_norm_on_another_stream():
    x = torch.randn(513, 2048, device="cuda", dtype=BF16)
    ref = ecc.ecc_layer_norm(x)[0]
    m, r = stats(x)
    gref = ecc.ecc_layer_norm_grad(x, x, None, m, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y = ecc.ecc_layer_norm(x, stream=s)[0]
        got = ecc.ecc_layer_norm_grad(x, x, None, m, r, stream=s)
        torch.randn(1 << 20, device="cuda")    # the default stream's allocations meanwhile
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and all(torch.equal(p, q) for p, q in zip(got, gref))


def test_norm_refusals():
    x = torch.randn(4, 64, device="cuda")
    bad = [lambda: ecc.ecc_layer_norm(x.double()), lambda: ecc.ecc_layer_norm(x.t()),
           lambda: ecc.ecc_layer_norm(x, eps=-1.0), lambda: ecc.ecc_layer_norm(x, eps=float("nan")),
           lambda: ecc.ecc_layer_norm(x, out_dtype=BF16), lambda: ecc.ecc_layer_norm(x, out_scale=2.0),
           lambda: ecc.ecc_layer_norm(x, weight=torch.ones(63, device="cuda")),
           lambda: ecc.ecc_layer_norm(x, weight=torch.ones(64, device="cuda", dtype=F16)),
           lambda: ecc.ecc_layer_norm(x, weight=torch.ones(64)), lambda: ecc.ecc_layer_norm(x.cpu()),
           lambda: ecc.ecc_layer_norm(x[:1].expand(4, 64)), lambda: ecc.ecc_layer_norm(x[:, :0]),
           lambda: ecc.ecc_layer_norm(x, out=x[:3]),
           lambda: ecc.ecc_layer_norm_grad(x, x[:3], None, x[:, 0].contiguous(), x[:, 0].contiguous()),
           lambda: ecc.ecc_layer_norm_grad(x, x, None, x[:, 0], x[:, 0]),
           lambda: ecc.ecc_layer_norm_grad(x, x, None, x[:, 0].contiguous(), x[:, 0].contiguous(),
                                           ws=torch.empty(64, dtype=torch.uint8, device="cuda"))]
    for call in bad:
        with pytest.raises(ecc.EccError) as e:
            call()
        assert e.value.code == ecc.ERR_ARG
