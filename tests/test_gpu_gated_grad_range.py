"""The gated projections' backward pass in float16, whose exponents do not hold
the products dy u and dy act(g): small and large ones, scales and halves far
apart, values that are not finite.

Tolerances: those of the operator's own tests (test_gpu_gated.check_grad), but
for the smallest steps of t = tg, tu.  A power of two brings an operand's
largest value to at least 2^14, so that half a smallest step, 2^-25 there, is
at most 2^-39 of that value: for the weights' gradients the largest of their
own half, for dx the larger of scale tg and up_scale tu."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_gated as gated  # noqa: E402

F32, F16 = torch.float32, torch.float16
U, TINY, STEP = 2.0**-11, {F16: 2.0**-25, F32: 2.0**-149}, 1.01 * 2.0**-39


def check(dy, x, wg, wu, g, u, act, scale=1.0, up=1.0, **kw):
    r = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, act=act, scale=scale, up_scale=up, dw_dtype=F32, **kw)
    torch.cuda.synchronize()
    assert int(r[5].item()) == ecc.OK
    M, N = dy.shape
    a, d, ud = g.double().requires_grad_(), dy.double(), u.double()
    h = gated.ACTS[act](a)
    slope, = torch.autograd.grad(h.sum(), a)
    a, h = a.detach(), h.detach()
    near = (1 + a.abs()) * (a.abs() < 20)
    es, eh = 2.0**-19 * slope.abs() + 2.0**-20 * near, 2.0**-19 * h.abs() + 2.0**-20 * near
    if act in ("none", "relu"):
        es = eh = torch.zeros_like(a)
    tg, tu = d * ud * slope, d * h
    eg, eu = (d * ud).abs() * es + 2.0**-21 * tg.abs(), d.abs() * eh + 2.0**-21 * tu.abs()
    mg, mu = tg.abs().amax(), tu.abs().amax()
    gd, wd, xd = wg.double(), wu.double(), x.double()
    if r[0] is not None:
        most = torch.maximum(abs(scale) * mg, abs(up) * mu)
        e = (abs(scale) * (eg + U * tg.abs()) + STEP * most) @ gd.abs() + (abs(up) * (eu + U * tu.abs()) + STEP * most) @ wd.abs()
        sums = abs(scale) * (tg.abs() @ gd.abs()) + abs(up) * (tu.abs() @ wd.abs())
        ref = scale * (tg @ gd) + up * (tu @ wd)
        e = 1.01 * U * ref.abs() + TINY[F16] + 1.01 * e + (2 * N + 136) * 2.0**-23 * sums
        assert bool(((r[0].double() - ref).abs() <= e).all()) and bool(torch.isfinite(r[0]).all())
    for got, t, e, m, s in ((r[1], tg, eg, mg, scale), (r[2], tu, eu, mu, up)):
        if got is not None:
            ref = s * (t.T @ xd)
            e = abs(s) * ((e + U * t.abs() + STEP * m).T @ xd.abs() + (M + 8) * 2.0**-23 * (t.T.abs() @ xd.abs()))
            assert bool(((got.double() - ref).abs() <= 2.0**-22 * ref.abs() + TINY[F32] + 1.01 * e).all())
    return r


# split and pair kernels, rows on any boundary, weight gradients through shared memory
SHAPES = [(3, 5, 7, 0), (70, 200, 96, 0), (257, 1000, 771, 0), (2100, 3008, 1024, 0), (200, 8200, 2048, 0), (1111, 2500, 1030, 3)]


def inputs(M, N, K, pad=0):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    return ([gated.rows_of(gen, r, K, F16, pad, std=s) for r, s in ((M, 1.0), (N, N**-0.5), (N, N**-0.5))],
            [gated.rows_of(gen, M, N, F32) for _ in range(3)])


@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
@pytest.mark.parametrize("sy,su,sx", [(1e-5, 1e-2, 64.0), (1e-4, 1e-4, 1.0), (300.0, 300.0, 2.0**-10), (1e-6, 1e4, 1.0), (2e4, 1e-6, 1.0)])
@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_products_beyond_the_range(M, N, K, pad, sy, su, sx, act):
    (x, wg, wu), (dy, g, u) = inputs(M, N, K, pad)
    dy, u = (dy * sy).clamp(-65000, 65000).to(F16), u * su
    # (dx in float16 itself: weights that bring it into the range)
    k = 1 / max(sy * max(su, 1.0), 1e-3)
    wg, wu = (w * min(k, 100.0) for w in (wg, wu))
    check(dy, x * sx, wg, wu, g, u, act)
    check(dy, x * sx, wg, wu, g.half(), u.clamp(-65000, 65000).half(), act)


@pytest.mark.parametrize("scales", [(1.0, 1e-4), (1e-4, 1.0), (-1.0, 3e-7), (1e3, 1e-3), (1.0, 0.0), (0.0, 0.5)])
@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_scales_far_apart(M, N, K, pad, scales):
    (x, wg, wu), (dy, g, u) = inputs(M, N, K, pad)
    r = check(dy.half(), x, wg, wu, g.half(), u.half(), "silu", *scales)
    # each half's gradient is what it is with equal scales, times its own
    one = check(dy.half(), x, wg, wu, g.half(), u.half(), "silu", 1.0, 1.0)
    for got, ref, s in zip(r[1:3], one[1:3], scales):
        assert bool(((got.double() - s * ref.double()).abs() <= 2.0**-22 * (s * ref.double()).abs()).all())


@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_values_that_are_not_finite_stay_in_place(M, N, K, pad):
    (x, wg, wu), (dy, g, u) = inputs(M, N, K, pad)
    dy = (dy * 1e-5).half()
    dy[1, 2] = 0
    want = check(dy, x, wg, wu, g, u * 1e-2, "silu")
    rows, cols = torch.arange(M, device="cuda") != 1, torch.arange(N, device="cuda") != 2
    for bad in (math.inf, math.nan):
        dy[1, 2] = bad
        got = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u * 1e-2, dw_dtype=F32)
        assert torch.equal(got[0][rows], want[0][rows]) and not bool(torch.isfinite(got[0][1]).all())
        for a, b in zip(got[1:5], want[1:5]):
            assert torch.equal(a[cols], b[cols]) and not bool(torch.isfinite(a[2]).all())


@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_what_is_wanted_changes_nothing_and_powers_of_two_only_scale(M, N, K, pad):
    (x, wg, wu), (dy, g, u) = inputs(M, N, K, pad)
    dy = dy.half()
    first = check(dy, x, wg, wu, g, u, "gelu_tanh", 0.5, 2.0)
    # (the same products in the same launches: their order of summation is the same)
    for pair in ((("dx", "dw", "dbias"), ("dx", "dw")), (("dx", "dbias"), ("dx",)), (("dw", "dbias"), ("dw",))):
        a, b = (ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, act="gelu_tanh", scale=0.5, up_scale=2.0, dw_dtype=F32, want=w) for w in pair)
        for name, p, q, f in zip(("dx", "dw", "dw", "dbias", "dbias"), a, b, first):
            assert (p is None) == (name not in pair[0]) and (q is None) == (name not in pair[1])
            assert q is None or torch.equal(p, q)
            assert name != "dbias" or p is None or torch.equal(p, f)
    small = dy.clone()
    small[small.abs() < 2.0**-8] = 0                      # (so that 2^-6 of it is exact)
    a = check(small, x, wg, wu, g, u, "gelu_tanh")
    b = check(small * 2.0**-6, x, wg, wu, g, u, "gelu_tanh")
    assert all(torch.equal(p, q * 64) for p, q in zip(a[1:3], b[1:3]))


def test_captured_and_replayed_and_in_one_workspace():
    """Each call finds its own powers of two, also one that the stream starts early behind another."""
    cases = []
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for M, N, K, pad in ((257, 1000, 771, 0), (600, 1500, 520, 3)):
        (x, wg, wu), (dy, g, u) = inputs(M, N, K, pad)
        dys = [(dy * s).half() for s in (1.0, 1e-4, 2e3)]
        alone = [ecc.ecc_gated_linear_grad(d, x, wg, wu, g, u, dw_dtype=F32, want=("dw",)) for d in dys]
        cases.append((x, wg, wu, g, u, dys, alone))
    got = [[ecc.ecc_gated_linear_grad(d, x, wg, wu, g, u, dw_dtype=F32, want=("dw",), ws=ws) for x, wg, wu, g, u, dys, _ in cases
            for d in dys] for _ in range(4)]
    torch.cuda.synchronize()
    flat = [a for c in cases for a in c[6]]
    assert all(torch.equal(p, q) for r in got for a, b in zip(r, flat) for p, q in zip(a[1:3], b[1:3]))
    for x, wg, wu, g, u, dys, alone in cases:
        d, stream, graph = dys[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            r = ecc.ecc_gated_linear_grad(d, x, wg, wu, g, u, dw_dtype=F32, want=("dw",), ws=ws)
        for dy, a in zip(dys, alone):
            d.copy_(dy)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(r[1:3], a[1:3])) and int(r[5].item()) == 0
