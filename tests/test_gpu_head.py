"""ecc_linear_logprob and ecc_linear_logprob_grad against a plain 64-bit
computation of the logits.

Tolerances.  A logit is off by ez = scale (K + 8) 2^-23 sum |x||w| (float32
sums, each addition truncated) and 2^-22 of itself (the scale with log2 e in
it, their product).  lse follows the largest of them, and its exponentials
(2^-22 each), sum and logarithm add 2^-20.  The entropy's slope in a logit is
-p (log p + H), and sum p |log p + H| is at most 2 log vocab + 1; its own terms
add 2^-20 of that.  p is off by a relative ez + 2^-22 (|z| + |lse|) + 2^-20; t
by that times its factor, by dentropy's own error, and by half a step of its
type, with F16's smallest step divided by the power of two that brings
max(|dlogprob| + 16 |dentropy|) to at least 2^14.  The products add their terms'
errors and (n + 8) 2^-23 of the sum of magnitudes (n + 16 for sums in pieces).
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
U = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}
TINY = {F32: 2.0**-149, BF16: 2.0**-133, F16: 2.0**-25}


def rows_of(gen, rows, cols, dtype, pad=0, off=0, std=1.0):
    base = torch.randn(rows * (cols + pad) + off, generator=gen, device="cuda") * std
    return base.to(dtype)[off:].view(rows, cols + pad)[:, :cols]


def tokens_of(gen, rows, vocab):
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[torch.rand(rows, generator=gen, device="cuda") < 0.2] = -1
    return t


def logits(x, w, scale):
    z = scale * (x.double() @ w.double().T)
    return z, abs(scale) * (x.shape[1] + 8) * 2.0**-23 * (x.double().abs() @ w.double().abs().T) + 2.0**-22 * z.abs()


def check(x, w, tokens=None, scale=1.0, **kw):
    r = ecc.ecc_linear_logprob(x, w, tokens, scale=scale, **kw)
    torch.cuda.synchronize()
    assert int(r.status.item()) == ecc.OK
    V = w.shape[0]
    z, ez = logits(x, w, scale)
    logp = torch.log_softmax(z, -1)
    lse, ent = torch.logsumexp(z, -1), -(logp.exp() * logp).sum(-1)
    far = ez.amax(-1) + 2.0**-20
    assert bool(((r.lse.double() - lse).abs() <= far + 2.0**-22 * lse.abs()).all())
    assert bool(((r.entropy.double() - ent).abs() <= (2 * math.log(V) + 1) * (2 * far + 2.0**-20)).all())
    if tokens is None:
        assert r.logprob is None
    else:
        has = tokens >= 0
        lp = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
        assert bool(((r.logprob.double() - lp).abs() <= 2 * far + 2.0**-22 * (lse.abs() + lp.abs()))[has].all())
        assert not r.logprob[~has].any()
    return r


# rows, vocab, K
SHAPES = [(1, 1, 1), (1, 2, 8), (3, 5, 7), (1, 1000, 512), (2, 64, 4096), (5, 4096, 64), (16, 2048, 2048), (17, 129, 65),
          (64, 513, 1000), (65, 1000, 129), (128, 128, 64), (128, 257, 8192), (129, 257, 192), (200, 333, 1001),
          (256, 256, 256), (511, 769, 520), (1000, 1024, 96), (2048, 641, 320), (33, 16384, 72), (6, 24, 16384),
          (1, 50021, 256), (7, 70001, 64), (300, 20000, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_head_shapes(M, V, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 3 * V + 7 * K)
    s = 2 / math.sqrt(K)
    for pad, off in ((0, 0), (16, 0), (5, 3)):
        x, w = rows_of(gen, M, K, dtype, pad, off), rows_of(gen, V, K, dtype, 2 * pad)
        check(x, w, tokens_of(gen, M, V), s)
    check(rows_of(gen, M, K, dtype, 3), rows_of(gen, V, K, dtype), None, -s)
    check(rows_of(gen, M, K, dtype), rows_of(gen, V, K, dtype, 3), torch.full((M,), V - 1, device="cuda"), 5 * s)


def test_head_agrees_with_the_logits_in_memory():
    gen = torch.Generator("cuda").manual_seed(1)
    x, w = rows_of(gen, 70, 256, BF16), rows_of(gen, 3001, 256, BF16, std=0.1)
    tok = tokens_of(gen, 70, 3001)
    a = check(x, w, tok, 1.5)
    z, st = ecc.ecc_linear(x, w, scale=1.5, out_dtype=F32)
    b = ecc.ecc_token_logprob(z, tok)
    assert int(st.item()) == 0
    for p, q in zip(a[:3], b[:3]):   # the same logits to 2^-18 each: K = 256 products of unit size, twice
        assert float((p - q).abs().max()) < 2.0**-14
    c = ecc.ecc_linear_logprob(x.view(7, 10, 256), w, tok.view(7, 10), scale=1.5)
    assert all(torch.equal(p.view(-1), q) for p, q in zip(c[:3], a[:3]))


def test_head_tokens_out_of_range_and_peaked_rows():
    x = torch.zeros(6, 64, dtype=BF16, device="cuda")
    w = torch.zeros(300, 64, dtype=BF16, device="cuda")
    w[7, 0] = 64
    x[1, 0], x[2, 0], x[3, 0], x[4, 0] = 4, -4, 100, -100      # logits of 256, -256, 6400, -6400 at index 7
    tok = torch.tensor([7, 7, 7, 300, -5, 1 << 40], device="cuda")
    r = ecc.ecc_linear_logprob(x, w, tok)
    lse = [math.log(300), 256, math.log(299), 6400, math.log(299), math.log(300)]
    ent = [math.log(300), 0, math.log(299), 0, math.log(299), math.log(300)]
    for i in range(6):
        assert abs(float(r.lse[i]) - lse[i]) < 1e-5 * (1 + lse[i]) and abs(float(r.entropy[i]) - ent[i]) < 1e-5
    assert abs(float(r.logprob[0]) + math.log(300)) < 1e-5 and abs(float(r.logprob[1])) < 1e-4
    assert abs(float(r.logprob[2]) + 256 + math.log(299)) < 1e-4
    assert math.isnan(float(r.logprob[3])) and float(r.logprob[4]) == 0 and math.isnan(float(r.logprob[5]))


def test_head_values_that_are_not_finite():
    gen = torch.Generator("cuda").manual_seed(4)
    for M, V, K in ((4, 300, 200), (300, 1400, 264)):
        x, w = rows_of(gen, M, K, BF16), rows_of(gen, V, K, BF16)
        tok = torch.zeros(M, dtype=torch.int64, device="cuda")
        clean = check(x, w, tok, 0.1)
        for bad in (math.nan, math.inf, -math.inf):
            x2 = x.clone()
            x2[1, 3] = bad
            r = ecc.ecc_linear_logprob(x2, w, tok, scale=0.1)
            for got, ref in zip(r[:3], clean[:3]):
                assert math.isnan(float(got[1])) and torch.equal(got[2:], ref[2:]) and torch.equal(got[0], ref[0])
            w2 = w.clone()
            w2[5, 3] = bad
            assert all(bool(t.isnan().all()) for t in ecc.ecc_linear_logprob(x, w2, tok, scale=0.1)[:3])


def test_head_zero_lengths_and_large_offsets():
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    r = ecc.ecc_linear_logprob(e(0, 16), e(8, 16), torch.empty(0, dtype=torch.int64, device="cuda"))
    assert r.lse.shape == (0,) and int(r.status.item()) == 0
    for M in (3, 200):
        r = ecc.ecc_linear_logprob(e(M, 0), e(40, 0), torch.zeros(M, dtype=torch.int64, device="cuda"))
        assert bool(((r.lse - math.log(40)).abs() < 1e-6).all()) and bool(((r.logprob + math.log(40)).abs() < 1e-6).all())
    dx, dw, st = ecc.ecc_linear_logprob_grad(e(0, 16), e(8, 16), torch.empty(0, dtype=torch.int64, device="cuda"),
                                             torch.empty(0, device="cuda"))
    assert dx.shape == (0, 16) and not dw.any() and int(st.item()) == 0
    dx, dw, st = ecc.ecc_linear_logprob_grad(e(3, 0), e(8, 0), None, torch.zeros(3, device="cuda"))
    assert dx.shape == (3, 0) and dw.shape == (8, 0) and int(st.item()) == 0
    gen = torch.Generator("cuda").manual_seed(3)
    buf = torch.zeros((1 << 32) + 4096, dtype=BF16, device="cuda")
    far = buf.as_strided((3, 512), ((1 << 31) + 8, 1))
    far.copy_(torch.randn(3, 512, device="cuda"))
    for M in (3, 150):
        near = rows_of(gen, M, 512, BF16)
        tok = torch.zeros(M, dtype=torch.int64, device="cuda")
        check(near, far, tok, 0.1)
        check_grad(near, far, tok, 0.1)
        check(far, near, tok[:3], 0.1)
        check_grad(far, near, tok[:3], 0.1)


def test_head_repeats_streams_and_graphs():
    gen = torch.Generator("cuda").manual_seed(6)
    for M, V, K in ((1, 4096, 512), (7, 1111, 900), (700, 3001, 321)):
        x, w, tok = rows_of(gen, M, K, F16), rows_of(gen, V, K, F16, std=0.1), tokens_of(gen, M, V)
        dlp, dh = torch.randn(M, generator=gen, device="cuda"), torch.randn(M, generator=gen, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            r = ecc.ecc_linear_logprob(x, w, tok)
            g = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, r.entropy, dlp, dh)
        for _ in range(3):
            x.copy_(torch.randn(M, K, generator=gen, device="cuda"))
            graph.replay()
            ref = check(x, w, tok)
            want = ecc.ecc_linear_logprob_grad(x, w, tok, ref.lse, ref.entropy, dlp, dh)
            assert all(torch.equal(a, b) for a, b in zip(r, ref)) and all(torch.equal(a, b) for a, b in zip(g, want))
        got = [ecc.ecc_linear_logprob(x, w, tok, stream=stream) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(t.lse, ref.lse) and int(t.status.item()) == 0 for t in got)


def check_grad(x, w, tokens, scale=1.0, dlogprob=None, dentropy=None, **kw):
    M, V = x.shape[0], w.shape[0]
    z, ez = logits(x, w, scale)
    logp = torch.log_softmax(z, -1)
    p, full = logp.exp(), torch.logsumexp(z, -1)
    ent = -(p * logp).sum(-1)
    if dlogprob is None and dentropy is None:
        dlogprob = torch.ones(M, device="cuda")
    dx, dw, st = ecc.ecc_linear_logprob_grad(x, w, tokens, full.float(), ent.float(), dlogprob, dentropy, scale=scale, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == ecc.OK
    zero = torch.zeros(M, dtype=torch.float64, device="cuda")
    dlp = zero if dlogprob is None or tokens is None else torch.where((tokens >= 0) & (tokens < V), dlogprob.double(), 0)
    dh = zero if dentropy is None else dentropy.double()
    if tokens is not None:
        hot = torch.zeros_like(z).scatter_(1, tokens.clamp(0, V - 1)[:, None], dlp[:, None])
    else:
        hot = torch.zeros_like(z)
    t = hot - p * dlp[:, None] - dh[:, None] * p * (logp + ent[:, None])
    q = dlp[:, None].abs() + (dh[:, None] * (logp + ent[:, None])).abs()
    off = ez + 2.0**-22 * (z.abs() + full.abs()[:, None]) + 2.0**-20
    et = p * (q * off + dh.abs()[:, None] * (off + 2.0**-22 * (full.abs() + ent)[:, None])) + 2.0**-22 * hot.abs()
    top = float((dlp.abs() + 16 * dh.abs()).max()) if M else 0.0
    tiny = TINY[x.dtype] * (2 * top * 2.0**-14 if x.dtype == F16 else 1.0)
    et = et + U[x.dtype] * t.abs() + tiny
    s = abs(scale)
    wd, xd = w.double(), x.double()
    if dx is not None:
        ref = scale * (t @ wd)
        e = s * (et @ wd.abs() + (V + 16) * 2.0**-23 * (t.abs() @ wd.abs()))
        assert bool(((dx.double() - ref).abs() <= 1.01 * U[dx.dtype] * ref.abs() + TINY[dx.dtype] + 1.01 * e).all())
    if dw is not None:
        ref = scale * (t.T @ xd)
        e = s * (et.T @ xd.abs() + (M + 8) * 2.0**-23 * (t.T.abs() @ xd.abs()))
        assert bool(((dw.double() - ref).abs() <= 1.01 * U[dw.dtype] * ref.abs() + TINY[dw.dtype] + 1.01 * e).all())
    return dx, dw


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_head_grad_shapes(M, V, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + 5 * V + 11 * K)
    s = 2 / math.sqrt(K)
    for pad, off in ((0, 0), (16, 0), (5, 3)):
        x, w = rows_of(gen, M, K, dtype, pad, off), rows_of(gen, V, K, dtype, 2 * pad)
        tok = tokens_of(gen, M, V)
        check_grad(x, w, tok, s, torch.randn(M, generator=gen, device="cuda"))
        check_grad(x, w, tok, s, torch.randn(M, generator=gen, device="cuda") * 1e-4, torch.randn(M, generator=gen, device="cuda") * 1e-3,
                   dw_dtype=F32)
    check_grad(x, w, None, -s, None, torch.randn(M, generator=gen, device="cuda") * 1e4)


def test_head_grad_in_pieces():
    """More rows times vocabulary than a piece of the workspace holds; the last piece is shorter."""
    gen = torch.Generator("cuda").manual_seed(8)
    M, V, K = 8192, 33000, 72
    for dtype in (BF16, F16):
        x, w, tok = rows_of(gen, M, K, dtype), rows_of(gen, V, K, dtype, std=0.2), tokens_of(gen, M, V)
        tok[:4] = torch.tensor([0, 16639, 16640, V - 1])
        dlp, dh = torch.randn(M, generator=gen, device="cuda"), torch.randn(M, generator=gen, device="cuda") * 0.1
        r = ecc.ecc_linear_logprob(x, w, tok)
        dx, dw, st = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, r.entropy, dlp, dh)
        only = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, r.entropy, dlp, dh, want=("dx",))
        assert int(st.item()) == 0 and torch.equal(only[0], dx) and only[1] is None
        # against the gradients of slices: a few rows for dx, a few of the vocabulary for dw
        pick = torch.arange(0, M, 1021, device="cuda")
        z = x[pick].double() @ w.double().T
        logp = torch.log_softmax(z, -1)
        p, ent = logp.exp(), r.entropy[pick].double()[:, None]
        lp = torch.where(tok[pick] >= 0, dlp[pick], 0).double()[:, None]
        t = -p * lp - dh[pick].double()[:, None] * p * (logp + ent)
        t.scatter_add_(1, tok[pick].clamp(min=0)[:, None], lp)
        ref = t @ w.double()
        # each term of t is off by at most half a step and 2^-12 of itself (logits of up to 30, lse)
        e = (U[dtype] + 2.0**-12) * (t.abs() @ w.double().abs()) + U[dtype] * ref.abs() + 2.0**-24
        assert bool(((dx[pick].double() - ref).abs() <= e).all())
        some = torch.tensor([0, 1, 16638, 16639, 16640, 32767, V - 1], device="cuda")
        full = r.lse.double()
        zs = x.double() @ w[some].double().T
        ps = (zs - full[:, None]).exp()
        lp = torch.where(tok >= 0, dlp, 0).double()[:, None]
        t = (tok[:, None] == some).double() * lp - ps * lp - dh.double()[:, None] * ps * (zs - full[:, None] + r.entropy.double()[:, None])
        ref = t.T @ x.double()
        e = (U[dtype] + 2.0**-12) * (t.T.abs() @ x.double().abs()) + U[dtype] * ref.abs() + 2.0**-24
        assert bool(((dw[some].double() - ref).abs() <= e).all())


def test_head_grad_calls_back_to_back_in_one_workspace():
    """F16's power of two is each call's own, also where the next call's first kernel could start early."""
    gen = torch.Generator("cuda").manual_seed(9)
    M, V, K = 256, 20000, 512
    x, w, tok = rows_of(gen, M, K, F16), rows_of(gen, V, K, F16, std=0.1), tokens_of(gen, M, V)
    r = ecc.ecc_linear_logprob(x, w, tok)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    scales = [torch.full((M,), 2.0**(12 * (i % 3) - 12), device="cuda") for i in range(12)]
    alone = []
    for s in scales[:3]:
        alone.append(ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, s, dw_dtype=F32, ws=ws))
        torch.cuda.synchronize()
    got = [ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, s, dw_dtype=F32, ws=ws) for s in scales]
    for i, (dx, dw, st) in enumerate(got):
        assert torch.equal(dx, alone[i % 3][0]) and torch.equal(dw, alone[i % 3][1]) and int(st.item()) == 0


def test_head_grad_wanted_outputs_and_given_tensors():
    gen = torch.Generator("cuda").manual_seed(12)
    for M, V, K in ((130, 300, 200), (600, 2000, 320)):
        x, w, tok = rows_of(gen, M, K, BF16), rows_of(gen, V, K, BF16, std=0.1), tokens_of(gen, M, V)
        dlp = torch.randn(M, generator=gen, device="cuda")
        first = check_grad(x, w, tok, 1.0, dlp)
        assert torch.equal(check_grad(x, w, tok, 1.0, dlp, want=("dx",))[0], first[0])
        assert torch.equal(check_grad(x, w, tok, 1.0, dlp, want=("dw",))[1], first[1])
        assert ecc.ecc_linear_logprob_grad(x, w, tok, torch.ones(M, device="cuda"), want=())[:2] == (None, None)
        whole = [torch.full((r + 2, K + 9), 7.0, dtype=BF16, device="cuda") for r in (M, V)]
        views = [t[1:-1, 4:-5] for t in whole]
        got = check_grad(x, w, tok, 1.0, dlp, dx=views[0], dw=views[1])
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        for t, v in zip(whole, views):
            v.fill_(7)
            assert bool((t == 7).all())


def test_head_grad_against_differences():
    gen = torch.Generator("cuda").manual_seed(13)
    x, w = rows_of(gen, 6, 24, BF16), rows_of(gen, 40, 24, BF16, std=0.3)
    tok = torch.tensor([3, -1, 39, 0, 3, 17], device="cuda")
    dlp, dh = rows_of(gen, 2, 6, F32)
    r = ecc.ecc_linear_logprob(x, w, tok, scale=0.7)
    dx, dw, _ = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, r.entropy, dlp, dh, scale=0.7, dw_dtype=F32)

    def loss(x, w):
        logp = torch.log_softmax(0.7 * x @ w.T, -1)
        lp = torch.where(tok >= 0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0], 0)
        return float((dlp.double() * lp - dh.double() * (logp.exp() * logp).sum(-1)).sum())

    args = [x.double(), w.double()]
    h = 1e-4
    for k in range(24):
        for at, grad in ((0, dx), (1, dw)):
            t = args[at]
            i = (k % t.shape[0], (5 * k) % t.shape[1])
            e = torch.zeros_like(t)
            e[i] = h
            up, down = list(args), list(args)
            up[at], down[at] = t + e, t - e
            diff = (loss(*up) - loss(*down)) / (2 * h)
            # t is rounded to bfloat16 (2^-8 of terms whose magnitudes sum to at most 8), dx too
            assert abs(diff - float(grad[i])) < 2.0**-8 * (abs(diff) + 8)


def test_head_refusals():
    x, w = torch.randn(4, 64, device="cuda").to(BF16), torch.randn(32, 64, device="cuda").to(BF16)
    tok, l = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    f, d = ecc.ecc_linear_logprob, ecc.ecc_linear_logprob_grad
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [lambda: f(x.float(), w.float(), tok), lambda: f(x, w.half(), tok), lambda: f(x, w[:, :63], tok), lambda: f(x, w[0], tok),
           lambda: f(x, w, tok[:3]), lambda: f(x, w, tok.int()), lambda: f(x, w, tok.cpu()), lambda: f(x, w[:0], tok),
           lambda: f(x, w, tok, scale=float("inf")), lambda: f(x.cpu(), w, tok), lambda: f(x, w.cpu(), tok),
           lambda: f(x, w, tok, ws=small), lambda: f(x, w, tok, status=l), lambda: f(x.t(), w.t()), lambda: f(x, None, tok),
           lambda: d(x, w, tok, None), lambda: d(x, w, tok, l[:3]), lambda: d(x, w, tok, l.double()),
           lambda: d(x, w, tok, l, None, l, l), lambda: d(x, w, tok, l, l, l[:3]), lambda: d(x, w, tok, l, l, l, scale=math.nan),
           lambda: d(x, w, tok, l, dw_dtype=F16), lambda: d(x, w, tok, l, dx=l), lambda: d(x, w, tok, l, dw=w[:31].clone()),
           lambda: d(x, w, tok, l, ws=small), lambda: d(x.to(E4M3), w.to(E4M3), tok, l), lambda: d(x, w[:0], tok, l)]
    for call in bad:
        with pytest.raises(ecc.EccError) as e:
            call()
        assert e.value.code == ecc.ERR_ARG
