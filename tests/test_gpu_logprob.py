"""ecc_token_logprob and its gradient against a plain 64-bit computation.

Tolerances.  A float32 sum of n terms over at least 32 lanes is off by at most
g = (n / 32 + 16) 2^-24 of the terms' magnitudes, an exponential by a relative
2^-21 + 2^-23 |argument| (its argument is rounded); so log s is off by
e = g + 2^-20 + 2^-23 Z, Z the row's span of finite z that matters (an
exponential of less than -100 is nothing), and lse by e + 2^-22 |lse|.
The entropy is an average of terms of at most log V + 40 with that error.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}
TINY = {F32: 2.0**-149, BF16: 2.0**-133, F16: 2.0**-25}
INF = math.inf


def logits_of(gen, rows, vocab, dtype, pad=0, off=0, std=2.5):
    base = torch.randn(rows * (vocab + pad) + off, generator=gen, device="cuda") * std
    return base.to(dtype)[off:].view(rows, vocab + pad)[:, :vocab]


def reference(z):
    """lse, entropy, log p in 64 bits of z [rows, vocab]; rows without a probability: -inf, 0, -inf."""
    z = z.double()
    m = z.amax(-1, keepdim=True)
    empty = m == -INF
    d = torch.where(empty, torch.zeros_like(z), z - torch.where(empty, 0.0, m))
    e = torch.where(empty, torch.zeros_like(z), d.exp())
    s = e.sum(-1, keepdim=True)
    logs = torch.where(empty, -INF, s.log())
    lse = torch.where(empty, -INF, m + logs)
    p = torch.where(empty, torch.zeros_like(z), e / s)
    logp = torch.where(empty, -INF, d - torch.where(empty, 0.0, logs))
    ent = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    return lse[:, 0], ent, logp, p


def error_of(V):
    return (V / 32 + 16) * 2.0**-24 + 2.0**-20 + 2.0**-23 * 100


def as_passed(scale):
    """The scale that a call receives: the C argument is a float32."""
    return float(torch.tensor(scale, dtype=F32))


def close(got, ref, tol):
    same = (got.double() == ref) | (got.isnan() & ref.isnan())
    return bool((same | ((got.double() - ref).abs() <= tol)).all())


def check(x, tok, top, scale=1.0, **kw):
    r = ecc.ecc_token_logprob(x, tok, top=top, scale=scale, **kw)
    torch.cuda.synchronize()
    scale = as_passed(scale)
    V = x.shape[-1]
    lse, ent, logp, _ = reference(x.double() * scale)
    e = error_of(V)
    tl = e + 2.0**-22 * torch.where(lse.isfinite(), lse.abs(), 0.0)
    assert close(r.lse, lse, tl)
    assert close(r.entropy, ent, e * (math.log(V + 1) + 40))
    if tok is not None:
        t = tok.clamp(min=0)[:, None]
        zt = (x.double() * scale).gather(1, t)[:, 0].abs()
        ref = torch.where(tok >= 0, logp.gather(1, t)[:, 0], 0.0)
        assert close(r.logprob, ref, tl + 2.0**-22 * torch.where(zt.isfinite(), zt, 0.0))
    if top:
        order = torch.sort(x.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(r.top_index.long(), order)
        ref = logp.gather(1, order)
        zt = (x.double() * scale).gather(1, order).abs()
        assert close(r.top_logprob, ref, tl[:, None] + 2.0**-22 * torch.where(zt.isfinite(), zt, 0.0))
    return r


SHAPES = [(1, 1), (2, 2), (3, 31), (5, 33), (2, 1000), (4, 4097), (3, 32000), (1, 50021), (2, 131072), (1, 262144),
          (400, 512), (700, 1003), (160, 10007), (33, 32768)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logprob_shapes(rows, vocab, dtype):
    gen = torch.Generator("cuda").manual_seed(rows + 3 * vocab)
    for pad, off, top, scale in ((0, 0, min(8, vocab), 1.0), (5, 3, min(32, vocab), 0.7), (8, 0, 0, 1.3),
                                 (1, 0, 1, 1.0)):
        x = logits_of(gen, rows, vocab, dtype, pad, off)
        tok = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        tok[::7] = -1
        check(x, tok, top, scale)
    check(x, None, 1)


@pytest.mark.parametrize("dtype,rows,vocab,top", [(F32, 1300, 50021, 20), (F32, 2000, 9001, 32), (BF16, 1300, 40003, 32),
                                                  (BF16, 3000, 4099, 5), (F16, 1000, 131072, 8)])
def test_logprob_many_long_rows(dtype, rows, vocab, top):
    """Several rows a block, the selection of a row slower than the next one's sums."""
    gen = torch.Generator("cuda").manual_seed(rows + vocab)
    x = logits_of(gen, rows, vocab, dtype)
    tok = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    first = check(x, tok, top, 0.7)
    for _ in range(3):
        again = ecc.ecc_token_logprob(x, tok, top=top, scale=0.7)
        assert torch.equal(again.lse, first.lse) and torch.equal(again.top_index, first.top_index)
        assert torch.equal(again.logprob, first.logprob) and torch.equal(again.entropy, first.entropy)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_logprob_masks(dtype):
    gen = torch.Generator("cuda").manual_seed(3)
    low = torch.finfo(dtype).min
    for V in (40, 5000, 131073):
        x = logits_of(gen, 9, V, dtype)
        x[0] = -INF                       # nothing left
        x[1] = low                        # everything at the lowest value: uniform
        x[2, 1:] = -INF                   # one token left, the first
        x[3, :-1] = -INF                  # ... the last
        x[4, 3:] = low
        x[5, ::2] = -INF
        x[6] = 0.0
        x[7, V // 2] = 60.0               # nearly certain
        x[8, :V - 1] = -INF
        x[8, V - 1] = low
        tok = torch.tensor([1, 2, 0, V - 1, 5, 2, 7, V // 2, V - 1], device="cuda")
        top = 32
        r = check(x, tok, top)
        assert float(r.entropy[0]) == 0 and float(r.lse[0]) == -INF and float(r.logprob[0]) == -INF
        assert float(r.logprob[5]) == -INF
        assert torch.equal(r.top_index[6].cpu(), torch.arange(top, dtype=torch.int32))   # ties by index
        assert torch.equal(r.top_index[0].cpu(), torch.arange(top, dtype=torch.int32))


def test_logprob_ties_orders_and_zeros():
    V = 70001
    x = torch.zeros(6, V, device="cuda", dtype=BF16)
    x[0] = torch.arange(V, device="cuda") % 3          # many ties
    x[1] = torch.linspace(-9, 9, V, device="cuda")     # ascending: every element displaces one
    x[2] = -x[1]
    x[3, ::2] = -0.0                                   # -0 equals +0
    x[4] = torch.randint(0, 2, (V,), device="cuda")
    x[5, -40:] = 1.0
    check(x, torch.arange(6, device="cuda"), 32)
    check(x.float(), torch.arange(6, device="cuda"), 20)


def test_logprob_non_finite():
    for V in (100, 60000):
        x = torch.randn(4, V, device="cuda")
        x[0, 50], x[1, 50] = math.nan, INF
        x[2, 7], x[2, 9] = INF, math.nan
        tok = torch.tensor([3, 3, 3, V], device="cuda")
        r = ecc.ecc_token_logprob(x, tok, top=3)
        torch.cuda.synchronize()
        assert r.lse[0].isnan() and r.entropy[0].isnan() and r.logprob[0].isnan()
        assert float(r.lse[1]) == INF and r.entropy[1].isnan() and float(r.logprob[1]) == -INF
        assert r.lse[2].isnan()
        assert r.logprob[3].isnan() and r.lse[3].isfinite()         # a token outside the vocabulary
        assert r.top_index[:3, 0].tolist() == [50, 50, 9] and int(r.top_index[2, 1]) == 7
        check(x[3:], torch.tensor([1], device="cuda"), 3)


def check_grad(x, tok, dlp, dent, scale, **kw):
    r = ecc.ecc_token_logprob(x, tok, scale=scale)
    kw["scale"], scale = scale, as_passed(scale)
    ref_lse, ref_ent, logp, p = reference(x.double() * scale)
    d = ecc.ecc_token_logprob_grad(x, tok, r.lse, r.entropy, dlp, dent, **kw)
    torch.cuda.synchronize()
    V = x.shape[-1]
    alive = (ref_lse > -INF)[:, None]
    a = torch.zeros_like(ref_lse) if dlp is None else torch.where(tok >= 0, dlp.double(), 0.0)
    b = torch.zeros_like(ref_lse) if dent is None else dent.double()
    one = torch.zeros_like(p)
    if tok is not None:
        one.scatter_(1, tok.clamp(min=0)[:, None], (tok >= 0).double()[:, None])
    mid = torch.where(p > 0, p * (logp + ref_ent[:, None]), 0.0)
    ref = torch.where(alive, scale * (a[:, None] * (one - p) - b[:, None] * mid), 0.0)
    e = 4 * error_of(V) + 2.0**-20 * (1 + torch.where(ref_lse.isfinite(), ref_lse.abs(), 0.0)[:, None])
    absl = torch.where(p > 0, logp.abs() + ref_ent[:, None] + math.log(V + 1) + 40, 0.0)
    slack = scale * e * (a.abs()[:, None] * (p + 2.0**-20 * one) + b.abs()[:, None] * p * (absl + 1))
    # exponentials below the smallest normal number may count as nothing
    slack = slack + scale * 2.0**-126 * 200 * (a.abs() + b.abs())[:, None]
    err = (d.double() - ref).abs()
    assert bool((err <= 1.01 * U[x.dtype] * ref.abs() + TINY[x.dtype] + slack).all())
    return d


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logprob_grad_shapes(rows, vocab, dtype):
    gen = torch.Generator("cuda").manual_seed(rows + 5 * vocab)
    for pad, off, scale in ((0, 0, 1.0), (5, 3, 0.7), (8, 0, 1.3)):
        x = logits_of(gen, rows, vocab, dtype, pad, off)
        tok = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        tok[::5] = -1
        dlp = -torch.rand(rows, generator=gen, device="cuda") - 0.5
        dent = torch.randn(rows, generator=gen, device="cuda")
        ref = check_grad(x, tok, dlp, dent, scale)
        check_grad(x, tok, dlp, None, scale)
        check_grad(x, None, None, dent, scale)
        r = ecc.ecc_token_logprob(x, tok, scale=scale)
        y = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda").copy_(x)
        ecc.ecc_token_logprob_grad(y, tok, r.lse, r.entropy, dlp, dent, scale=scale, dlogits=y)
        assert torch.equal(y, ref)       # in place


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logprob_grad_masks(dtype):
    gen = torch.Generator("cuda").manual_seed(4)
    V = 9001
    x = logits_of(gen, 5, V, dtype)
    x[0] = -INF
    x[1] = torch.finfo(dtype).min
    x[2, 5:] = -INF
    x[3, V // 2] = 60.0
    tok = torch.tensor([1, 2, 3, 4, V], device="cuda")
    one = torch.ones(5, device="cuda")
    r = ecc.ecc_token_logprob(x, tok)
    d = ecc.ecc_token_logprob_grad(x, tok, r.lse, r.entropy, one, one)
    torch.cuda.synchronize()
    assert bool(d.isfinite().all()) and not d[0].any() and not d[2, 5:].any()
    check_grad(x[:4], tok[:4], one[:4], one[:4], 1.0)
    # a token outside the vocabulary takes no part
    e = ecc.ecc_token_logprob_grad(x[4:], tok[4:], r.lse[4:], None, one[4:], None)
    assert not e.any()


def test_logprob_grad_against_differences():
    gen = torch.Generator("cuda").manual_seed(8)
    x = logits_of(gen, 4, 50, F32, std=1.0)
    tok = torch.tensor([3, 49, -1, 0], device="cuda")
    dlp, dent, scale = torch.randn(4, device="cuda"), torch.randn(4, device="cuda"), 0.8
    r = ecc.ecc_token_logprob(x, tok, scale=scale)
    d = ecc.ecc_token_logprob_grad(x, tok, r.lse, r.entropy, dlp, dent, scale=scale)

    def loss(x):
        _, ent, logp, _ = reference(x * scale)
        lp = torch.where(tok >= 0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0], 0.0)
        return float((lp * dlp + ent * dent).sum())

    h = 1e-4
    for k in range(20):
        i, j = k % 4, (7 * k) % 50 if k % 3 else max(0, int(tok[k % 4]))
        e = torch.zeros(4, 50, dtype=torch.float64, device="cuda")
        e[i, j] = h
        diff = (loss(x.double() + e) - loss(x.double() - e)) / (2 * h)
        assert abs(diff - float(d[i, j])) < 1e-5


def test_logprob_offsets_past_32_bits_streams_and_empty():
    buf = torch.zeros((1 << 32) + 70000, dtype=BF16, device="cuda")
    x = buf.as_strided((3, 33333), ((1 << 31) + 8, 1))
    x.copy_(torch.randn(3, 33333, device="cuda"))
    tok = torch.tensor([5, 33332, 0], device="cuda")
    ref = check(x, tok, 5)
    one = torch.ones(3, device="cuda")
    check_grad(x.contiguous(), tok, one, one, 1.0)
    dref = ecc.ecc_token_logprob_grad(x.contiguous(), tok, ref.lse, ref.entropy, one, one)
    d = ecc.ecc_token_logprob_grad(x, tok, ref.lse, ref.entropy, one, one)
    assert torch.equal(d, dref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = ecc.ecc_token_logprob(x, tok, top=5, stream=s)
    d = ecc.ecc_token_logprob_grad(x, tok, r.lse, r.entropy, one, one, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r.logprob, ref.logprob) and torch.equal(r.top_index, ref.top_index) and torch.equal(d, dref)
    r = ecc.ecc_token_logprob(torch.empty(0, 7, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=2)
    assert r.lse.shape == (0,) and r.top_index.shape == (0, 2)


def test_logprob_refusals():
    x = torch.randn(4, 64, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [lambda: ecc.ecc_token_logprob(x.double(), tok), lambda: ecc.ecc_token_logprob(x, tok.int()),
           lambda: ecc.ecc_token_logprob(x, tok[:3]), lambda: ecc.ecc_token_logprob(x, tok, top=33),
           lambda: ecc.ecc_token_logprob(x[:, :5], tok, top=6), lambda: ecc.ecc_token_logprob(x, tok, top=-1),
           lambda: ecc.ecc_token_logprob(x, tok, scale=0.0), lambda: ecc.ecc_token_logprob(x, tok, scale=-1.0),
           lambda: ecc.ecc_token_logprob(x, tok, scale=math.inf), lambda: ecc.ecc_token_logprob(x.t(), tok),
           lambda: ecc.ecc_token_logprob(x.cpu(), tok), lambda: ecc.ecc_token_logprob(x[:, :0], tok),
           lambda: ecc.ecc_token_logprob(x[:1].expand(4, 64), tok),
           lambda: ecc.ecc_token_logprob_grad(x, None, x[:, 0].contiguous(), None, x[:, 0].contiguous()),
           lambda: ecc.ecc_token_logprob_grad(x, tok, x[:, 0].contiguous(), None, None, x[:, 0].contiguous()),
           lambda: ecc.ecc_token_logprob_grad(x, tok, None, None, x[:, 0].contiguous()),
           lambda: ecc.ecc_token_logprob_grad(x, tok, x[:, 0], None),
           lambda: ecc.ecc_token_logprob_grad(x, tok, x[:, 0].contiguous(), None, dlogits=x.half())]
    for call in bad:
        with pytest.raises(ecc.EccError) as e:
            call()
        assert e.value.code == ecc.ERR_ARG
