"""The language-model operators at the ends of their ranges: arguments and
logits that are huge, infinite or NaN, rows of many equal logits, batches
without rows, arguments by name."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
from test_gpu_linear import ACTS, check_grad as check_linear_grad, rows_of  # noqa: E402
from test_gpu_logprob import U, as_passed, error_of, reference  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = math.inf


# ---------------------------------------------------------------- linear layer
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("pre_dtype", [F32, BF16])
def test_slopes_at_large_arguments(act, pre_dtype):
    """A finite argument of any size has a finite slope (beyond the curves' bends it is 0 or 1)."""
    gen = torch.Generator("cuda").manual_seed(1)
    far = [1e4, 1e9, 1.1e13, 1.2e13, 3e15, 1e19, 2e19, 1e25, 3e38]
    far = torch.tensor([0.0, 5.0, -5.0] + far + [-v for v in far], device="cuda")
    N = far.numel()
    for M in (3, 130):
        dy, x, w = rows_of(gen, M, N, BF16), rows_of(gen, M, 40, BF16), rows_of(gen, N, 40, BF16)
        pre = far.expand(M, N).contiguous().to(pre_dtype)
        dx, dw, db = check_linear_grad(dy, x, w, pre, act)
        assert bool(dx.isfinite().all()) and bool(dw.isfinite().all()) and bool(db.isfinite().all())


# ---------------------------------------------------------------- log probabilities
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [50, 9001, 40003])
def test_gradient_of_rows_without_a_number_is_nan(V, dtype):
    """Rows with a NaN or +infinity, the token at the row's start, middle and end, on the logits' boundary and another."""
    rows = 9
    x = torch.randn(rows, V + 5, generator=torch.Generator("cuda").manual_seed(V), device="cuda").to(dtype)[:, :V]
    tok = torch.tensor([0, 1, V // 2, V - 1, V // 2 + 1, 3, -1, V - 1, 5], device="cuda")
    clean = [1, 7]
    x[0, 5], x[2, V // 2], x[3, 0], x[4, V - 1], x[5, 3] = math.nan, math.nan, math.nan, INF, INF
    x[6, 7], x[8, 0], x[8, 1] = math.nan, INF, math.nan
    r = ecc.ecc_token_logprob(x, tok)
    one, half = torch.ones(rows, device="cuda"), torch.full((rows,), 0.5, device="cuda")
    for off in (0, 1, 3):
        out = torch.empty(rows * (V + 5) + 8, dtype=dtype, device="cuda")[off:off + rows * (V + 5)].view(rows, V + 5)[:, :V]
        for dlp, dent in ((one, None), (one, half), (None, half)):
            d = ecc.ecc_token_logprob_grad(x, tok, r.lse, r.entropy, dlp, dent, dlogits=out)
            bad = [i for i in range(rows) if i not in clean]
            assert bool(d[bad].isnan().all())
            c = ecc.ecc_token_logprob_grad(x[clean], tok[clean], r.lse[clean], r.entropy[clean],
                                           None if dlp is None else dlp[clean], None if dent is None else dent[clean])
            assert bool(d[clean].isfinite().all()) and torch.allclose(d[clean].float(), c.float(), rtol=1e-2, atol=1e-5)


def order_of(x, top):
    """NaN first, then larger logits, equal ones by the lower index."""
    key = torch.where(x.isnan(), 2.0, 1.0).double()
    v = torch.where(x.isnan(), 0.0, x.double() + 0.0)
    by_value = torch.sort(v, dim=-1, descending=True, stable=True).indices
    by_nan = torch.sort(key.gather(1, by_value), dim=-1, descending=True, stable=True).indices
    return by_value.gather(1, by_nan)[:, :top]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,V", [(7, 40), (5, 2000), (1300, 3001), (3, 60000), (400, 20011), (2, 131072)])
def test_alternatives_among_many_candidates(rows, V, dtype):
    """More values at the bound than are ranked at a time: NaN, constants, few levels, ascending runs, plateaus."""
    gen = torch.Generator("cuda").manual_seed(rows + V)
    top = 32
    at = torch.arange(V, device="cuda")
    kinds = [torch.full((V,), math.nan, device="cuda"), torch.zeros(V, device="cuda"),
             torch.randint(0, 3, (V,), generator=gen, device="cuda").float(),
             torch.where(at % 2 == 0, math.nan, 1.0), torch.where(at == 0, math.nan, 4.0),
             torch.where(at < 20, -INF, 2.5), (at // 700).float(), torch.where((at >= 17) & (at < 1500), at * 2.0 ** -12 + 1, 0.0),
             torch.where(at % 3 == 1, -INF, -0.0), torch.where(at == V - 1, 7.0, -3.0)]
    z = torch.stack([kinds[r % len(kinds)].roll((r // len(kinds)) * 37) for r in range(rows)]).to(dtype)
    pad = torch.full((rows, V + 3), 9.0, device="cuda", dtype=dtype)
    pad[:, :V] = z
    want = order_of(z.float(), top)
    for x in (z, pad[:, :V]):
        r = ecc.ecc_token_logprob(x, None, top=top)
        assert torch.equal(r.top_index.long(), want)
        has = ~z.float().isnan().any(-1)
        assert bool(r.top_logprob[~has].isnan().all()) and bool(r.lse[has].isfinite().all())
        if bool(has.any()):
            logp = reference(z[has])[2].gather(1, want[has])
            assert torch.allclose(r.top_logprob[has].double(), logp, rtol=1e-5, atol=float(error_of(V)) + 1e-5)


def test_rows_of_equal_logits_keep_up():
    """The alternatives of a constant row (a head that starts at zero) cost a pass over it, not one for each of them."""
    x = torch.randn(1000, 50021, device="cuda")
    flat = torch.zeros_like(x)

    def ms(z):
        best = INF
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ecc.ecc_token_logprob(z, None, top=32)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    usual, equal = ms(x), ms(flat)
    assert equal < 20 * usual, (usual, equal)


@pytest.mark.parametrize("dtype,scale", [(F32, 1.4), (BF16, 1.4), (BF16, 3.0), (F16, 1e34)])
@pytest.mark.parametrize("V", [40, 5000, 131073])
def test_logits_whose_scaled_values_leave_float32(V, dtype, scale):
    """scale * logits past float32's range: lse is infinite there, the probabilities are what they are."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.randn(6, V, generator=torch.Generator("cuda").manual_seed(V), device="cuda").to(dtype)
    x[0] = low                               # a mask that left nothing, by the type's lowest value
    x[1] = low
    x[1, ::3] = -INF
    x[2] = high
    x[3, 3], x[3, 9] = high, high
    x[4] = -INF
    tok = torch.tensor([1, 2, V - 1, 9, 0, 5], device="cuda")
    top = 5
    r = ecc.ecc_token_logprob(x, tok, top=top, scale=scale)
    s = as_passed(scale)
    lse, ent, logp, p = reference(x.double() * s)
    e = error_of(V) * (math.log(V + 1) + 40)
    assert r.lse[:5].tolist() == [-INF, -INF, INF, INF, -INF]
    want = order_of(x.float(), top)
    assert torch.equal(r.top_index.long(), want)
    for got, ref in ((r.entropy[:4], ent[:4]), (r.logprob[:4], logp.gather(1, tok[:, None])[:4, 0]),
                     (r.top_logprob[:4], logp.gather(1, want)[:4])):
        ref = ref.float().double()           # (a logarithm below float32's range is -infinity there)
        assert bool(((got.double() == ref) | ((got.double() - ref).abs() <= e)).all())
    assert float(r.entropy[4]) == 0 and float(r.logprob[4]) == -INF
    if dtype == F16:                         # (its gradient is as large as the scale)
        return
    one, half = torch.ones(6, device="cuda"), torch.full((6,), 0.5, device="cuda")
    hot = torch.zeros_like(p).scatter_(1, tok[:, None], 1.0)
    mid = torch.where(p > 0, p * (logp + ent[:, None]), 0.0)
    for dent in (None, half):
        for out in (None, x.clone()):        # also in place
            d = ecc.ecc_token_logprob_grad(x if out is None else out, tok, r.lse, r.entropy, one, dent, scale=scale, dlogits=out)
            ref = s * (hot - p - (0.0 if dent is None else 0.5) * mid)
            assert not d[4].any()
            assert bool(((d.double() - ref).abs()[:4] <= 1.01 * U[dtype] * ref.abs()[:4] + 4 * s * error_of(V)).all())


# ---------------------------------------------------------------- the calls
def test_batches_without_rows():
    def e(*s, dtype=BF16):
        return torch.empty(*s, dtype=dtype, device="cuda")

    w, stat = torch.randn(24, 16, device="cuda").to(BF16), e(2, 0, 3, dtype=F32)
    for lead in ((2, 0, 3), (2, 0), (0, 2), (3, 1, 0)):
        stat = e(*lead, dtype=F32)
        y, mean, rstd = ecc.ecc_layer_norm(e(*lead, 16))
        assert y.shape == (*lead, 16) and mean.shape == lead and rstd.shape == lead
        dx, dweight, dbias = ecc.ecc_layer_norm_grad(e(*lead, 16), e(*lead, 16), None, stat, stat)
        assert dx.shape == (*lead, 16) and not dweight.any() and not dbias.any()
        y, st = ecc.ecc_linear(e(*lead, 16), w, residual=e(*lead, 24), pre=e(*lead, 24))
        assert y.shape == (*lead, 24) and int(st.item()) == 0
        dx, dw, db, st = ecc.ecc_linear_grad(e(*lead, 24), e(*lead, 16), w, e(*lead, 24), act="gelu")
        assert dx.shape == (*lead, 16) and not dw.any() and not db.any() and int(st.item()) == 0
        r = ecc.ecc_token_logprob(e(*lead, 50), e(*lead, dtype=torch.int64), top=4)
        assert r.lse.shape == lead and r.top_index.shape == (*lead, 4)
        d = ecc.ecc_token_logprob_grad(e(*lead, 50), e(*lead, dtype=torch.int64), stat, None, stat)
        assert d.shape == (*lead, 50)


def test_arguments_by_name():
    gen = torch.Generator("cuda").manual_seed(2)
    x, dy, w = rows_of(gen, 8, 64, BF16), rows_of(gen, 8, 32, BF16), rows_of(gen, 32, 64, BF16)
    tok = torch.arange(8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def same(a, b):
        torch.cuda.synchronize()
        return all(p is q or torch.equal(p, q) for p, q in zip(a, b))

    y, mean, rstd = ref = ecc.ecc_layer_norm(x)
    r = ecc.ecc_token_logprob(x, tok)
    for kw in ({}, {"stream": s}):
        assert same(ecc.ecc_layer_norm(x=x, **kw), ref)
        assert same(ecc.ecc_layer_norm_grad(dy=y, x=x, weight=None, mean=mean, rstd=rstd, **kw),
                    ecc.ecc_layer_norm_grad(y, x, None, mean, rstd))
        assert same(ecc.ecc_layer_norm_grad(y, x=x, weight=None, mean=mean, rstd=rstd, **kw),
                    ecc.ecc_layer_norm_grad(y, x, None, mean, rstd))
        assert same(ecc.ecc_linear(x=x, w=w, **kw), ecc.ecc_linear(x, w))
        assert same(ecc.ecc_linear_grad(dy=dy, x=x, w=w, **kw), ecc.ecc_linear_grad(dy, x, w))
        assert same(ecc.ecc_token_logprob(logits=x, tokens=tok, **kw), r)
        assert same([ecc.ecc_token_logprob_grad(logits=x, tokens=tok, lse=r.lse, dlogprob=mean, **kw)],
                    [ecc.ecc_token_logprob_grad(x, tok, r.lse, None, mean)])


def test_scratch_of_the_caller():
    """A given workspace is the device's, in one piece and long enough, or the call is refused."""
    gen = torch.Generator("cuda").manual_seed(3)
    x, dy, w = rows_of(gen, 30, 64, BF16, 5), rows_of(gen, 30, 40, BF16, 5), rows_of(gen, 40, 64, BF16, 5)   # copied to ws
    y, mean, rstd = ecc.ecc_layer_norm(x)
    calls = [lambda ws: ecc.ecc_layer_norm_grad(x, x, None, mean, rstd, ws=ws), lambda ws: ecc.ecc_linear(x, w, ws=ws),
             lambda ws: ecc.ecc_linear_grad(dy, x, w, dy, act="gelu", ws=ws)]
    for call in calls:
        ref = call(None)
        for ws in (torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.empty(64, 4096, device="cuda")):
            got = call(ws)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.uint8).pin_memory(),
                   torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20),
                   torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2],
                   torch.empty(1024, 1024, device="cuda").t(), torch.empty(16, dtype=torch.uint8, device="cuda"),
                   torch.empty((1 << 20) + 8, dtype=torch.uint8, device="cuda")[8:]):
            with pytest.raises(ecc.EccError) as e:
                call(ws)
            assert e.value.code == ecc.ERR_ARG


def test_memory_that_is_not_there():
    """An output that does not fit raises what torch raises for its own."""
    x = torch.zeros(1 << 20, 8, device="cuda", dtype=BF16)
    with pytest.raises(torch.OutOfMemoryError):
        ecc.ecc_linear(x, x)
    y, st = ecc.ecc_linear(x[:16], x[:24])
    assert int(st.item()) == 0 and not y.any()
