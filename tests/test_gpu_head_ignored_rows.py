"""The gradient of the log probabilities of hidden states with rows that take
no part in dlogprob: what dlogprob holds there must change nothing, neither a
float16 operand's power of two nor anything else; so too for a row whose own
gradient is not finite, as far as the other rows' dx goes.  The comparison is
with zeros in those places, to the bit."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_head as head  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
CASES = [(40, 600, 72), (70, 3001, 321), (2100, 1300, 64)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("filler", [1e30, 3e38, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("M,V,K", CASES)
def test_ignored_tokens(M, V, K, filler, dtype):
    gen = torch.Generator("cuda").manual_seed(M)
    x, w = head.rows_of(gen, M, K, dtype), head.rows_of(gen, V, K, dtype, std=0.1)
    tok = head.tokens_of(gen, M, V)
    tok[3], tok[7], tok[M - 1] = V, 1 << 40, -1
    ignored = (tok < 0) | (tok >= V)
    dlp = torch.randn(M, generator=gen, device="cuda") * 1e-5 / M
    dh = torch.randn(M, generator=gen, device="cuda") * 1e-6 / M
    zeros, filled = torch.where(ignored, 0.0, dlp), torch.where(ignored, filler, dlp)
    r = ecc.ecc_linear_logprob(x, w, tok)
    for entropy, dentropy in ((None, None), (r.entropy, dh)):
        want = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, entropy, zeros, dentropy, dw_dtype=torch.float32)
        got = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, entropy, filled, dentropy, dw_dtype=torch.float32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool(want[1].any())
        assert bool(torch.isfinite(got[0]).all()) and bool(torch.isfinite(got[1]).all())
    # no tokens at all: dlogprob takes no part (dw in float32: it is below 40 * 4e-6 / M * max p |log p + H| |x|, about
    # 1e-8 for V = 600, where float16's smallest step is 6e-8)
    f32 = dict(dw_dtype=torch.float32)
    want = ecc.ecc_linear_logprob_grad(x, w, None, r.lse, r.entropy, None, dh, **f32)
    got = ecc.ecc_linear_logprob_grad(x, w, None, r.lse, r.entropy, torch.full_like(dlp, filler), dh, **f32)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(want[1].any())


@pytest.mark.parametrize("M,V,K", CASES)
def test_a_row_that_is_not_finite_leaves_the_others_dx(M, V, K):
    gen = torch.Generator("cuda").manual_seed(M)
    x, w = head.rows_of(gen, M, K, F16), head.rows_of(gen, V, K, F16, std=0.1)
    tok = torch.randint(0, V, (M,), generator=gen, device="cuda")
    dlp = torch.randn(M, generator=gen, device="cuda") * 0.1
    dlp[5] = 0
    r = ecc.ecc_linear_logprob(x, w, tok)
    want = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, dlp, want=("dx",))[0]
    others = torch.arange(M, device="cuda") != 5
    for bad in (math.inf, math.nan):
        dlp[5] = bad
        got = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, dlp, want=("dx",))[0]
        assert torch.equal(got[others], want[others]) and not bool(torch.isfinite(got[5]).all())


@pytest.mark.parametrize("size", [-100, -66, -13, 13, 99, 120])
def test_gradients_of_any_size(size):
    """float16 operands, float32 weight gradients: the same bits, but for a power of two, whatever dlogprob's size."""
    gen = torch.Generator("cuda").manual_seed(2)
    M, V, K = 70, 900, 72
    x, w, tok = head.rows_of(gen, M, K, F16), head.rows_of(gen, V, K, F16, std=0.1), head.tokens_of(gen, M, V)
    dlp = torch.randn(M, generator=gen, device="cuda")
    r = ecc.ecc_linear_logprob(x, w, tok)
    want = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, dlp, dw_dtype=torch.float32, want=("dw",))[1]
    got = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, dlp * 2.0**size, dw_dtype=torch.float32, want=("dw",))[1]
    # (values below float32's smallest normal one, which size -100 may reach, are rounded)
    assert bool(((got.double() - want.double() * 2.0**size).abs() <= 2.0**-150).all()) and bool(want.any())
