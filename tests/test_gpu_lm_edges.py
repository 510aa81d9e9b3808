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
