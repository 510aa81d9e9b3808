"""Results of short reductions leave the products' pair kernel through two
stages of shared memory a warp.  A stage may only be written again once the
copies from it have read it, also where a tile ends after an odd number of 32
rows (1 to 32 rows, or 65 to 96, in one of its halves of 128) and the warp
goes on with another tile: the rows below leave one or three such chunks, and
there are more tiles than pairs of CTAs.  The same values into rows off
16-byte boundaries go past the stages: they have to agree to the bit, each
time.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_gated as gated  # noqa: E402
import test_gpu_head as head  # noqa: E402
import test_gpu_linear as linear  # noqa: E402

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
REPEATS = 12


def off_boundaries(rows, cols, dtype):
    return torch.zeros(rows, cols + 1 + cols % 2, dtype=dtype, device="cuda")[:, 1:cols + 1]


# rows modulo 256: 32 and 80 (one and three chunks in the first half), 160 and 208 (in the second), 202
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(2336, 16384, 64), (2128, 16384, 64), (2208, 16384, 1024), (2000, 16384, 512), (2250, 20000, 264),
                                   (1090, 40000, 192)])
def test_plain_results(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    x, w, bias = linear.rows_of(gen, M, K, BF16), linear.rows_of(gen, N, K, BF16), linear.rows_of(gen, 1, N, F32)[0]
    args = dict(bias=bias, act="silu", scale=1 / math.sqrt(K))
    want = linear.check(x, w, bias, None, "silu", 1 / math.sqrt(K), dtype)
    past = off_boundaries(M, N, dtype)
    ecc.ecc_linear(x, w, out=past, **args)
    assert torch.equal(past, want)
    outs = [torch.empty_like(want) for _ in range(REPEATS)]
    for out in outs:
        ecc.ecc_linear(x, w, out=out, **args)
    assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("M,N,K", [(64, 16416, 4096), (1000, 8288, 4096)])
def test_weight_gradients(M, N, K):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    x, w, dy = linear.rows_of(gen, M, K, BF16), linear.rows_of(gen, N, K, BF16), linear.rows_of(gen, M, N, BF16)
    past = off_boundaries(N, K, BF16)
    ecc.ecc_linear_grad(dy, x, w, dw=past, want=())
    ref = dy.double().T @ x.double()
    sums = dy.double().abs().T @ x.double().abs()
    assert bool(((past.double() - ref).abs() <= 1.01 * 2.0**-8 * ref.abs() + (M + 8) * 2.0**-23 * sums).all())
    outs = [torch.empty(N, K, dtype=BF16, device="cuda") for _ in range(REPEATS)]
    for out in outs:
        ecc.ecc_linear_grad(dy, x, w, dw=out, want=())
    assert all(torch.equal(out, past) for out in outs)


@pytest.mark.parametrize("out_dtype,pre_dtype", [(BF16, BF16), (E4M3, F16), (F32, BF16)])
@pytest.mark.parametrize("M,N,K", [(2080, 8192, 64), (2128, 8208, 712), (2208, 8208, 264), (2250, 8208, 1024)])
def test_gated_results(M, N, K, out_dtype, pre_dtype):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    x, wg, wu = (gated.rows_of(gen, r, K, BF16) for r in (M, N, N))
    args = dict(act="silu", scale=1 / math.sqrt(K), out_scale=8.0 if out_dtype == E4M3 else 1.0)
    want = gated.check(x, wg, wu, act="silu", scale=args["scale"], out_dtype=out_dtype, out_scale=args["out_scale"], pre_dtype=pre_dtype)
    past = [off_boundaries(M, N, t) for t in (out_dtype, pre_dtype, pre_dtype)]
    ecc.ecc_gated_linear(x, wg, wu, out=past[0], pre_gate=past[1], pre_up=past[2], **args)
    assert torch.equal(past[0].float(), want.float())
    sets = [[torch.empty(M, N, dtype=t, device="cuda") for t in (out_dtype, pre_dtype, pre_dtype)] for _ in range(REPEATS)]
    for out, g, u in sets:
        ecc.ecc_gated_linear(x, wg, wu, out=out, pre_gate=g, pre_up=u, **args)
    assert all(torch.equal(a.float(), b.float()) for s in sets for a, b in zip(s, past))


# (the logits' gradient of 1 x 32 rows and more of the vocabulary in the last tile; small heads, a hidden size of 1024)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,V,K", [(4000, 6432, 256), (2500, 12704, 64), (3000, 8224, 512), (2500, 12752, 1024), (64, 16416, 4096)])
def test_logits_gradients(M, V, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + V + K)
    x, w, tok = head.rows_of(gen, M, K, dtype), head.rows_of(gen, V, K, dtype, std=K**-0.5), head.tokens_of(gen, M, V)
    tok[:4] = torch.tensor([V - 1, V - 32, V - 33, V - 64])
    dlp = torch.randn(M, generator=gen, device="cuda")
    dx, dw = head.check_grad(x, w, tok, 1.5, dlp)
    lse = torch.logsumexp(1.5 * (x.double() @ w.double().T), -1).float()
    sets = [ecc.ecc_linear_logprob_grad(x, w, tok, lse, None, dlp, scale=1.5) for _ in range(REPEATS)]
    assert all(torch.equal(a, dx) and torch.equal(b, dw) for a, b, _ in sets)
