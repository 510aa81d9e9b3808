"""Products of more tiles than the GPU has pairs of SMs, in every operand
layout: a pair of CTAs works on several 256-column tiles one after the other,
with two accumulators in turn, ragged tiles at the ends of rows, columns and
the reduction."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_linear import BF16, E4M3, F16, F32, check, check_grad, rows_of  # noqa: E402


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,N,K", [(2600, 5000, 200), (2603, 5001, 1032), (1300, 4100, 100), (700, 20000, 1100)])
def test_linear_many_tiles(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    s, p_dtype = 1 / math.sqrt(K), BF16 if dtype == E4M3 else dtype
    for pad in (0, 5):
        x, w = rows_of(gen, M, K, dtype, pad), rows_of(gen, N, K, dtype, pad)
        bias, res = rows_of(gen, 1, N, p_dtype)[0], rows_of(gen, M, N, p_dtype, pad)
        check(x, w, bias, res, "gelu", s, pre_dtype=p_dtype)
    check(x, w, None, res.float(), "none", s, out_dtype=F32)
    check(x, w, bias.float(), None, "silu", s, out_dtype=E4M3, out_scale=8.0, pre_dtype=F32)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K", [(3000, 6000, 2100), (2100, 5200, 4104), (4101, 3001, 5007)])
def test_linear_grad_many_tiles(M, N, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    x, w = rows_of(gen, M, K, dtype), rows_of(gen, N, K, dtype, std=1 / math.sqrt(N))
    dy, pre = rows_of(gen, M, N, dtype), rows_of(gen, M, N, dtype)
    check_grad(dy, x, w, pre, "gelu")
    check_grad(dy, x, w, None, "none", 0.5, dw_dtype=F32)
