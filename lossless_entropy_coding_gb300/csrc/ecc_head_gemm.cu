// ecc_head_gemm.cu -- the matrix products' kernels for logits that are never
// stored: their softmax statistics, and their gradient as an operand of the
// backward products.

#include "ecc_gemm.cuh"

namespace ecc {

const void *stats_kernel(bool f8, bool pair)
{
    return f8 ? gemm_kernel<false, false, true, kStats>(pair) : gemm_kernel<false, false, false, kStats>(pair);
}
const void *slopes_kernel(bool pair) { return gemm_kernel<false, false, false, kSlopes>(pair); }

} // namespace ecc
