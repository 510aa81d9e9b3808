// ecc_gated_gemm.cu -- the matrix products' kernels for the gated
// feed-forward projections: both projections with their product, and the
// backward product over both weights.

#include "ecc_gemm.cuh"

namespace ecc {

const void *gated_kernel(bool f8, bool pair)
{
    return f8 ? gemm_kernel<false, false, true, kGated>(pair) : gemm_kernel<false, false, false, kGated>(pair);
}
const void *dual_kernel(bool pair) { return gemm_kernel<true, false, false, kDual>(pair); }
const void *dual_both_kernel() { return (const void *)gemm_both_kernel<kDual>; }

} // namespace ecc
