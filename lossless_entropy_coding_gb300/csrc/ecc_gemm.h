// ecc_gemm.h -- the matrix product the linear operators are made of.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ecc_lm.h"

namespace ecc {

// What a kernel makes of its products (ecc_gemm.cuh)
enum GemmMode { kPlain, kGated, kDual, kStats, kSlopes };

// out[r, c] = act(scale * sum over k of Q[r, k] P[c, k] + bias[c]) + residual[r, c]
struct Epilogue {
    const void *bias, *residual;
    void *out, *pre;
    uint64_t ldres, ldout, ldpre;
    float scale, out_scale;
    uint32_t bias_type, res_type, out_type, pre_type, act;
    // gated products: act(scale * sum + bias) * (scale2 * sum2 + bias2); pre2 beside pre
    const void *bias2;
    void *pre2;
    uint64_t ldpre2;
    float scale2;
    bool swapped; // the ups' rows come before the gates' in each turn
    // a second output: rows from rswitch on (a multiple of 64, of 128 where the
    // scales differ) go to out2, by scale2, and both have rows2 rows
    void *out2;
    uint64_t ldout2, rswitch, rows2;
    const float *factor; // multiplies scale (read on the device; a second output's scale2: the next one); NULL: 1
    // logits, never stored: columns are tokens, rows the vocabulary from `first` on
    const int64_t *tokens;
    uint64_t first;
    float4 *part;       // kStats: [share of the vocabulary][token]: maximum, sum, entropy sum (base 2)
    float *token_logit; // kStats: [token], scaled by log2 e
    // kSlopes, of each token; dlogprob and dentropy may be NULL; out: [token][vocabulary] of out_type
    const float *lse, *entropy, *dlogprob, *dentropy;
    uint64_t vocab;
};

// An operand: `rows` x K values, either stored a matrix row after the other
// (mn = false: the reduction is contiguous) or a reduction index after the
// other (mn = true).  16-byte aligned rows.
struct Operand {
    const void *p;
    uint64_t ld;
    bool mn;
};

// whether an array of `rows` rows can be read by tiled TMA as it is
bool tma_rows(const void *p, uint64_t ld, uint32_t type, uint64_t rows);
// rows x cols values from a reduction of K; P holds the output's columns, Q its rows
// (kGated: P and P2 hold the columns' gates and ups;
// kDual: the reduction's indices from kswitch on, a multiple of 64, are
// P2's; both have kfirst of them)
struct Product {
    Operand P, Q;
    uint64_t rows, cols, K;
    Epilogue e;
    GemmMode mode = kPlain;
    Operand P2{};
    uint64_t kswitch = 0, kfirst = 0;
};
// clear_status: the launch sets *status to ECC_OK; behind: the stream's last
// launch is one of the same call's that lets this one start early
ecc_status gemm(const Product &x, uint32_t type, uint32_t *status, bool clear_status, bool behind, cudaStream_t st);
// a layer's two backward products: dx with Q along its rows, dw with both
// operands down their columns (16-bit types)
ecc_status gemm_backward(const Product &dx, const Product &dw, uint32_t type, uint32_t *status, bool clear_status, bool behind,
                         cudaStream_t st);

// kernels that are built apart
const void *gated_kernel(bool f8, bool pair);
const void *dual_kernel(bool pair);
const void *dual_both_kernel();
const void *stats_kernel(bool f8, bool pair);
const void *slopes_kernel(bool pair);
const void *stats_stream(bool f8);
// shares of the vocabulary that a kStats product writes parts for
uint32_t stats_parts(const Product &x, uint32_t type);

} // namespace ecc
