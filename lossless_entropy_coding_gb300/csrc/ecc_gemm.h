// ecc_gemm.h -- the matrix product the linear operators are made of.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ecc_lm.h"

namespace ecc {

// out[r, c] = act(scale * sum over k of Q[r, k] P[c, k] + bias[c]) + residual[r, c]
struct Epilogue {
    const void *bias, *residual;
    void *out, *pre;
    uint64_t ldres, ldout, ldpre;
    float scale, out_scale;
    uint32_t bias_type, res_type, out_type, pre_type, act;
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
struct Product {
    Operand P, Q;
    uint64_t rows, cols, K;
    Epilogue e;
};
// clear_status: the launch sets *status to ECC_OK; behind: the stream's last
// launch is one of the same call's that lets this one start early
ecc_status gemm(const Product &x, uint32_t type, uint32_t *status, bool clear_status, bool behind, cudaStream_t st);
// a layer's two backward products: dx with Q along its rows, dw with both
// operands down their columns (16-bit types)
ecc_status gemm_backward(const Product &dx, const Product &dw, uint32_t type, uint32_t *status, bool clear_status, bool behind,
                         cudaStream_t st);

} // namespace ecc
