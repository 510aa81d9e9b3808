// ecc_gemm.cuh -- the matrix products' kernels (tcgen05, operands by tiled
// TMA, accumulators in tensor memory) with their epilogues.
//
// out[r, c] = act(scale * sum_k Q[r, k] P[c, k] + bias[c]) + residual[r, c].
// P, whose rows are the output's columns, is the product's 128-row side, so
// that a lane of tensor memory is a column of the output: a warp stores 32
// neighbouring values of a row at once, whatever the rows' alignment, and a
// thread needs one bias value a tile.  The other side, Q, gives the tile's
// width: 16 for a few tokens up to 256 for a training batch.
//
// gemm_pair_kernel: pairs of CTAs (tcgen05 cta_group::2) on 256 x `bn` tiles;
// per CTA a TMA warp, a product warp (of the pair's first CTA) and four
// or eight epilogue warps.  The pairs are persistent, and the epilogue works on one
// accumulator while the products fill the other.  For many tiles.
// gemm_split_kernel: one 128 x `bn` tile a cluster of up to 8 CTAs that share
// its reduction, for few tiles: the parts are joined through distributed
// shared memory, in the order of the CTAs' ranks.  Two CTAs an SM, or one
// with twice the stages where there are no more CTAs than SMs.

#pragma once

#include "ecc_act.cuh"
#include "ecc_gemm.h"
#include "ecc_tensor.cuh"

namespace ecc {

constexpr int kSplitThreads = 192; // TMA warp, product warp, 4 epilogue warps
constexpr int kPairThreads = 320;  // 8 of them: half a tile's rows each (reductions of 1024 are shorter than an epilogue)
constexpr uint32_t kPTile = 128;  // P rows of a CTA
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kPBytes = kPTile * kTileBytes;
constexpr uint32_t kAloneSmem = 226 * 1024, kSharedSmem = 112 * 1024; // of a CTA that has an SM to itself, or half of it
constexpr uint32_t kSmemHead = 1024; // room to align the stages to 1024 bytes

// The modes:
// kPlain: the linear operators' epilogue.
// kGated: the same of two products at once, act(gate) * up.  P's rows are
// those of two matrices in turns of 16, so that a warp's lanes 0 to 15 hold
// 16 columns' gates and lanes 16 to 31 the same columns' ups: one shuffle
// brings them together, in place of shared memory and a barrier.
// kDual: kPlain, with a reduction over two matrices P, one behind the other.
// kStats, kSlopes: P's rows are hidden states and Q's are the head's, so that a
// lane has one token and a thread's 32 values are 32 logits of it: the softmax
// needs no exchange between lanes.  kStats keeps the running maximum, sum and
// entropy sum of a share of the vocabulary, kSlopes stores the gradient with
// respect to the logits as the next products' operand.

struct GemmArgs {
    Epilogue e;
    uint32_t kswitch; // kDual: the reduction block where the second matrix starts
    bool pwide, qwide; // operands down their columns: one box for all of a tile's rows
    uint32_t staged;  // bytes of a warp's 32 rows if results leave through shared memory, or 0
    uint32_t odd;     // then: whether the last tile's rows are an odd number of 32s in its first half (1), its second (2)
    bool one_box;     // kGated: P's map has both matrices, in turns of 16 rows
    uint64_t rows, cols;
    uint32_t kblocks; // reduction blocks of 128 bytes (64 reduction indices for MN-major operands)
    uint32_t ptiles, qtiles, bn, stages, idesc, split;
    uint32_t *status;
    bool clear_status;
    uint64_t limit_ns;
};

struct GemmBars {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
    uint32_t tmem;
};
// kStats: reduction blocks (512 indices of 16 bits, 1024 of 8) after which an
// accumulator is read and the sum goes on in registers: the tensor cores'
// additions truncate, and 4096 products in one accumulator leave logits a
// relative 1e-5 short (lse off by 3e-6 of itself; by segments: 4e-7).  The
// other accumulator is filled meanwhile, so the products do not wait.
constexpr uint32_t kSegment = 8;
// P's rows of a CTA that are columns of the output
template <int MODE> constexpr uint32_t kPCols = MODE == kGated ? kPTile / 2 : kPTile;

// the head streamed past a few tokens (ecc_head_gemm.cu)
constexpr int kStreamThreads = 192; // TMA warp, product warp, 4 epilogue warps
struct StreamArgs {
    Epilogue e;
    uint64_t vocab, tokens;
    uint32_t kblocks, tiles, bn, segs, stages, idesc;
    uint32_t *status;
    uint64_t limit_ns;
};
struct StreamBars {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
    uint32_t tmem;
    int32_t token[64];
};

// ---------------------------------------------------------------- epilogue
template <uint32_t ACT, int W> __device__ __forceinline__ void activate(float (&a)[W])
{
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        const float2 v = act_value2<ACT>(make_float2(a[j], a[j + 1]));
        a[j] = v.x;
        a[j + 1] = v.y;
    }
}

template <int W> __device__ __forceinline__ void activate_by(uint32_t act, float (&a)[W])
{
    if (act == ECC_ACT_RELU)
        activate<ECC_ACT_RELU>(a);
    else if (act == ECC_ACT_GELU)
        activate<ECC_ACT_GELU>(a);
    else if (act == ECC_ACT_GELU_TANH)
        activate<ECC_ACT_GELU_TANH>(a);
    else if (act == ECC_ACT_SILU)
        activate<ECC_ACT_SILU>(a);
}

// W rows of a column, the first n of them in range.  The rows' addresses are
// the same for the whole warp (uniform registers); a lane adds its column.
// A reduction of less than about 1024 takes as long as this does, 3.5 us a tile
// of 256 x 256 (8192 x 16384 x 64: 103 us, 2.6 TB/s, and as long with e4m3
// results; finish_staged: 68).  Slower: four values a store, lanes' rows
// exchanged for columns by shuffles; whole rows by four warps through shared
// memory; eight warps of 16 rows at a time.
template <typename T, int W>
__device__ __forceinline__ void store_rows(void *base, uint64_t ld, uint64_t r0, uint32_t n, uint32_t c, const float (&a)[W],
                                           float s)
{
    T *row = static_cast<T *>(base) + r0 * ld;
    if (n == W) {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            row[c] = from_f32<T>(sizeof(T) == 1 ? a[j] * s : a[j]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            if (j < n)
                row[c] = from_f32<T>(sizeof(T) == 1 ? a[j] * s : a[j]);
    }
}
// The residual of W rows of a column, as it is stored: asked for before the
// products are waited for (with the loads after them a 8192 x 16384 x 4096
// product took 906 us instead of 560).
template <typename T, int W>
__device__ __forceinline__ void load_rows(const void *base, uint64_t ld, uint64_t r0, uint32_t n, uint32_t c, uint32_t (&v)[W])
{
    const T *row = static_cast<const T *>(base) + r0 * ld;
    if (n == W) {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            v[j] = row[c];
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            if (j < n)
                v[j] = row[c];
    }
}
template <int W>
__device__ __forceinline__ void ask_residual(const Epilogue &e, uint32_t (&v)[W], uint64_t r0, uint32_t n, uint32_t c)
{
    if (!e.residual)
        return;
    if (e.res_type == ECC_F32)
        load_rows<uint32_t>(e.residual, e.ldres, r0, n, c, v);
    else
        load_rows<uint16_t>(e.residual, e.ldres, r0, n, c, v);
}
template <int W> __device__ __forceinline__ void add_residual(uint32_t type, const uint32_t (&v)[W], float (&a)[W])
{
    if (type == ECC_F32) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __uint_as_float(v[j]);
    } else if (type == ECC_BF16) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __uint_as_float(v[j] << 16);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __half2float(__ushort_as_half((unsigned short)v[j]));
    }
}

// W rows from row `r0` (the first n of them in range) of this thread's column c
template <int W>
__device__ __forceinline__ void finish(const Epilogue &e, float (&a)[W], const uint32_t (&res)[W], uint64_t r0, uint32_t n,
                                       uint32_t c, float bias, float scale)
{
#pragma unroll
    for (int j = 0; j < W; ++j)
        a[j] = a[j] * scale + bias;
    if (e.pre) {
        if (e.pre_type == ECC_F32)
            store_rows<float>(e.pre, e.ldpre, r0, n, c, a, 1.f);
        else if (e.pre_type == ECC_BF16)
            store_rows<bf16>(e.pre, e.ldpre, r0, n, c, a, 1.f);
        else
            store_rows<__half>(e.pre, e.ldpre, r0, n, c, a, 1.f);
    }
    activate_by(e.act, a);
    if (e.residual)
        add_residual(e.res_type, res, a);
    void *out = e.out;
    uint64_t ld = e.ldout;
    if (e.rswitch && r0 >= e.rswitch) { // rows of the second output (no chunk has rows of both)
        out = e.out2;
        ld = e.ldout2;
        r0 -= e.rswitch;
        n = r0 < e.rows2 ? (uint32_t)min((uint64_t)n, e.rows2 - r0) : 0;
    } else if (e.rswitch) { // (rows between the first one's end and the second's start are padding)
        n = r0 < e.rows2 ? (uint32_t)min((uint64_t)n, e.rows2 - r0) : 0;
    }
    if (e.out_type == ECC_F32)
        store_rows<float>(out, ld, r0, n, c, a, 1.f);
    else if (e.out_type == ECC_BF16)
        store_rows<bf16>(out, ld, r0, n, c, a, 1.f);
    else if (e.out_type == ECC_F16)
        store_rows<__half>(out, ld, r0, n, c, a, 1.f);
    else
        store_rows<e4m3>(out, ld, r0, n, c, a, e.out_scale);
}
template <int MODE> __device__ __forceinline__ float scale_of(const Epilogue &e)
{
    if constexpr (MODE == kStats || MODE == kSlopes)
        return e.scale * 1.44269504f;
    else
        return e.factor ? e.scale * *e.factor : e.scale;
}

// the scale of the output that row r0 belongs to (only products of two operands down their columns have two)
template <bool TWO> __device__ __forceinline__ float scale_at(const Epilogue &e, uint64_t r0, float scale)
{
    if (!TWO || !e.rswitch || r0 < e.rswitch)
        return scale;
    return e.factor ? e.scale2 * e.factor[1] : e.scale2;
}

// Results that leave through shared memory take a warp's two stages in turns:
// 32 rows' stage is written once all copies but the last 32 rows' have read
// theirs, which is the other stage's.  A tile starts with the first stage: behind
// one that ended with it, after an odd number of 32 rows, the last copies have to
// have read theirs too.  (A stage that turns on over the tiles took a register
// too many, and spills: 8192 x 16384 x 64 76 us, 72 so.)
__device__ __forceinline__ void first_stage_read(const GemmArgs &g, uint32_t lane, uint32_t j0)
{
    if (lane == 0 && (g.odd & (j0 ? 2 : 1)))
        tma_stores_read<0>();
}
// The same for results that leave through shared memory (no pre, no residual):
// a warp's 32 rows of 32 columns at `stage`, a row after the other.  8192 x
// 16384 x 64 68 us, 4 TB/s (103 by store_rows); at a reduction of 1024 156 us
// (167).  For 16-bit and float32 results on 16-byte boundaries.
template <typename T> __device__ __forceinline__ void stage_rows(uint8_t *stage, uint32_t lane, const float (&a)[32])
{
    T *s = reinterpret_cast<T *>(stage) + lane;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        s[j * 32] = from_f32<T>(a[j]);
}
__device__ __forceinline__ void finish_staged(const Epilogue &e, float (&a)[32], uint8_t *stage, uint32_t lane, float bias, float scale)
{
#pragma unroll
    for (int j = 0; j < 32; ++j)
        a[j] = a[j] * scale + bias;
    activate_by(e.act, a);
    if (e.out_type == ECC_F32)
        stage_rows<float>(stage, lane, a);
    else if (e.out_type == ECC_BF16)
        stage_rows<bf16>(stage, lane, a);
    else
        stage_rows<__half>(stage, lane, a);
}

// ---------------------------------------------------------------- gated epilogue
// Lanes 0 to 15: W rows of column c's gate; lanes 16 to 31: of its up (or the
// other way round).  Each lane keeps its half of the rows, the even ones or the
// odd ones, gets the other matrix's value of them and makes the result.  a
// becomes g or u.
template <int W>
__device__ __forceinline__ void gated_values(const Epilogue &e, float (&a)[W], float (&out)[W / 2], float bias, uint32_t lane)
{
    const bool second = lane & 16, up = e.swapped != second;
    const float scale = up ? e.scale2 : e.scale;
#pragma unroll
    for (int j = 0; j < W; ++j)
        a[j] = a[j] * scale + bias;
    float other[W / 2];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        const float got = __shfl_xor_sync(~0u, second ? a[2 * j] : a[2 * j + 1], 16), own = second ? a[2 * j + 1] : a[2 * j];
        out[j] = up ? got : own;
        other[j] = up ? own : got;
    }
    activate_by(e.act, out);
#pragma unroll
    for (int j = 0; j < W / 2; ++j)
        out[j] *= other[j];
}
template <int W>
__device__ __forceinline__ void finish_gated(const Epilogue &e, float (&a)[W], uint64_t r0, uint32_t n, uint32_t c, bool col_ok,
                                             float bias, uint32_t lane)
{
    float out[W / 2];
    gated_values(e, a, out, bias, lane);
    if (!col_ok)
        return;
    const uint32_t second = lane >> 4;
    if (e.pre) {
        const bool up = e.swapped != (bool)second;
        void *pre = up ? e.pre2 : e.pre;
        const uint64_t ld = up ? e.ldpre2 : e.ldpre;
        if (e.pre_type == ECC_F32)
            store_rows<float>(pre, ld, r0, n, c, a, 1.f);
        else if (e.pre_type == ECC_BF16)
            store_rows<bf16>(pre, ld, r0, n, c, a, 1.f);
        else
            store_rows<__half>(pre, ld, r0, n, c, a, 1.f);
    }
    // every second row from r0 + second on
    const uint64_t first = (r0 + second) * e.ldout;
    n = (n + 1 - second) / 2;
    if (e.out_type == ECC_F32)
        store_rows<float>(static_cast<float *>(e.out) + first, 2 * e.ldout, 0, n, c, out, 1.f);
    else if (e.out_type == ECC_BF16)
        store_rows<bf16>(static_cast<bf16 *>(e.out) + first, 2 * e.ldout, 0, n, c, out, 1.f);
    else if (e.out_type == ECC_F16)
        store_rows<__half>(static_cast<__half *>(e.out) + first, 2 * e.ldout, 0, n, c, out, 1.f);
    else
        store_rows<e4m3>(static_cast<e4m3 *>(e.out) + first, 2 * e.ldout, 0, n, c, out, e.out_scale);
}
// Results through shared memory: 32 rows of 16 columns of the output, of g and
// of u.
template <typename T, int STEP, int N>
__device__ __forceinline__ void stage_gated(uint8_t *stage, uint32_t at, const float (&v)[N], float s)
{
    T *p = reinterpret_cast<T *>(stage) + at;
#pragma unroll
    for (int j = 0; j < N; ++j)
        p[j * STEP] = from_f32<T>(sizeof(T) == 1 ? v[j] * s : v[j]);
}
__device__ __forceinline__ void finish_gated_staged(const Epilogue &e, float (&a)[32], uint8_t *stage, float bias, uint32_t lane)
{
    float out[16];
    gated_values(e, a, out, bias, lane);
    const uint32_t second = lane >> 4, col = lane & 15, at = second * 16 + col;
    if (e.out_type == ECC_F32)
        stage_gated<float, 32>(stage, at, out, 1.f);
    else if (e.out_type == ECC_BF16)
        stage_gated<bf16, 32>(stage, at, out, 1.f);
    else if (e.out_type == ECC_F16)
        stage_gated<__half, 32>(stage, at, out, 1.f);
    else
        stage_gated<e4m3, 32>(stage, at, out, e.out_scale);
    stage += 512 * (e.out_type == ECC_F32 ? 4 : e.out_type == ECC_E4M3 ? 1 : 2);
    const uint32_t from = (e.swapped != (bool)second ? 512 : 0) + col;
    if (e.pre_type == ECC_F32)
        stage_gated<float, 16>(stage, from, a, 1.f);
    else if (e.pre_type == ECC_BF16)
        stage_gated<bf16, 16>(stage, from, a, 1.f);
    else
        stage_gated<__half, 16>(stage, from, a, 1.f);
}

// ---------------------------------------------------------------- logits' epilogues
// A share of the vocabulary of one token: y = log2 e * logit, m the largest, s
// the sum of 2^(y - m), t the sum of 2^(y - m) (y - m).  A logit that is not
// finite makes t NaN, and with it the row's results.
struct LogitsPart {
    float m = -INFINITY, s = 0.f, t = 0.f;
};
// v = x if i is j (in assembly, so that no array is moved to memory to be indexed)
__device__ __forceinline__ void pick(float &v, int i, int j, float x)
{
    asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, %2;\n\t@p mov.f32 %0, %3;\n\t}" : "+f"(v) : "r"(i), "r"(j), "f"(x));
}
// the next W logits, the first n of them in range; rel: the token's place among them
template <int W>
__device__ __forceinline__ void add_logits(const Epilogue &e, float (&a)[W], uint32_t n, float scale, int64_t rel, uint32_t c,
                                           LogitsPart &p)
{
    float2 y[W / 2];
#pragma unroll
    for (int j = 0; j < W / 2; ++j)
        y[j] = mul2(make_float2(a[2 * j], a[2 * j + 1]), both(scale));
    float top = -INFINITY;
    if (n == W) {
#pragma unroll
        for (int j = 0; j < W / 2; ++j)
            top = fmaxf(top, fmaxf(y[j].x, y[j].y));
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < n)
                top = fmaxf(top, j & 1 ? y[j / 2].y : y[j / 2].x);
    }
    const float m = fmaxf(p.m, top), back = p.s > 0.f ? p.m - m : 0.f, r = exp2_approx(back);
    float2 s = make_float2(p.s * r, 0.f), t = make_float2(r * fmaf(back, p.s, p.t), 0.f);
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        float2 d = add2(y[j], both(-m)), x = exp2_both(d);
        if (n < W) { // outside the vocabulary
            if (2 * j >= n)
                d.x = x.x = 0.f;
            if (2 * j + 1 >= n)
                d.y = x.y = 0.f;
        }
        s = add2(s, x);
        t = fma2(x, d, t);
    }
    p.m = m;
    p.s = s.x + s.y;
    p.t = t.x + t.y;
    if (rel >= 0 && rel < (int64_t)n) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j)
            pick(v, (int)rel, j, j & 1 ? y[j / 2].y : y[j / 2].x);
        e.token_logit[c] = v;
    }
}

// All of a share: the first n of W logits, at once (one maximum, one pass of exponentials)
template <int W, bool ALL>
__device__ __forceinline__ LogitsPart whole_part(const Epilogue &e, float2 (&a)[W / 2], uint32_t n, float scale, int64_t rel, uint32_t c)
{
    LogitsPart p;
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        a[j] = mul2(a[j], both(scale));
        if (ALL || 2 * j < n)
            top[j % 4] = fmaxf(top[j % 4], a[j].x);
        if (ALL || 2 * j + 1 < n)
            top[j % 4] = fmaxf(top[j % 4], a[j].y);
    }
    if (rel >= 0 && rel < (int64_t)n) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            pick(v, (int)rel, 2 * j, a[j].x);
            pick(v, (int)rel, 2 * j + 1, a[j].y);
        }
        e.token_logit[c] = v;
    }
    p.m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    float2 s[2] = {both(0.f), both(0.f)}, t[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        float2 d = add2(a[j], both(-p.m)), x = exp2_both(d);
        if (!ALL) { // outside the vocabulary
            if (2 * j >= n)
                d.x = x.x = 0.f;
            if (2 * j + 1 >= n)
                d.y = x.y = 0.f;
        }
        s[j % 2] = add2(s[j % 2], x);
        t[j % 2] = fma2(x, d, t[j % 2]);
    }
    s[0] = add2(s[0], s[1]);
    t[0] = add2(t[0], t[1]);
    p.s = s[0].x + s[0].y;
    p.t = t[0].x + t[0].y;
    return p;
}

// What a token's gradient with respect to its logits is made of:
// t = dlogprob 1[token] - p (dlogprob + dentropy (log p + H))
struct LogitsSlope {
    float lse = 0.f, one = 0.f, all = 0.f, each = 0.f; // log2 e lse; dlogprob; dlogprob + dentropy H; dentropy log 2
    int64_t token = -1;
};
__device__ __forceinline__ LogitsSlope slope_of_token(const Epilogue &e, uint32_t c, bool col_ok)
{
    LogitsSlope s;
    if (!col_ok)
        return s;
    const float factor = e.factor ? *e.factor : 1.f;
    s.lse = e.lse[c] * 1.44269504f;
    s.token = e.tokens ? e.tokens[c] : -1;
    if (e.dlogprob && s.token >= 0 && s.token < (int64_t)e.vocab)
        s.one = e.dlogprob[c] * factor;
    else
        s.token = -1;
    s.all = s.one;
    if (e.dentropy) {
        const float dh = e.dentropy[c] * factor;
        s.all = fmaf(dh, e.entropy[c], s.one);
        s.each = dh * 0.69314718f;
    }
    return s;
}
// t of W logits; rel: the token's place among them
template <int W>
__device__ __forceinline__ void slope_values(float2 (&t)[W / 2], const float (&a)[W], float scale, int64_t rel, const LogitsSlope &s)
{
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        const float2 d = fma2(make_float2(a[2 * j], a[2 * j + 1]), both(scale), both(-s.lse));
        t[j] = mul2(mul2(exp2_both(d), both(-1.f)), fma2(d, both(s.each), both(s.all)));
    }
    if (rel >= 0 && rel < W) {
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            t[j].x += 2 * j == (int)rel ? s.one : 0.f;
            t[j].y += 2 * j + 1 == (int)rel ? s.one : 0.f;
        }
    }
}
// W logits from vocabulary index v of this launch's part (a multiple of 8) on
template <int W>
__device__ __forceinline__ void store_slopes(const Epilogue &e, const float (&a)[W], uint64_t v, uint32_t c, float scale, int64_t rel,
                                             const LogitsSlope &s)
{
    float2 t[W / 2];
    slope_values(t, a, scale, rel, s);
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(e.out) + c * e.ldout + v);
#pragma unroll
    for (int j = 0; j < W / 8; ++j)
        out[j] = e.out_type == ECC_BF16 ? pack2<bf16>(t + 4 * j) : pack2<__half>(t + 4 * j);
}
// 32 logits of a lane's token to shared memory, rows of 64 bytes in the 64-byte
// swizzle (the lanes' 16-byte stores would otherwise meet in two groups of banks)
__device__ __forceinline__ void stage_slopes(const Epilogue &e, const float (&a)[32], uint8_t *stage, uint32_t lane, float scale, int64_t rel,
                                             const LogitsSlope &s)
{
    float2 t[16];
    slope_values(t, a, scale, rel, s);
    uint4 *row = reinterpret_cast<uint4 *>(stage + lane * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        row[j ^ (lane >> 1 & 3)] = e.out_type == ECC_BF16 ? pack2<bf16>(t + 4 * j) : pack2<__half>(t + 4 * j);
}

template <int MODE> __device__ __forceinline__ float bias_of(const Epilogue &e, uint32_t c, bool col_ok, uint32_t lane)
{
    const void *bias = MODE == kGated && e.swapped != (bool)(lane & 16) ? e.bias2 : e.bias;
    return bias && col_ok ? load_any(bias, c, e.bias_type) : 0.f;
}
// this thread's column of the output
template <int MODE> __device__ __forceinline__ uint32_t column_of(uint32_t p0, uint32_t quad, uint32_t lane)
{
    return MODE == kGated ? p0 + quad * 16 + (lane & 15) : p0 + quad * 32 + lane;
}

// This CTA's part of a tile, [column of tensor memory][lane], for the join.
template <int W> __device__ __forceinline__ void keep_part(float *parts, const float (&a)[W], uint32_t j, uint32_t row)
{
#pragma unroll
    for (int i = 0; i < W; ++i)
        parts[(j + i) * kPTile + row] = a[i];
}
// Share `share` of a tile's rows [r0, ...): the sum of the g.split CTAs'
// parts, eight rows at a time so that their loads are in flight together,
// then the epilogue.  `at`: this lane's first value in its CTA's part;
// `base`: the cluster's rank of the first of those CTAs.
template <int MODE>
__device__ __forceinline__ void join_parts(const GemmArgs &g, uint32_t at, uint32_t base, uint32_t share, uint64_t r0, uint32_t c,
                                           uint32_t lane)
{
    const uint32_t n = (uint32_t)min((uint64_t)g.bn, g.rows - r0), even = (n + g.split - 1) / g.split;
    const uint32_t per = MODE == kSlopes ? (even + 7) & ~7u : even; // (slopes are stored by eights)
    const uint32_t j0 = share * per, j1 = min(n, j0 + per);
    const bool col_ok = c < g.cols;
    if (MODE != kGated && !col_ok)
        return;
    const float bias = bias_of<MODE>(g.e, c, col_ok, lane), scale = scale_of<MODE>(g.e);
    LogitsPart p;
    const LogitsSlope slope = MODE == kSlopes ? slope_of_token(g.e, c, col_ok) : LogitsSlope();
    const int64_t token = MODE == kStats && g.e.tokens ? g.e.tokens[c] : -1;
    for (uint32_t j = j0; j < j1; j += 8) {
        float a[8] = {};
        uint32_t res[8];
        if constexpr (MODE == kPlain || MODE == kDual)
            ask_residual(g.e, res, r0 + j, min(8u, j1 - j), c);
        for (uint32_t k = 0; k < g.split; ++k) {
            const uint32_t from = cluster_addr(at + j * kPTile * 4, base + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (j + i < j1)
                    a[i] += cluster_load(from + i * kPTile * 4);
        }
        if constexpr (MODE == kGated)
            finish_gated(g.e, a, r0 + j, min(8u, j1 - j), c, col_ok, bias, lane);
        else if constexpr (MODE == kStats)
            add_logits(g.e, a, min(8u, j1 - j), scale, token - (int64_t)(r0 + j), c, p);
        else if constexpr (MODE == kSlopes)
            store_slopes(g.e, a, r0 + j, c, scale, slope.token - (int64_t)(g.e.first + r0 + j), slope);
        else
            finish(g.e, a, res, r0 + j, min(8u, j1 - j), c, bias, scale_at<true>(g.e, r0 + j, scale));
    }
    if constexpr (MODE == kStats)
        g.e.part[(r0 / g.bn * g.split + share) * g.cols + c] = make_float4(p.m, p.s, p.t, 0.f);
}

// ---------------------------------------------------------------- loads and products of a reduction block
// rows [r0, r0 + n) of reduction block kb -> dst.  Down the columns, `wide`:
// one box over groups of 64 rows where there are only whole groups, or a box
// for each (a copy unit takes a box in about 120 cycles, and four of them
// a block kept the tensor pipe 80% active).
template <int CG, bool MN, bool F8>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, uint64_t r0, uint32_t n, uint32_t kb, bool wide,
                                             uint32_t bar)
{
    constexpr int per = F8 ? 128 : 64; // reduction indices of a block
    if constexpr (MN) {
        if (wide)
            tma_load_groups<CG>(dst, map, (int)(kb * 64), (int)(r0 / 64), bar);
        else
            for (uint32_t c = 0; c < n; c += 64)
                tma_load<CG>(dst + c * kTileBytes, map, (int)(r0 + c), (int)(kb * 64), bar);
    } else {
        tma_load<CG>(dst, map, (int)(kb * per), (int)r0, bar);
    }
}

// P's rows for columns [p0, ...) of the output.  Gated: one box of a map over
// both matrices where one can be made, or eight of 16 rows (which the copies'
// rate does not keep up with: 8192 x 16384 x 4096 takes 1594 us with them, the
// tensor pipe 56% active).
template <int CG, bool MN, bool F8, int MODE>
__device__ __forceinline__ void load_p(uint32_t dst, const CUtensorMap *map, const CUtensorMap *map2, uint64_t p0, uint32_t kb,
                                       const GemmArgs &g, uint32_t bar)
{
    if constexpr (MODE == kGated) {
        constexpr int per = F8 ? 128 : 64;
        if (g.one_box)
            tma_load_turns<CG>(dst, map, (int)(kb * per), (int)(p0 / 16), bar);
        else
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            tma_load<CG>(dst + q * 32 * kTileBytes, map, (int)(kb * per), (int)(p0 + q * 16), bar);
            tma_load<CG>(dst + (q * 32 + 16) * kTileBytes, map2, (int)(kb * per), (int)(p0 + q * 16), bar);
        }
    } else if (MODE == kDual && kb >= g.kswitch) {
        load_operand<CG, MN, F8>(dst, map2, p0, kPTile, kb - g.kswitch, g.pwide, bar);
    } else {
        load_operand<CG, MN, F8>(dst, map, p0, kPTile, kb, g.pwide, bar);
    }
}

template <int CG, bool PMN, bool QMN, bool F8>
__device__ __forceinline__ void multiply_block(uint32_t d, uint32_t pa, uint32_t qa, uint32_t idesc, bool first)
{
    const uint64_t a = operand_desc<PMN>(pa, 64 * kTileBytes), b = operand_desc<QMN>(qa, 64 * kTileBytes);
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
        tensor_product<CG, F8>(d, a + k * operand_step<PMN>(), b + k * operand_step<QMN>(), idesc, !first || k > 0);
}

// behind the launch's own preparation: wait for what it reads
__device__ __forceinline__ void begin(const GemmArgs &g)
{
    wait_for_previous();
    let_next_start();
    if (g.clear_status && blockIdx.x == 0 && threadIdx.x == 0) // waits that give up do so a second from now at the earliest
        *(volatile uint32_t *)g.status = ECC_OK;
}

// ---------------------------------------------------------------- pairs of CTAs, many tiles
// Tiles in groups of 8 column tiles, a group row tile by row tile: the tiles
// in work at a time form a block that shares its operands through L2.
struct TilePos {
    uint32_t p, q;
};
__device__ __forceinline__ TilePos tile_pos(uint32_t t, uint32_t ptiles, uint32_t qtiles)
{
    const uint32_t g = t / (8 * qtiles), p0 = g * 8, w = min(8u, ptiles - p0), r = t - g * 8 * qtiles;
    return {p0 + r % w, r / w};
}

// kStats: the sums of 128 columns stay in a thread's registers, which the warps
// that hold none of them give up: four warps of 40 and eight of 232, together
// what twelve warps of 168 are launched with (the build checks that the
// compiler gives this kernel 168, and the launch that it has them; 12 bytes a
// thread spill).
constexpr int kStatsThreads = 384, kStatsRegisters = 168;
constexpr int kFewRegisters = 40, kManyRegisters = 232;
static_assert(kFewRegisters + 2 * kManyRegisters <= 3 * kStatsRegisters, "more registers than the launch has");
template <int MODE> constexpr int kThreadsOf = MODE == kStats ? kStatsThreads : kPairThreads;
template <int MODE> constexpr uint32_t kFirstEpilogueWarp = MODE == kStats ? 4 : 2;
template <int N> __device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

template <bool PMN, bool QMN, bool F8, int MODE>
__global__ void __launch_bounds__(kThreadsOf<MODE>, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap pmap2,
                     const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap,
                     const __grid_constant__ CUtensorMap omap2, const __grid_constant__ CUtensorMap omap3,
                     const __grid_constant__ GemmArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t stage0 = (smem_u32(smem_raw) + kSmemHead - 1) & ~(kSmemHead - 1);
    const uint32_t qn = g.bn / 2, stage_bytes = kPBytes + qn * kTileBytes;
    const uint32_t tiles = g.ptiles * g.qtiles, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < g.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 16); // eight epilogue warps of each CTA
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&pmap);
        if constexpr (MODE == kGated || MODE == kDual)
            prefetch_map(&pmap2);
        prefetch_map(&qmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&s.tmem), 512);
        tmem_fence_before();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&s.tmem;
    begin(g);
    if (warp < kFirstEpilogueWarp<MODE>) {
        if constexpr (MODE == kStats)
            give_registers<kFewRegisters>();
        if (warp == 0 && lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            for (uint32_t t = pair; t < tiles && ok; t += pairs) {
                const TilePos pos = tile_pos(t, g.ptiles, g.qtiles);
                const uint64_t p0 = (uint64_t)(pos.p * 2 + rank) * kPCols<MODE>, q0 = (uint64_t)pos.q * g.bn + rank * qn;
                for (uint32_t kb = 0; kb < g.kblocks; ++kb) {
                    if (!(ok = mbar_wait(&s.empty[st], ph ^ 1, g.limit_ns)))
                        break;
                    const uint32_t bar = cluster_addr(smem_u32(&s.full[st]), 0), at = stage0 + st * stage_bytes;
                    if (rank == 0)
                        mbar_expect_tx(&s.full[st], 2 * stage_bytes);
                    load_p<2, PMN, F8, MODE>(at, &pmap, &pmap2, p0, kb, g, bar);
                    load_operand<2, QMN, F8>(at + kPBytes, &qmap, q0, qn, kb, g.qwide, bar);
                    ++issued;
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) { // give the copies in flight a last wait
                set_status(g.status, ECC_ERR_TIMEOUT);
                if (rank == 0)
                    for (uint32_t i = 0; i < min(issued, g.stages); ++i) {
                        if (st == 0) {
                            st = g.stages;
                            ph ^= 1;
                        }
                        --st;
                        (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                    }
            }
        }
        if (warp == 1 && lane == 0 && rank == 0) {
            uint32_t st = 0, ph = 0, acc = 0, aph = 0;
            bool ok = true;
            uint32_t k0 = 0; // the accumulator's first reduction block
            for (uint32_t t = pair; t < tiles && ok; k0 + kSegment < g.kblocks && MODE == kStats ? k0 += kSegment : (k0 = 0, t += pairs)) {
                if (!(ok = mbar_wait(&s.tempty[acc], aph ^ 1, g.limit_ns)))
                    break;
                tmem_fence_after();
                const uint32_t k1 = MODE == kStats ? min(g.kblocks, k0 + kSegment) : g.kblocks;
                for (uint32_t kb = k0; kb < k1; ++kb) {
                    if (!(ok = mbar_wait(&s.full[st], ph, g.limit_ns))) {
                        (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t at = stage0 + st * stage_bytes;
                    multiply_block<2, PMN, QMN, F8>(tmem + acc * g.bn, at, at + kPBytes, g.idesc, kb == k0);
                    tensor_commit<2>(smem_u32(&s.empty[st]));
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                tensor_commit<2>(smem_u32(&s.tfull[acc]));
                if (acc)
                    aph ^= 1;
                acc ^= 1;
            }
            if (!ok)
                set_status(g.status, ECC_ERR_TIMEOUT);
        }
    } else {
        if constexpr (MODE == kStats)
            take_registers<kManyRegisters>();
        const uint32_t quad = warp & 3; // a warp reads the lanes of its number modulo 4
        const uint32_t j0 = warp < kFirstEpilogueWarp<MODE> + 4 ? 0 : g.bn / 2, j1 = j0 + g.bn / 2;
        uint32_t acc = 0, aph = 0;
        const float scale = scale_of<MODE>(g.e);
        for (uint32_t t = pair; t < tiles; t += pairs) {
            const TilePos pos = tile_pos(t, g.ptiles, g.qtiles);
            const uint32_t c = column_of<MODE>((pos.p * 2 + rank) * kPCols<MODE>, quad, lane);
            const uint64_t r0 = (uint64_t)pos.q * g.bn;
            const bool col_ok = c < g.cols;
            const float bias = bias_of<MODE>(g.e, c, col_ok, lane);
            const uint64_t left = g.rows - r0;
            // (where there are two scales no half of a tile has rows of both; asked for with each 32 rows, 64 x 65536 x 4096
            // down the columns takes 144 us in place of 139)
            const float half_scale = scale_at<PMN && QMN>(g.e, r0 + j0, scale);
            if constexpr (MODE == kStats) {
                const int64_t token = g.e.tokens && col_ok ? g.e.tokens[c] : -1;
                float2 a[64]; // (kStats: bn is 256)
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    a[i] = both(0.f);
                bool ok = true;
                for (uint32_t k0 = 0; ok && k0 < g.kblocks; k0 += kSegment) {
                    if (!(ok = __all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))))
                        break;
                    tmem_fence_after();
#pragma unroll
                    for (uint32_t i = 0; i < 128; i += 16)
                        tmem_add16(tmem + (quad * 32 << 16) + acc * 256 + j0 + i, a + i / 2);
                    tmem_fence_before(); // the accumulator is read: products may fill it again
                    __syncwarp();
                    if (lane == 0)
                        cluster_arrive(cluster_addr(smem_u32(&s.tempty[acc]), 0));
                    if (acc)
                        aph ^= 1;
                    acc ^= 1;
                }
                if (!ok) {
                    if (lane == 0)
                        set_status(g.status, ECC_ERR_TIMEOUT);
                    break;
                }
                LogitsPart p;
                const int64_t rel = token - (int64_t)(r0 + j0);
                if (col_ok && left >= j1)
                    p = whole_part<128, true>(g.e, a, 128, scale, rel, c);
                else if (col_ok && left > j0)
                    p = whole_part<128, false>(g.e, a, (uint32_t)(left - j0), scale, rel, c);
                if (col_ok)
                    g.e.part[(pos.q * 2 + (j0 ? 1 : 0)) * g.cols + c] = make_float4(p.m, p.s, p.t, 0.f);
                continue;
            }
            if constexpr (MODE == kSlopes) {
                const LogitsSlope slope = slope_of_token(g.e, c, col_ok);
                if (!__all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))) {
                    if (lane == 0)
                        set_status(g.status, ECC_ERR_TIMEOUT);
                    break;
                }
                tmem_fence_after();
                if (g.staged)
                    first_stage_read(g, lane, j0);
                for (uint32_t j = j0; j < j1; j += 32) {
                    float a[32];
                    tmem_load32(tmem + (quad * 32 << 16) + acc * g.bn + j, a);
                    if (j + 32 == j1) { // the accumulator is read: products may fill it again
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            cluster_arrive(cluster_addr(smem_u32(&s.tempty[acc]), 0));
                    }
                    if (j >= left)
                        continue;
                    const int64_t rel = slope.token - (int64_t)(g.e.first + r0 + j);
                    if (!g.staged) {
                        if (col_ok)
                            store_slopes(g.e, a, r0 + j, c, scale, rel, slope);
                        continue;
                    }
                    // (through shared memory for short reductions: a store of 16 bytes in each of 32 rows takes 4.8 us a tile,
                    // 4096 x 25088 x 256 101 us)
                    const uint32_t c0 = c - lane;
                    if (c0 >= g.cols)
                        continue;
                    uint8_t *at = smem_raw + (stage0 - smem_u32(smem_raw)) + g.stages * stage_bytes + (warp - 2) * 2 * g.staged +
                                  (j & 32 ? g.staged : 0);
                    if (lane == 0)
                        tma_stores_read<1>();
                    __syncwarp();
                    stage_slopes(g.e, a, at, lane, scale, rel, slope);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store(&omap, smem_u32(at), (int)(r0 + j), (int)c0);
                        tma_stores_commit();
                    }
                }
                if (acc)
                    aph ^= 1;
                acc ^= 1;
                continue;
            }
            if ((MODE == kPlain || MODE == kGated) && g.staged) {
                // Short reductions: results through shared memory, two stages a
                // warp, by copies of 32 rows.  (Half the instructions of
                // store_rows, none of them an address.)
                if (!__all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))) {
                    if (lane == 0)
                        set_status(g.status, ECC_ERR_TIMEOUT);
                    break;
                }
                tmem_fence_after();
                uint8_t *stage = smem_raw + (stage0 - smem_u32(smem_raw)) + g.stages * stage_bytes + (warp - 2) * 2 * g.staged;
                const uint32_t c0 = c - (MODE == kGated ? lane & 15 : lane);
                first_stage_read(g, lane, j0);
                for (uint32_t j = j0; j < j1; j += 32) {
                    float a[32];
                    tmem_load32(tmem + (quad * 32 << 16) + acc * g.bn + j, a);
                    if (j + 32 == j1) { // the accumulator is read: products may fill it again
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            cluster_arrive(cluster_addr(smem_u32(&s.tempty[acc]), 0));
                    }
                    if (j >= left || c0 >= g.cols)
                        continue;
                    uint8_t *at = stage + (j & 32 ? g.staged : 0);
                    if (lane == 0)
                        tma_stores_read<1>();
                    __syncwarp();
                    if constexpr (MODE == kGated)
                        finish_gated_staged(g.e, a, at, bias, lane);
                    else
                        finish_staged(g.e, a, at, lane, bias, half_scale);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        const uint64_t r = r0 + j;
                        if constexpr (MODE == kGated) {
                            const uint32_t pre = smem_u32(at) + 512 * (g.e.out_type == ECC_F32 ? 4 : g.e.out_type == ECC_E4M3 ? 1 : 2);
                            tma_store(&omap, smem_u32(at), (int)c0, (int)r);
                            tma_store(&omap2, pre, (int)c0, (int)r);
                            tma_store(&omap3, pre + 512 * (g.e.pre_type == ECC_F32 ? 4 : 2), (int)c0, (int)r);
                        } else if (g.e.rswitch && r >= g.e.rswitch) {
                            tma_store(&omap2, smem_u32(at), (int)c0, (int)(r - g.e.rswitch));
                        } else {
                            tma_store(&omap, smem_u32(at), (int)c0, (int)r);
                        }
                        tma_stores_commit();
                    }
                }
                if (acc)
                    aph ^= 1;
                acc ^= 1;
                continue;
            }
            uint32_t res[2][32]; // of this chunk of 32 rows and the next
            auto ask = [&](uint32_t j, uint32_t (&v)[32]) {
                if (MODE != kGated && col_ok && j < j1 && j < left)
                    ask_residual(g.e, v, r0 + j, (uint32_t)min((uint64_t)32, left - j), c);
            };
            ask(j0, res[0]);
            if (!__all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))) {
                if (lane == 0)
                    set_status(g.status, ECC_ERR_TIMEOUT);
                break;
            }
            tmem_fence_after();
            auto chunk = [&](uint32_t j, const uint32_t (&v)[32]) {
                float a[32];
                tmem_load32(tmem + (quad * 32 << 16) + acc * g.bn + j, a);
                if (j + 32 == j1) { // the accumulator is read: products may fill it again
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        cluster_arrive(cluster_addr(smem_u32(&s.tempty[acc]), 0));
                }
                if constexpr (MODE == kGated) {
                    if (j < left)
                        finish_gated(g.e, a, r0 + j, (uint32_t)min((uint64_t)32, left - j), c, col_ok, bias, lane);
                } else {
                    if (col_ok && j < left)
                        finish(g.e, a, v, r0 + j, (uint32_t)min((uint64_t)32, left - j), c, bias, half_scale);
                }
            };
            for (uint32_t j = j0; j < j1; j += 64) { // (bn is 128 or 256)
                ask(j + 32, res[1]);
                chunk(j, res[0]);
                ask(j + 64, res[0]);
                chunk(j + 32, res[1]);
            }
            if (acc)
                aph ^= 1;
            acc ^= 1;
        }
    }
    if ((MODE == kPlain || MODE == kGated || MODE == kSlopes) && g.staged && lane == 0)
        tma_stores_done();
    __syncthreads();
    __syncwarp();
    tmem_fence_before();
    cluster_sync(); // both CTAs are done with each other's barriers and tensor memory
    tmem_fence_after();
    if (warp == 1)
        tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- clusters that share a tile's reduction
// `wait` waits for the products (the first residual is asked for before);
// `used`: accumulators to add up (kStats)
template <int W, int MODE, typename Wait>
__device__ __forceinline__ void split_columns(const GemmArgs &g, uint32_t tmem, uint32_t quad, uint32_t lane, uint32_t c,
                                              uint64_t r0, bool col_ok, float bias, bool direct, float *part, uint32_t used, Wait wait)
{
    const uint64_t left = g.rows - r0;
    const float scale = scale_of<MODE>(g.e);
    LogitsPart p;
    const int64_t token = MODE == kStats && direct && g.e.tokens && col_ok ? g.e.tokens[c] : -1;
    const LogitsSlope slope = MODE == kSlopes && direct ? slope_of_token(g.e, c, col_ok) : LogitsSlope();
    for (uint32_t j = 0; j < g.bn && j < left; j += W) {
        float a[W];
        uint32_t res[W];
        const uint32_t n = (uint32_t)min((uint64_t)W, left - j);
        if ((MODE == kPlain || MODE == kDual) && direct && col_ok)
            ask_residual(g.e, res, r0 + j, n, c);
        if (j == 0 && g.kblocks && !wait())
            return;
        if (g.kblocks) {
            auto load = [&](uint32_t at, float (&v)[W]) {
                if constexpr (W == 32)
                    tmem_load32(tmem + (quad * 32 << 16) + at, v);
                else
                    tmem_load16(tmem + (quad * 32 << 16) + at, v);
            };
            load(j, a);
            if constexpr (MODE == kStats)
                for (uint32_t i = 1; i < used; ++i) {
                    float v[W];
                    load(i * g.bn + j, v);
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        a[k] += v[k];
                }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                a[i] = 0.f;
        }
        if (direct) {
            if constexpr (MODE == kGated)
                finish_gated(g.e, a, r0 + j, n, c, col_ok, bias, lane);
            else if constexpr (MODE == kStats) {
                if (col_ok)
                    add_logits(g.e, a, n, scale, token - (int64_t)(r0 + j), c, p);
            } else if constexpr (MODE == kSlopes) {
                if (col_ok)
                    store_slopes(g.e, a, r0 + j, c, scale, slope.token - (int64_t)(g.e.first + r0 + j), slope);
            } else if (col_ok)
                finish(g.e, a, res, r0 + j, n, c, bias, scale_at<true>(g.e, r0 + j, scale));
        } else {
            keep_part(part, a, j, quad * 32 + lane);
        }
    }
    if (MODE == kStats && direct && col_ok)
        g.e.part[r0 / g.bn * g.cols + c] = make_float4(p.m, p.s, p.t, 0.f);
}

// block: this CTA's number among the product's
template <bool PMN, bool QMN, bool F8, int MODE>
__device__ __forceinline__ void split_tile(const CUtensorMap &pmap, const CUtensorMap &pmap2, const CUtensorMap &qmap,
                                           const GemmArgs &g, uint32_t block, uint8_t *smem_raw, GemmBars &s)
{
    // the CTAs that share a tile are g.split neighbours of the cluster, `base` the first of them
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, crank = cluster_rank();
    const uint32_t rank = crank & (g.split - 1), base = crank - rank;
    const uint32_t off = (kSmemHead - (smem_u32(smem_raw) & (kSmemHead - 1))) & (kSmemHead - 1);
    const uint32_t stage0 = smem_u32(smem_raw) + off;
    const uint32_t stage_bytes = kPBytes + g.bn * kTileBytes;
    const uint32_t tile = block / g.split;
    if (tile >= g.ptiles * g.qtiles) { // fills up the last cluster
        if (g.split > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    const uint64_t p0 = (uint64_t)(tile % g.ptiles) * kPCols<MODE>, q0 = (uint64_t)(tile / g.ptiles) * g.bn;
    const uint32_t kb0 = (uint32_t)((uint64_t)g.kblocks * rank / g.split);
    const uint32_t kb1 = (uint32_t)((uint64_t)g.kblocks * (rank + 1) / g.split);
    // kStats: the reduction in up to 256 / bn accumulators, a segment each
    const uint32_t segs = MODE == kStats ? min(g.bn < 64 ? 4u : 256u / g.bn, max(1u, (kb1 - kb0 + kSegment - 1) / kSegment)) : 1u;
    const uint32_t tcols = MODE == kStats ? max(32u, g.bn * (segs == 3 ? 4 : segs)) : g.bn < 32 ? 32 : g.bn;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < g.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(&s.tfull[0], 1);
        fence_mbar_init();
        fence_proxy_async();
    }
    if (threadIdx.x == 32 && g.kblocks) {
        prefetch_map(&pmap);
        if constexpr (MODE == kGated || MODE == kDual)
            prefetch_map(&pmap2);
        prefetch_map(&qmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), tcols);
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&s.tmem;
    begin(g);

    const uint32_t quad = warp & 3;
    const uint32_t c = column_of<MODE>((uint32_t)p0, quad, lane);
    const bool col_ok = c < g.cols;
    float bias = 0.f;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!(ok = mbar_wait(&s.empty[st], ph ^ 1, g.limit_ns)))
                    break;
                const uint32_t at = stage0 + st * stage_bytes;
                mbar_expect_tx(&s.full[st], stage_bytes);
                load_p<1, PMN, F8, MODE>(at, &pmap, &pmap2, p0, kb, g, smem_u32(&s.full[st]));
                load_operand<1, QMN, F8>(at + kPBytes, &qmap, q0, g.bn, kb, g.qwide, smem_u32(&s.full[st]));
                if (++st == g.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) {
                set_status(g.status, ECC_ERR_TIMEOUT);
                for (uint32_t i = 0; i < g.stages; ++i) { // the copies in flight: a last wait each
                    if (st == 0) {
                        st = g.stages;
                        ph ^= 1;
                    }
                    --st;
                    (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && kb1 > kb0) {
            uint32_t st = 0, ph = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!(ok = mbar_wait(&s.full[st], ph, g.limit_ns))) {
                    (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                    break;
                }
                tmem_fence_after();
                const uint32_t at = stage0 + st * stage_bytes;
                if constexpr (MODE == kStats) {
                    const uint32_t per = (kb1 - kb0 + segs - 1) / segs, i = (kb - kb0) / per;
                    multiply_block<1, PMN, QMN, F8>(tmem + i * g.bn, at, at + kPBytes, g.idesc, kb == kb0 + i * per);
                } else {
                    multiply_block<1, PMN, QMN, F8>(tmem, at, at + kPBytes, g.idesc, kb == kb0);
                }
                tensor_commit<1>(smem_u32(&s.empty[st]));
                if (++st == g.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            tensor_commit<1>(smem_u32(&s.tfull[0]));
            if (!ok)
                set_status(g.status, ECC_ERR_TIMEOUT);
        }
    } else {
        bias = bias_of<MODE>(g.e, c, col_ok, lane);
        auto wait = [&] {
            ok = __all_sync(~0u, mbar_wait(&s.tfull[0], 0, g.limit_ns));
            if (!ok && lane == 0)
                set_status(g.status, ECC_ERR_TIMEOUT);
            tmem_fence_after();
            return ok;
        };
        // accumulators in use
        const uint32_t per = (kb1 - kb0 + segs - 1) / segs, used = per ? (kb1 - kb0 + per - 1) / per : 1;
        // once every product of this CTA is complete, the stages' memory holds its part
        float *part = reinterpret_cast<float *>(smem_raw + off);
        if (g.bn == 16)
            split_columns<16, MODE>(g, tmem, quad, lane, c, q0, col_ok, bias, g.split == 1, part, used, wait);
        else
            split_columns<32, MODE>(g, tmem, quad, lane, c, q0, col_ok, bias, g.split == 1, part, used, wait);
        tmem_fence_before();
    }
    __syncwarp();
    if (g.split > 1) {
        cluster_sync(); // all parts are written
        if (warp >= 2)
            join_parts<MODE>(g, stage0 + (quad * 32 + lane) * 4, base, rank, q0, c, lane);
        __syncwarp();
        cluster_sync(); // nobody reads this CTA's part any more
    } else {
        __syncthreads();
        __syncwarp();
    }
    tmem_fence_after();
    if (warp == 1)
        tmem_free<1>(tmem, tcols);
}

template <bool PMN, bool QMN, bool F8, int MODE>
__global__ void __launch_bounds__(kSplitThreads, 2)
    gemm_split_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap pmap2,
                      const __grid_constant__ CUtensorMap qmap, const __grid_constant__ GemmArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    split_tile<PMN, QMN, F8, MODE>(pmap, pmap2, qmap, g, blockIdx.x, smem_raw, s);
}

// A layer's two backward products in one launch: the first `n1` CTAs work on
// dx (w down its columns, t along its rows), the others on dw (both down
// their columns).  For layers whose products leave SMs idle: one after the
// other they took 22 us for 100 x 1000 x 1000, of which the kernels' starts and
// ends are most.  MODE: dx's.
template <int MODE>
__global__ void __launch_bounds__(kSplitThreads, 2)
    gemm_both_kernel(const __grid_constant__ CUtensorMap p1, const __grid_constant__ CUtensorMap p12,
                     const __grid_constant__ CUtensorMap q1, const __grid_constant__ GemmArgs g1,
                     const __grid_constant__ CUtensorMap p2, const __grid_constant__ CUtensorMap q2,
                     const __grid_constant__ GemmArgs g2, uint32_t n1)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    if (blockIdx.x < n1)
        split_tile<true, false, false, MODE>(p1, p12, q1, g1, blockIdx.x, smem_raw, s);
    else
        split_tile<true, true, false, kPlain>(p2, p2, q2, g2, blockIdx.x - n1, smem_raw, s);
}

template <bool PMN, bool QMN, bool F8, int MODE> const void *gemm_kernel(bool pair)
{
    return pair ? (const void *)gemm_pair_kernel<PMN, QMN, F8, MODE> : (const void *)gemm_split_kernel<PMN, QMN, F8, MODE>;
}

} // namespace ecc
