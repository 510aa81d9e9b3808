// ecc_head.cu -- log probabilities of tokens straight from hidden states and a
// language model's head, and their gradient, without the logits in memory.
//
// Forward: one matrix product whose epilogue keeps a token's running maximum,
// sum and entropy sum over a share of the vocabulary (ecc_gemm.cuh, kStats),
// and a kernel that joins the shares.  Backward, for a piece of the vocabulary
// at a time: the logits again, their gradient t written as the next products'
// operand (kSlopes), then dx += t w and dw = t^T x.  The pieces bound the
// workspace.
//
// Forward: 4096 x 50021 x 4096 bf16 0.90 ms in a burst (1.86 PFLOP/s), 1.03 ms
// under the power limit; 8 x 131072 x 4096 173 us (6.2 TB/s).  Backward: 4096 x
// 131072 x 2048 3.56 ms in a burst, 4.03 ms under the power limit (1.64 PFLOP/s).

#include <cmath>

#include "ecc_linear.cuh"

namespace ecc {

constexpr int kJoinThreads = 256;

struct JoinParams {
    const float4 *part; // [parts][rows]
    const float *token_logit;
    const int64_t *tokens;
    uint64_t rows, vocab;
    uint32_t parts, each; // rows of a block: a power of two
    float *logprob, *entropy, *lse;
};

__device__ __forceinline__ float4 join_two(const float4 &a, const float4 &b)
{
    if (b.y == 0.f) // an empty share
        return a;
    if (a.y == 0.f)
        return b;
    const float m = fmaxf(a.x, b.x), da = a.x - m, db = b.x - m, ra = exp2f(da), rb = exp2f(db);
    return make_float4(m, a.y * ra + b.y * rb, ra * fmaf(da, a.y, a.z) + rb * fmaf(db, b.y, b.z), 0.f);
}

// a row's shares over kJoinThreads / each threads, joined in a fixed order
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ JoinParams p)
{
    __shared__ float4 s[kJoinThreads];
    wait_for_previous();
    const uint32_t at = threadIdx.x & (p.each - 1), lane = threadIdx.x / p.each, lanes = kJoinThreads / p.each;
    const uint64_t row = (uint64_t)blockIdx.x * p.each + at;
    float4 v = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (row < p.rows)
#pragma unroll 4
        for (uint32_t k = lane; k < p.parts; k += lanes)
            v = join_two(v, p.part[k * p.rows + row]);
    s[threadIdx.x] = v;
    for (uint32_t n = lanes / 2; n; n /= 2) {
        __syncthreads();
        if (lane < n)
            s[threadIdx.x] = v = join_two(v, s[threadIdx.x + n * p.each]);
    }
    if (lane || row >= p.rows)
        return;
    const float logs = log2f(v.y), bad = v.z != v.z ? v.z : 0.f; // a logit that is not finite: NaN everywhere
    if (p.lse)
        p.lse[row] = (v.x + logs) * 0.69314718f + bad;
    if (p.entropy)
        p.entropy[row] = (logs - v.z / v.y) * 0.69314718f;
    if (p.logprob && p.tokens) {
        const int64_t t = p.tokens[row];
        p.logprob[row] = t < 0                  ? 0.f
                         : t >= (int64_t)p.vocab ? __int_as_float(0x7FC00000)
                                                 : ((p.token_logit[row] - v.x) - logs) * 0.69314718f + bad;
    }
}

// f[0] = 2^k, f[1] = 2^-k: t's magnitudes are at most max(|dlogprob| + |dentropy|
// (log p + H) p), the latter below 16, and f[0] brings that to 2^14, so that a
// float16 t keeps probabilities down to 2^-28 of it to 10 bits.  Only what t is
// made of counts: no dlogprob of a row without a token, whatever it holds, and
// no row whose t is not finite (dx of the other rows is).
__global__ void __launch_bounds__(1024)
    factor_kernel(const float *dlogprob, const float *dentropy, const int64_t *tokens, uint64_t rows, uint64_t vocab, float *f)
{
    __shared__ float s[32];
    let_next_start();
    float top = 0.f;
    for (uint64_t i = threadIdx.x; i < rows; i += 1024) {
        const bool has = dlogprob && tokens && tokens[i] >= 0 && tokens[i] < (int64_t)vocab;
        const float most = (has ? fabsf(dlogprob[i]) : 0.f) + (dentropy ? 16.f * fabsf(dentropy[i]) : 0.f);
        top = fmaxf(top, most < INFINITY ? most : 0.f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = s[threadIdx.x];
#pragma unroll
        for (int o = 16; o; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const int k = half_power(top);
        if (threadIdx.x < 2)
            f[threadIdx.x] = ldexpf(1.f, threadIdx.x ? -k : k);
    }
    // (launched behind the padding: whatever waits for this kernel waits for both)
    wait_for_previous();
}

namespace {

// Bytes of t for a piece of the vocabulary: pieces of 8192 tokens and more for
// up to 16384 rows, so that dx's sum in float32 (8 bytes a value for each piece)
// is a few percent of what the products move.
constexpr size_t kPieceBytes = 256ull << 20;

constexpr float kMostScale = 0x1p127f; // times log2 e it is finite

bool head_ok(const ecc_linear_logprob_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16 && j.in_type != ECC_E4M3) || !(std::fabs(j.scale) < kMostScale) || j.rows >= kMostDim ||
        !j.vocab || j.vocab >= kMostDim || j.K >= kMostDim || j.reserved)
        return false;
    if (!j.rows)
        return true;
    if (j.K && (!j.x || !j.w || j.ldx < j.K || j.ldw < j.K || !aligned_to(j.x, j.in_type) || !aligned_to(j.w, j.in_type)))
        return false;
    return ((uintptr_t)j.tokens & 7) == 0 && aligned_to(j.logprob, ECC_F32) && aligned_to(j.entropy, ECC_F32) &&
           aligned_to(j.lse, ECC_F32);
}
Product head_product(const ecc_linear_logprob_job &j)
{
    Product p{};
    p.P = {j.x, j.ldx, false};
    p.Q = {j.w, j.ldw, false};
    p.rows = j.vocab;
    p.cols = j.rows;
    p.K = j.K;
    p.mode = kStats;
    p.e.scale = j.scale;
    p.e.tokens = j.tokens;
    return p;
}

bool head_grad_ok(const ecc_linear_logprob_grad_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16) || !(std::fabs(j.scale) < kMostScale) || j.rows >= kMostDim || !j.vocab ||
        j.vocab >= kMostDim || j.K >= kMostDim || j.reserved || (j.dw && j.dw_type != j.in_type && j.dw_type != ECC_F32))
        return false;
    if (j.rows && (!j.lse || !aligned_to(j.lse, ECC_F32) || (j.dentropy && !j.entropy) || !aligned_to(j.entropy, ECC_F32) ||
                   !aligned_to(j.dlogprob, ECC_F32) || !aligned_to(j.dentropy, ECC_F32) || ((uintptr_t)j.tokens & 7)))
        return false;
    if (j.rows && j.K && (!j.x || !j.w || j.ldx < j.K || j.ldw < j.K || !aligned_to(j.x, j.in_type) || !aligned_to(j.w, j.in_type)))
        return false;
    if (j.dx && j.rows && j.K && (j.lddx < j.K || !aligned_to(j.dx, j.in_type)))
        return false;
    return !j.dw || !j.K || (j.lddw >= j.K && aligned_to(j.dw, j.dw_type));
}

struct HeadGradPlan {
    uint64_t piece; // of the vocabulary: a multiple of 256, or all of it
    uint64_t ldt;
    size_t t_bytes, sum_bytes, bytes;
};
HeadGradPlan head_grad_plan(const ecc_linear_logprob_grad_job &j)
{
    HeadGradPlan g{};
    const uint64_t most = std::max<uint64_t>(256, kPieceBytes / 2 / std::max<uint64_t>(j.rows, 1) / 256 * 256);
    const uint64_t pieces = (j.vocab + most - 1) / most;
    g.piece = pieces == 1 ? j.vocab : (((j.vocab + pieces - 1) / pieces) + 255) / 256 * 256;
    g.ldt = (g.piece + 63) / 64 * 64;
    g.t_bytes = pad256(j.rows * g.ldt * 2);
    g.sum_bytes = j.dx && g.piece < j.vocab ? pad256(j.rows * j.K * sizeof(float)) : 0;
    g.bytes = 256 + g.t_bytes + g.sum_bytes + copy_bytes(j.x, j.ldx, j.rows, j.K, j.in_type) +
              copy_bytes(j.w, j.ldw, j.vocab, j.K, j.in_type);
    return g;
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

size_t ecc_linear_logprob_workspace_bytes(const ecc_linear_logprob_job *job)
{
    if (!job || !job->rows || !head_ok(*job))
        return 0;
    const ecc_linear_logprob_job &j = *job;
    return pad256(j.rows * sizeof(float)) + pad256((size_t)stats_parts(head_product(j), j.in_type) * j.rows * sizeof(float4)) +
           copy_bytes(j.x, j.ldx, j.rows, j.K, j.in_type) + copy_bytes(j.w, j.ldw, j.vocab, j.K, j.in_type);
}

ecc_status ecc_linear_logprob(const ecc_linear_logprob_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !head_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_logprob_job &j = *job;
    cudaStream_t st = (cudaStream_t)stream;
    if (!j.rows)
        return launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    if (!ws || !aligned16(ws) || ws_bytes < ecc_linear_logprob_workspace_bytes(job))
        return ECC_ERR_ARG;
    uint8_t *w = (uint8_t *)ws;
    Product p = head_product(j);
    const uint32_t parts = stats_parts(p, j.in_type);
    p.e.token_logit = (float *)w;
    w += pad256(j.rows * sizeof(float));
    p.e.part = (float4 *)w;
    w += pad256((size_t)parts * j.rows * sizeof(float4));
    bool copied;
    ecc_status rc = readable({{j.x, j.ldx, j.rows, j.K, &p.P}, {j.w, j.ldw, j.vocab, j.K, &p.Q}}, j.in_type, w, st, copied);
    if (rc == ECC_OK)
        rc = gemm(p, j.in_type, status, true, copied, st);
    if (rc != ECC_OK)
        return rc;
    uint32_t each = 1; // rows of a joining block: as many as leave a block an SM
    while (each < 32 && 2 * each * (uint64_t)sms <= j.rows)
        each *= 2;
    const JoinParams join{p.e.part, p.e.token_logit, j.tokens, j.rows, j.vocab, parts, each, j.logprob, j.entropy, j.lse};
    return launch_status(launch_behind(join_kernel, dim3((unsigned)((j.rows + each - 1) / each)), kJoinThreads, 0, st, join));
}

size_t ecc_linear_logprob_grad_workspace_bytes(const ecc_linear_logprob_grad_job *job)
{
    return job && head_grad_ok(*job) ? head_grad_plan(*job).bytes : 0;
}

ecc_status ecc_linear_logprob_grad(const ecc_linear_logprob_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !head_grad_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_logprob_grad_job &j = *job;
    const HeadGradPlan g = head_grad_plan(j);
    cudaStream_t st = (cudaStream_t)stream;
    if (!ws || !aligned16(ws) || ws_bytes < g.bytes)
        return ECC_ERR_ARG;
    const bool want_dx = j.dx && j.rows && j.K, want_dw = j.dw && j.K;
    if (!want_dx && !want_dw)
        return launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    uint8_t *at = (uint8_t *)ws;
    float *factor = j.in_type == ECC_F16 ? (float *)at : nullptr;
    at += 256;
    void *t = at;
    at += g.t_bytes;
    void *sum = at;
    at += g.sum_bytes;
    Operand x, w;
    bool behind;
    ecc_status rc = readable({{j.x, j.ldx, j.rows, j.K, &x}, {j.w, j.ldw, j.vocab, j.K, &w}}, j.in_type, at, st, behind);
    if (rc != ECC_OK)
        return rc;
    if (factor) {
        // (as the call's first launch it starts after the one before it has ended, which may read this workspace)
        cudaError_t e = cudaSuccess;
        if (behind) {
            e = launch_behind(factor_kernel, dim3(1), 1024, 0, st, j.dlogprob, j.dentropy, j.tokens, j.rows, j.vocab, factor);
        } else {
            factor_kernel<<<1, 1024, 0, st>>>(j.dlogprob, j.dentropy, j.tokens, j.rows, j.vocab, factor);
            e = cudaGetLastError();
        }
        if ((rc = launch_status(e)) != ECC_OK)
            return rc;
        behind = true;
    }
    bool clear = true;
    for (uint64_t v = 0; rc == ECC_OK && v < j.vocab; v += g.piece) {
        const uint64_t n = std::min(g.piece, j.vocab - v);
        const Operand piece{(const uint8_t *)w.p + v * w.ld * 2, w.ld, false};
        if (j.rows) {
            Product s{};
            s.P = x;
            s.Q = piece;
            s.rows = n;
            s.cols = j.rows;
            s.K = j.K;
            s.mode = kSlopes;
            s.e.scale = j.scale;
            s.e.out = t;
            s.e.ldout = g.ldt;
            s.e.out_type = j.in_type;
            s.e.tokens = j.tokens;
            s.e.first = v;
            s.e.lse = j.lse;
            s.e.entropy = j.entropy;
            s.e.dlogprob = j.dlogprob;
            s.e.dentropy = j.dentropy;
            s.e.vocab = j.vocab;
            s.e.factor = factor;
            rc = gemm(s, j.in_type, status, clear, behind, st);
            clear = false;
            behind = true;
        }
        Product dx{}, dw{};
        dx.P = {piece.p, piece.ld, true};
        dx.Q = {t, g.ldt, false};
        dx.rows = j.rows;
        dx.cols = j.K;
        dx.K = n;
        const bool last = v + n == j.vocab;
        dx.e.residual = v ? sum : nullptr; // the pieces before
        dx.e.ldres = j.K;
        dx.e.res_type = ECC_F32;
        dx.e.out = last ? j.dx : sum;
        dx.e.ldout = last ? j.lddx : j.K;
        dx.e.out_type = last ? j.in_type : (uint32_t)ECC_F32;
        dw.P = {x.p, x.ld, true};
        dw.Q = {t, g.ldt, true};
        dw.rows = n;
        dw.cols = j.K;
        dw.K = j.rows;
        dw.e.out = want_dw ? (uint8_t *)j.dw + v * j.lddw * type_bytes(j.dw_type) : nullptr;
        dw.e.ldout = j.lddw;
        dw.e.out_type = j.dw_type;
        dx.e.scale = dw.e.scale = j.scale;
        dx.e.out_scale = dw.e.out_scale = 1.f;
        dx.e.factor = dw.e.factor = factor ? factor + 1 : nullptr;
        if (rc == ECC_OK && want_dx && want_dw)
            rc = gemm_backward(dx, dw, j.in_type, status, clear, behind, st);
        else if (rc == ECC_OK)
            rc = gemm(want_dx ? dx : dw, j.in_type, status, clear, behind, st);
        clear = false;
        behind = true;
    }
    return rc;
}

} // extern "C"
