// ecc_tensor.cuh -- the tensor-core building blocks of the matrix products:
// tiled TMA loads, tcgen05 products into tensor memory, their barriers.
//
// Both operands lie in shared memory in the 128-byte swizzle, in chunks whose
// rows are 128 bytes.  "K-major": a row is one matrix row's next 128 bytes
// along the reduction; 8 rows (1024 bytes) form an atom, atoms follow each
// other, and a product step (32 bytes of the reduction) starts 32 bytes
// further.  "MN-major" (16-bit types): a row is one reduction index's 64
// consecutive matrix rows; 8 reduction indices form an atom, a chunk holds
// 64 of them, chunks of 64 matrix rows follow each other, and a step of 16
// reduction indices starts 2048 bytes further.
#pragma once

#include <cuda.h>

#include "ecc_device.cuh"
#include "ecc_lm.cuh"

namespace ecc {

constexpr uint32_t kTileBytes = 128; // reduction bytes of a stage (a swizzled row)

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of the same shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// (Release at the CTA's scope: what the arrival publishes is that tensor memory
// has been read, which the tcgen05 fences order.  At the cluster's scope it
// would wait for all of the warp's global stores: 8192 x 16384 x 64 took 107 us.)
__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float cluster_load(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// box at (x, y) of a 2-D tensor map -> dst; bytes counted on bar (with CG = 2
// a barrier of either CTA of the pair)
template <int CG> __device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(y), "r"(bar)
                     : "memory");
}
// box at (0, y, z) of a 3-D map
template <int CG> __device__ __forceinline__ void tma_load_groups(uint32_t dst, const CUtensorMap *map, int y, int z, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                     "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                     "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
                     : "memory");
}
// box at (x, 0, 0, z) of a 4-D map
template <int CG> __device__ __forceinline__ void tma_load_turns(uint32_t dst, const CUtensorMap *map, int x, int z, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %3, %4}], [%5];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(0), "r"(z), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %3, %4}], [%5];" ::"r"(dst),
                     "l"(map), "r"(x), "r"(0), "r"(z), "r"(bar)
                     : "memory");
}
// shared memory -> box at (x, y); tma_stores_commit ends a group of a thread's copies
__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all but the last N groups of this thread have read their shared memory
template <int N> __device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

template <int CG> __device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if constexpr (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int CG> __device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if constexpr (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes (one lane a thread), complete on return
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}
// 16 columns
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

// 16 columns added to v (in one block of assembly, so that no more than 16
// loaded values are held at a time)
__device__ __forceinline__ void tmem_add16(uint32_t addr, float2 *v)
{
    asm volatile("{\n\t.reg .b32 t<16>;\n\t.reg .b64 u<8>;\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;\n\t"
                 "mov.b64 u0, {t0, t1};\n\t"
                 "mov.b64 u1, {t2, t3};\n\t"
                 "mov.b64 u2, {t4, t5};\n\t"
                 "mov.b64 u3, {t6, t7};\n\t"
                 "mov.b64 u4, {t8, t9};\n\t"
                 "mov.b64 u5, {t10, t11};\n\t"
                 "mov.b64 u6, {t12, t13};\n\t"
                 "mov.b64 u7, {t14, t15};\n\t"
                 "add.rn.f32x2 %0, %0, u0;\n\t"
                 "add.rn.f32x2 %1, %1, u1;\n\t"
                 "add.rn.f32x2 %2, %2, u2;\n\t"
                 "add.rn.f32x2 %3, %3, u3;\n\t"
                 "add.rn.f32x2 %4, %4, u4;\n\t"
                 "add.rn.f32x2 %5, %5, u5;\n\t"
                 "add.rn.f32x2 %6, %6, u6;\n\t"
                 "add.rn.f32x2 %7, %7, u7;\n\t"
                 "}"
                 : "+l"(reinterpret_cast<unsigned long long &>(v[0])), "+l"(reinterpret_cast<unsigned long long &>(v[1])), "+l"(reinterpret_cast<unsigned long long &>(v[2])), "+l"(reinterpret_cast<unsigned long long &>(v[3])), "+l"(reinterpret_cast<unsigned long long &>(v[4])), "+l"(reinterpret_cast<unsigned long long &>(v[5])), "+l"(reinterpret_cast<unsigned long long &>(v[6])), "+l"(reinterpret_cast<unsigned long long &>(v[7]))
                 : "r"(addr)
                 : "memory");
}

// Shared-memory operand descriptor: start address, the strides of the layout
// above, descriptor version 1, 128-byte swizzle.  K-major: 1024 bytes between
// groups of 8 rows (the other stride is unused).  MN-major: 1024 bytes
// between groups of 8 reduction indices, `chunk` bytes between groups of 64
// matrix rows.
template <bool MN> __device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t chunk)
{
    const uint64_t lbo = MN ? (uint64_t)(chunk >> 4) : 1ull;
    return (uint64_t)((addr >> 4) & 0x3FFF) | lbo << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// descriptor step between products of a stage, in its 16-byte units
template <bool MN> __device__ constexpr uint32_t operand_step() { return MN ? 2048 / 16 : 32 / 16; }

// D[tmem] (+)= A B^T, issued by one thread
template <int CG, bool F8>
__device__ __forceinline__ void tensor_product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
#define ECC_MMA(cg, kind)                                                                                              \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"                                                     \
                 "tcgen05.mma.cta_group::" cg ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                    \
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)                                                 \
                 : "memory")
    if constexpr (CG == 2 && F8)
        ECC_MMA("2", "f8f6f4");
    else if constexpr (CG == 2)
        ECC_MMA("2", "f16");
    else if constexpr (F8)
        ECC_MMA("1", "f8f6f4");
    else
        ECC_MMA("1", "f16");
#undef ECC_MMA
}
// the barrier (of both CTAs of a pair) gets one arrival when this thread's
// products so far are complete
template <int CG> __device__ __forceinline__ void tensor_commit(uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Instruction descriptor: float32 accumulator, operand types (16-bit kinds: 0
// f16, 1 bf16; 8-bit kind: 0 e4m3), operand layouts, tile size m x n.
inline uint32_t product_desc(uint32_t type, bool a_mn, bool b_mn, uint32_t m, uint32_t n)
{
    const uint32_t t = type == ECC_BF16 ? 1u : 0u;
    return 1u << 4 | t << 7 | t << 10 | (a_mn ? 1u : 0u) << 15 | (b_mn ? 1u : 0u) << 16 | (n >> 3) << 17 | (m >> 4) << 24;
}

} // namespace ecc
