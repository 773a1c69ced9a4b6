// What the kernels on the vocabulary head share: tensor memory and tcgen05
// products fed by TMA, the soft cap of scores, and their tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"

namespace tsa {

constexpr float kLog2eH = 1.4426950408889634f;

// (m, Z) of two parts against the larger maximum; c2 = log2(e) / T.  An empty
// part is (-inf, 0).
__device__ __forceinline__ float2 lm_join(float2 a, float2 b, float c2) {
    const bool up = b.x > a.x;
    const float2 hi = up ? b : a, lo = up ? a : b;
    const float f = hi.x == lo.x ? 1.f : ex2_approx(fmaxf((lo.x - hi.x) * c2, -1.0e4f));
    return make_float2(hi.x, fmaf(lo.y, f, hi.y));
}
// cap tanh(z / cap), within 2^-21 of itself for every cap.  With x = z / cap:
//   |x| <= 5/8  z P(x^2), P a polynomial of degree 5 with P(0) = 1, fitted to equal relative error (Remez's exchange;
//               with its coefficients in fp32 within 2^-26 of tanh(x) / x).
//   else        cap (1 - 2 / (1 + e^(2 |x|))) with z's sign.  Near x = 0 that difference is off by 2^-23 of the cap, not of
//               the score: 6e-5 at a score of 3 and a cap of 1,000, and 8e-3 at a cap of 100,000.
// Scores of a model rarely pass 5/8 of the cap, and the polynomial needs no exponential and no division: 2,048 rows x
// 130,000 x 256 at a cap of 30 309 us, 198 us without a cap (336 us with the second form alone).  With every thread's
// scores on both sides (cap 8) it is 456 us, and 1,681 instead of 1,630 us for 128,256 x 5,120.
struct Cap {
    float cap, inv, k, bend;  // 1 / cap, 2 log2(e) / cap, 5/8 cap
};
__device__ __forceinline__ Cap make_cap(float cap) {
    const float inv = cap > 0.f ? fminf(1.f / cap, 3.4028234e38f) : 0.f;
    return Cap{cap, inv, inv * (2.f * kLog2eH), 0.625f * cap};
}
constexpr float kCap1 = -0.3333328068256378f, kCap2 = 0.13331441581249237f, kCap3 = -0.05373971536755562f,
                kCap4 = 0.0206390880048275f, kCap5 = -0.005704986862838268f;
__device__ __forceinline__ void cap_near(float &a, float &b, const Cap &c) {
    const auto both = [](float x) { return pair_of(x, x); };
    const unsigned long long z = pair_of(a, b), x = mul2(z, both(c.inv)), s = mul2(x, x);
    unsigned long long p = fma2(both(kCap5), s, both(kCap4));
    p = fma2(fma2(fma2(p, s, both(kCap3)), s, both(kCap2)), s, both(kCap1));
    split_pair(mul2(z, fma2(p, s, both(1.f))), a, b);
}
// n scores, a multiple of 8.
template <int n>
__device__ __forceinline__ void soft_cap(float *z, const Cap &c) {
    float top = 0.f;
#pragma unroll
    for (int q = 0; q < n; ++q) top = fmaxf(top, fabsf(z[q]));
    if (top > c.bend) {
        // eight at a time, in this order: all at once they do not fit the registers
#pragma unroll
        for (int g = 0; g < n; g += 8) {
            float u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(u[q]) : "f"(fabsf(z[g + q]) * c.k));
#pragma unroll
            for (int q = 0; q < 8; ++q)
                asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(u[q]) : "f"(fmaf(0.5f, u[q], 0.5f)));
#pragma unroll
            for (int q = 0; q < 8; ++q) u[q] = copysignf(fmaf(-c.cap, u[q], c.cap), z[g + q]);
#pragma unroll
            for (int q = 0; q < 8; q += 2) {
                float a = z[g + q], b = z[g + q + 1];
                cap_near(a, b, c);
                z[g + q] = fabsf(z[g + q]) > c.bend ? u[q] : a;
                z[g + q + 1] = fabsf(z[g + q + 1]) > c.bend ? u[q + 1] : b;
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < n; q += 2) cap_near(z[q], z[q + 1], c);
    }
}

// ------------------------------------------------------------ tensor memory
// tcgen05 (PTX ISA): one thread issues D[128, N] += A[128, 16] B[N, 16]^T from
// two shared-memory tiles into tensor memory; a warp reads its 32 lanes of D.
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void mma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrive on `bar` once every MMA this thread has issued so far is complete.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// The same by P CTAs of a cluster together (P = 2: each holds 128 of the 256 rows
// of A and D, and half of B's; the first one issues, from the same places in
// both, and tells both).
template <int P>
__device__ __forceinline__ void tmem_alloc_by(uint32_t *slot, uint32_t cols) {
    if constexpr (P == 1) {
        tmem_alloc(slot, cols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int P>
__device__ __forceinline__ void tmem_free_by(uint32_t addr, uint32_t cols) {
    if constexpr (P == 1)
        tmem_free(addr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
template <int P>
__device__ __forceinline__ void mma_bf16_by(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (P == 1)
        mma_bf16(d, a, b, idesc, add);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
template <int P>
__device__ __forceinline__ void mma_commit_by(uint64_t *bar) {
    if constexpr (P == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}
// To this CTA alone: nothing arrives at one that may be gone.
template <int P>
__device__ __forceinline__ void mma_commit_own(uint64_t *bar) {
    if constexpr (P == 1)
        mma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
}
template <int N> struct TmemLoad;
template <> struct TmemLoad<16> {
    __device__ static __forceinline__ void ld(uint32_t a, uint32_t (&r)[16]) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(a)
            : "memory");
    }
};
template <> struct TmemLoad<32> {
    __device__ static __forceinline__ void ld(uint32_t a, uint32_t (&r)[32]) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
              "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
              "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(a)
            : "memory");
    }
};
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A tile of 64 bf16 columns, 128 bytes a row, as TMA writes it with the
// 128-byte swizzle: rows follow one another, eight rows (1,024 bytes) repeat
// the pattern, K is contiguous.  The 16 columns of step k start 32 k bytes in.
__device__ __forceinline__ uint64_t smem_tile(const void *p) {
    return ((uint64_t)(smem_u32(p) >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// The same tile where M or N is contiguous in memory: boxes of 64 of it by K
// rows of 128 bytes, `box` bytes each, side by side.  The 16 K rows of step k
// start 2,048 k bytes in.
__device__ __forceinline__ uint64_t smem_tile_across(const void *p, uint32_t box) {
    return ((uint64_t)(smem_u32(p) >> 4) & 0x3FFFu) | ((uint64_t)(box >> 4) << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}
// A box of shared memory to global memory; the part outside the map is left out.
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read their source / are finished.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *map, int32_t x, int32_t y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_tile_3d(void *dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Copies whose barrier, given by its address in the cluster, may be in the first
// CTA of the pair.
template <int P>
__device__ __forceinline__ void tma_tile_by(void *dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    if constexpr (P == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                "r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int P>
__device__ __forceinline__ void tma_blocks_by(void *dst, const CUtensorMap *map, int32_t y, int32_t z, uint32_t bar) {
    if constexpr (P == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
                "r"(smem_u32(dst)),
            "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// ------------------------------------------------------------ tensor maps
constexpr int kTcK = 64;  // bf16 columns of a tile: 128 bytes

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encoder() {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return (EncodeFn) nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}

// bf16 [rows, cols] with `stride` elements a row, in boxes of 64 columns.
inline bool make_map(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t stride, int box_rows) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {kTcK, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same seen as blocks of 64 columns, [cols / 64][rows][64], cols a multiple
// of 64: a box is box_rows rows of `blocks` of them, one block after another.
inline bool make_map_blocks(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t stride, int box_rows,
                            int blocks) {
    const EncodeFn fn = encoder();
    if (!fn || cols % kTcK != 0) return false;
    const cuuint64_t dims[3] = {kTcK, (cuuint64_t)rows, (cuuint64_t)(cols / kTcK)};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, kTcK * 2};
    const cuuint32_t box[3] = {kTcK, (cuuint32_t)box_rows, (cuuint32_t)blocks}, step[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 152;
    return n;
}

}  // namespace tsa
