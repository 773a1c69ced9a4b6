// The head's scores from 8-bit integers with a scale for each hidden row and
// each vocabulary entry:
//     z[m, v] = hs[m] ws[v] sum_k h[m, k] w[v, k]  (+ b[v]),
// the sum over integers exact.
//
// The tensor cores of this GPU have next to no rate for 8-bit integers, but
// f16 holds every one of them exactly, and the fp32 sums of 1,024 of their
// products, at most 2^24 of them, are exact too.  So the weight, which is what
// there is most of, goes through memory in 8 bits and becomes f16 on the way
// into tensor memory; sums of 1,024 columns are added up as integers in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_tcgen05.cuh"

namespace tsa {

namespace {

__device__ unsigned int g_int8_status;

__device__ __forceinline__ bool int8_wait(uint64_t *bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, &g_int8_status);
}
__device__ __forceinline__ bool int8_warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, int8_wait(bar, parity));
}

// D[128, N] += A[128, 16] B[N, 16]^T with A in tensor memory: a lane a row,
// two f16 values a column.  B's descriptor comes in its two halves.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 x, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], x, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t a, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 8-bit integers as f16.  An f16 of bits 0x6400 | u is 1024 + u for u
// under 1024: with u = x + 128 what is left is to subtract 1152, exactly.
__device__ __forceinline__ void to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 k = __half2half2(__ushort_as_half((unsigned short)0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 p = __hsub2(*reinterpret_cast<__half2 *>(&a), k), q = __hsub2(*reinterpret_cast<__half2 *>(&b), k);
    lo = *reinterpret_cast<uint32_t *>(&p);
    hi = *reinterpret_cast<uint32_t *>(&q);
}

// The hidden rows in f16, their columns filled up to whole stages with zeros:
// 16 columns a thread.
__global__ void __launch_bounds__(256) int8_hidden_kernel(const Int8Args a) {
    pdl_launch_dependents();
    const int64_t padded = int8_padded(a.H), cols = padded / 16, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.M * cols) return;
    const int64_t m = i / cols, k = i % cols * 16;
    uint4 x = make_uint4(0, 0, 0, 0), y, z;
    if (k < a.H) x = *reinterpret_cast<const uint4 *>(a.hidden + m * a.hstride + k);
    to_f16(x.x, y.x, y.y);
    to_f16(x.y, y.z, y.w);
    to_f16(x.z, z.x, z.y);
    to_f16(x.w, z.z, z.w);
    uint4 *out = reinterpret_cast<uint4 *>(a.half + m * padded + k);
    out[0] = y;
    out[1] = z;
}

// One persistent CTA an SM.  Warp 0 fetches 128 columns of the weight's rows
// (a lane of tensor memory each) by TMA into one ring of stages, warp 2 the same
// columns of N hidden rows into another; four or eight warps turn the weight's bytes
// into f16 in four slots of tensor memory, groups of four taking steps in turn;
// warp 1 issues the products; four or eight warps take finished sums from one
// half of the accumulators while the next products fill the other half.
//
// Rings of their own: a stage of the weight is free as soon as it is in tensor
// memory, 700 cycles after it landed, and not after its products, 1,500 to 2,000
// cycles later; with one ring for both (112 KB of the weight under way) 16 rows x
// 128,256 x 5,120 took 134 us.
//
// Up to 128 hidden rows the kernel is a stream of the weight, and the vocabulary
// is cut into one run of rows a CTA, a multiple of 32, so that every SM moves
// the same bytes; a run's last tile copies only the rows that it needs.  With
// more hidden rows tiles go through those first, so that a weight tile comes from
// HBM once and from L2 for the other blocks.  V x H = 128,256 x 5,120: 16 rows 112
// us, 5.9 TB/s (88 % of a copy), 64 rows 117 us, 128 rows 142 us; 2,048 rows x 32,000
// x 4,096 376 us, 1,430 TFLOP/s, bound by copies from L2 and the conversions.
//
// A copy or product that one thread issues costs it some 100 cycles, ten times
// what it costs a warp that goes through its loop together: whole tiles are one
// copy each (with six a stage and single threads issuing, 16 rows took 235 us).
constexpr int kI8K = kInt8Stage;       // columns of a step
constexpr int kI8Chunk = 1024 / kI8K;  // steps whose sums are exact
constexpr int kI8Slots = 4;            // of the weight in tensor memory, 64 columns each

template <int N>
struct Int8Shape {
    static constexpr int A_BYTES = 128 * kI8K, B_BYTES = N * kI8K * 2;
    // Stages of the two rings; the weight's even, as two groups of warps take them in turn.  The hidden rows' copies
    // come from L2 but take longer, as all SMs ask for the same lines at once: 64 rows x 128,256 x 5,120 take 136 us
    // with ten stages and four, 120 with eight and six, and 128 rows 153 with six and four, 147 with four and five.
    static constexpr int A_STAGES = N <= 32 ? 10 : N == 64 ? 8 : 4;
    static constexpr int B_STAGES = N <= 16 ? 16 : N <= 64 ? 6 : 5;
    static_assert(A_STAGES % 2 == 0 && kI8Slots % 2 == 0, "a group of warps meets a stage in each of its phases");
    static constexpr int SMEM = A_STAGES * A_BYTES + B_STAGES * B_BYTES + 1024;
    static constexpr int EPI = N <= 32 ? 4 : 8;  // warps that take the sums
    static constexpr int NC = N <= 32 ? N : N / 2;
    // Groups of four warps that convert: one needs 600 to 700 cycles a step, and 128 rows' products take 1,000.
    static constexpr int GROUPS = N == 128 ? 1 : 2;
    static constexpr int THREADS = 128 + 128 * GROUPS + 32 * EPI;
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(N / 8) << 17) | (8u << 24);  // f16, fp32 sums, M = 128
};

// A warp's way round a ring: the stage, and the phase that it waits for.
template <int STAGES>
struct Int8Place {
    uint32_t s = 0, phase;
    __device__ __forceinline__ explicit Int8Place(uint32_t p) : phase(p) {}
    __device__ __forceinline__ void next() {
        if (++s == STAGES) s = 0, phase ^= 1u;
    }
};

template <int DT>
__device__ __forceinline__ void store_score(void *p, int64_t i, float x) {
    if constexpr (DT == 0)
        static_cast<float *>(p)[i] = x;
    else if constexpr (DT == 1)
        static_cast<__half *>(p)[i] = __float2half_rn(x);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

template <int N, int DT>
__global__ void __launch_bounds__(Int8Shape<N>::THREADS, 1)
    int8_scores_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_part,
                       const __grid_constant__ CUtensorMap map_h, const Int8Args a, int32_t row_blocks, int32_t tiles, int32_t run) {
    using S = Int8Shape<N>;
    constexpr int NA = S::A_STAGES, NB = S::B_STAGES, NC = S::NC;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t w_full[NA], w_empty[NA], h_full[NB], h_empty[NB], a_full[kI8Slots], a_empty[kI8Slots], done[2],
        drained[2], last;
    __shared__ uint32_t tmem_slot;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *ring_h = ring + NA * S::A_BYTES;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int steps = (int)((a.H + kI8K - 1) / kI8K);
    // run > 0: this CTA's vocabulary rows; else whole tiles, in turn
    const int32_t V = (int32_t)a.V, v_first = run > 0 ? (int32_t)blockIdx.x * run : 0;
    const int32_t v_end = run > 0 && v_first + run < V ? v_first + run : V;
    const int32_t t_first = run > 0 ? 0 : blockIdx.x, t_step = run > 0 ? 1 : gridDim.x;
    const int32_t t_end = run > 0 ? (v_end - v_first + 127) / 128 : tiles;
    const auto tile_v = [&](int32_t t) { return run > 0 ? v_first + t * 128 : t / row_blocks * 128; };
    const auto tile_m = [&](int32_t t) { return run > 0 ? 0 : t % row_blocks * N; };
    if (threadIdx.x == 0) {
        for (int i = 0; i < NA; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], 128);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&h_full[i], 1);
            mbar_init(&h_empty[i], 1);
        }
        for (int i = 0; i < kI8Slots; ++i) {
            mbar_init(&a_full[i], 128);
            mbar_init(&a_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&drained[i], 32 * S::EPI);
        }
        mbar_init(&last, 1);
        mbar_init_fence();
    }
    if (warp == 3) tmem_alloc(&tmem_slot, 512);
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    const uint32_t tmem = tmem_slot, slots = tmem + 256;

    if (warp == 0) {
        Int8Place<NA> at(1);
        uint32_t uses = 0;
        bool ok = true;
        for (int32_t t = t_first; ok && t < t_end; t += t_step) {
            const int32_t v = tile_v(t), left = v_end - v;
            for (int k = 0; k < steps; ++k, ++uses, at.next()) {
                ok = int8_warp_wait(&w_empty[at.s], at.phase);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t *st = ring + at.s * S::A_BYTES;
                    if (left > 96) {
                        mbar_arrive_expect_tx(&w_full[at.s], S::A_BYTES);
                        tma_tile(st, &map_w, k * kI8K, v, &w_full[at.s]);
                    } else {
                        const int groups = (left + 31) / 32;
                        mbar_arrive_expect_tx(&w_full[at.s], (uint32_t)(groups * (S::A_BYTES / 4)));
                        for (int i = 0; i < groups; ++i)
                            tma_tile(st + i * (S::A_BYTES / 4), &map_part, k * kI8K, v + 32 * i, &w_full[at.s]);
                    }
                }
                __syncwarp();
            }
        }
        // no copy may land after the CTA is gone
        for (uint32_t i = uses < NA ? 0 : uses - NA; i < uses; ++i) int8_warp_wait(&w_full[i % NA], (i / NA) & 1u);
    } else if (warp == 2) {
        pdl_wait_primary();  // (the weight does not wait for the kernel that makes the hidden rows)
        Int8Place<NB> at(1);
        uint32_t uses = 0;
        bool ok = true;
        for (int32_t t = t_first; ok && t < t_end; t += t_step) {
            const int32_t m = tile_m(t);
            for (int k = 0; k < steps; ++k, ++uses, at.next()) {
                ok = int8_warp_wait(&h_empty[at.s], at.phase);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&h_full[at.s], S::B_BYTES);
                    tma_tile_3d(ring_h + at.s * S::B_BYTES, &map_h, 0, m, 2 * k, &h_full[at.s]);
                }
                __syncwarp();
            }
        }
        for (uint32_t i = uses < NB ? 0 : uses - NB; i < uses; ++i)
            int8_warp_wait(ok ? &h_empty[i % NB] : &h_full[i % NB], (i / NB) & 1u);
    } else if (warp == 1) {
        Int8Place<kI8Slots> slot(0);
        Int8Place<NB> at(0);
        uint32_t j = 0, uses = 0;
        const uint64_t desc = smem_tile(ring_h);
        const uint32_t lo = (uint32_t)desc, hi = (uint32_t)(desc >> 32);
        bool ok = true, ready = false;
        for (int32_t t = t_first; ok && t < t_end; t += t_step) {
            for (int k = 0; k < steps; ++k) {
                const uint32_t b = j & 1u, s = at.s, l = slot.s;
                if (k % kI8Chunk == 0) ok = int8_warp_wait(&drained[b], ((j >> 1) & 1u) ^ 1u);
                ok = ok && (ready || (int8_warp_wait(&h_full[s], at.phase) && int8_warp_wait(&a_full[l], slot.phase)));
                if (!ok) break;
                mma_fence_after();
                // a look at the next step, whose answer comes while this one's products are issued
                at.next();
                slot.next();
                const bool seen = mbar_test_wait(&h_full[at.s], at.phase) && mbar_test_wait(&a_full[slot.s], slot.phase);
                const uint32_t d = tmem + b * 128, sa = slots + l * 64, sb = lo + s * (S::B_BYTES >> 4);
                const bool end = k % kI8Chunk == kI8Chunk - 1 || k == steps - 1;
                ++uses;
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        mma_f16_ts(d, sa + p * 8, sb + (p >> 2) * (S::B_BYTES / 2 >> 4) + (p & 3) * 2, hi, S::IDESC,
                                   k % kI8Chunk > 0 || p > 0);
                    mma_commit(&h_empty[s]);
                    mma_commit(&a_empty[l]);
                    if (end) mma_commit(&done[b]);
                }
                ready = __all_sync(0xFFFFFFFFu, seen);
                if (end) ++j;
            }
        }
        // no commit may arrive after the CTA is gone, and the products are finished before tensor memory is freed
        if (elect_one()) mma_commit(&last);
        int8_warp_wait(&last, 0);
        for (uint32_t i = uses < kI8Slots ? 0 : uses - kI8Slots; i < uses; ++i)
            int8_warp_wait(&a_empty[i % kI8Slots], (i / kI8Slots) & 1u);
    } else if (warp >= 4 && warp < 4 + 4 * S::GROUPS) {
        const int quarter = warp & 3, group = (warp - 4) >> 2;
        const uint32_t at = slots + ((uint32_t)quarter << 21);
        const int row = quarter * 32 + lane;
        uint32_t it = 0;
        bool ok = true;
        for (int32_t t = t_first; ok && t < t_end; t += t_step) {
            for (int k = 0; k < steps; ++k, ++it) {
                // The rings are even, so that a group sees every phase of the barriers that it waits for.  (A wait
                // for a phase passes while the one before it is open.)
                if (it % S::GROUPS != (uint32_t)group) continue;
                const uint32_t s = it % NA, l = it % kI8Slots;
                ok = int8_warp_wait(&w_full[s], (it / NA) & 1u) && int8_warp_wait(&a_empty[l], ((it / kI8Slots) & 1u) ^ 1u);
                if (!ok) break;
                mma_fence_after();
                const uint8_t *src = ring + s * S::A_BYTES + row * kI8K;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src + (((h * 4 + c) ^ (row & 7)) << 4));
                        to_f16(x.x, r[8 * c], r[8 * c + 1]);
                        to_f16(x.y, r[8 * c + 2], r[8 * c + 3]);
                        to_f16(x.z, r[8 * c + 4], r[8 * c + 5]);
                        to_f16(x.w, r[8 * c + 6], r[8 * c + 7]);
                    }
                    __syncwarp();
                    tmem_store(at + l * 64 + h * 32, r);
                }
                mbar_arrive(&w_empty[s]);
                tmem_wait_st();
                mma_fence_before();
                mbar_arrive(&a_full[l]);
            }
        }
    } else if (warp >= 4 + 4 * S::GROUPS) {
        const int quarter = warp & 3, half = (warp - 4 - 4 * S::GROUPS) >> 2;
        const uint32_t at = tmem + ((uint32_t)quarter << 21) + half * NC;
        const int chunks = (steps + kI8Chunk - 1) / kI8Chunk;
        uint32_t j = 0;
        bool ok = true;
        for (int32_t t = t_first; ok && t < t_end; t += t_step) {
            const int32_t v = tile_v(t) + quarter * 32 + lane, m0 = tile_m(t) + half * NC;
            const bool in = v < v_end;
            const float ws = in ? __ldg(a.wscale + v) : 0.f, bias = in && a.bias ? __ldg(a.bias + v) : 0.f;
            int sum[NC];  // (of one chunk the fp32 sums as they are, exact and whole)
            for (int c = 0; c < chunks; ++c, ++j) {
                const uint32_t b = j & 1u;
                ok = int8_warp_wait(&done[b], (j >> 1) & 1u);
                if (!ok) break;
                mma_fence_after();
#pragma unroll
                for (int q = 0; q < NC; q += 16) {
                    uint32_t r[16];
                    __syncwarp();
                    TmemLoad<16>::ld(at + b * 128 + q, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (chunks == 1)
                            sum[q + i] = (int)r[i];
                        else
                            sum[q + i] = (c == 0 ? 0 : sum[q + i]) + __float2int_rn(__uint_as_float(r[i]));
                    }
                }
                mma_fence_before();
                mbar_arrive(&drained[b]);
            }
            if (!ok) break;
#pragma unroll
            for (int q0 = 0; q0 < NC; q0 += 16) {
                // a lane brings one row's scale, and every lane gets them in turn
                const int32_t m = m0 + q0, rows = (int32_t)min((int64_t)16, a.M - m);
                const float hs = lane < rows ? __ldg(a.hscale + m + lane) : 0.f;
                float z[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float x = chunks == 1 ? __int_as_float(sum[q0 + q]) : (float)sum[q0 + q];
                    z[q] = x * __shfl_sync(0xFFFFFFFFu, hs, q) * ws + bias;
                }
                // 16 stores in a row, where none is left out (each of those is a branch, and nothing overlaps: 2,048 rows x
                // 50,000 x 256 took 242 us with a store to a score, 137 so)
                const int64_t to = (int64_t)m * a.ostride + v;
                if (rows == 16) {
                    if (in) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) store_score<DT>(a.out, to + q * a.ostride, z[q]);
                    }
                } else if (in) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (q < rows) store_score<DT>(a.out, to + q * a.ostride, z[q]);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 3) tmem_free(tmem, 512);
}

// 8-bit [rows, cols] in boxes of 128 columns.
bool make_int8_map(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t stride, int box_rows) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {kI8K, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int DT>
int launch_scores(const Int8Args &args, cudaStream_t st) {
    using S = Int8Shape<N>;
    const void *fn = reinterpret_cast<const void *>(&int8_scores_kernel<N, DT>);
    CUtensorMap mw, mp, mh;
    const int64_t padded = int8_padded(args.H);
    if (!make_int8_map(&mw, args.weight, args.H, args.V, args.wstride, 128) ||
        !make_int8_map(&mp, args.weight, args.H, args.V, args.wstride, 32) ||
        !make_map_blocks(&mh, args.half, padded, args.M, padded, N, 2) || prepare_kernel(fn, S::SMEM, 1) != 0)
        return -1;
    const int64_t sms = sm_count(), blocks = (args.M + N - 1) / N, all = blocks * ((args.V + 127) / 128);
    const int64_t each = ((args.V + sms - 1) / sms + 31) / 32 * 32;
    Int8Args a = args;
    int32_t row_blocks = (int32_t)blocks, tiles = (int32_t)all, run = blocks == 1 ? (int32_t)each : 0;
    const int64_t grid = run > 0 ? (args.V + run - 1) / run : all < sms ? all : sms;
    void *params[] = {&mw, &mp, &mh, &a, &row_blocks, &tiles, &run};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, params) == cudaSuccess ? 0 : -1;
}
template <int DT>
int launch_rows(const Int8Args &a, cudaStream_t st) {
    return a.M <= 16   ? launch_scores<16, DT>(a, st)
           : a.M <= 32 ? launch_scores<32, DT>(a, st)
           : a.M <= 64 ? launch_scores<64, DT>(a, st)
                       : launch_scores<128, DT>(a, st);
}

}  // namespace

unsigned int *int8_status_ptr() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_int8_status) != cudaSuccess) return nullptr;
    return reinterpret_cast<unsigned int *>(p);
}

int int8_launch(const Int8Args &args, cudaStream_t st) {
    Int8Args a = args;
    void *params[] = {&a};
    const int64_t threads = a.M * (int8_padded(a.H) / 16);
    if (cudaLaunchKernel(reinterpret_cast<const void *>(&int8_hidden_kernel), dim3((unsigned)((threads + 255) / 256)),
                         dim3(256), params, 0, st) != cudaSuccess)
        return -1;
    return a.dtype == 0 ? launch_rows<0>(a, st) : a.dtype == 1 ? launch_rows<1>(a, st) : launch_rows<2>(a, st);
}

}  // namespace tsa
