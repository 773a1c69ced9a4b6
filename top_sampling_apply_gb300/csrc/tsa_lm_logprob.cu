// The log-probability of one token a row straight from the hidden rows:
//     z = h W^T + b,  z <- cap tanh(z / cap),
//     out = z_i / T - ln sum_{j allowed} exp(z_j / T)
// without writing the scores.  A first kernel forms, for every part of the
// vocabulary and every row, the largest score m and Z = sum exp((z - m) / T),
// and stores the token's own score; a second one joins a row's parts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_tcgen05.cuh"

namespace tsa {

namespace {

__device__ __forceinline__ float row_temp(const LmLogprobArgs &a, int64_t row) {
    const float T = a.temperature ? __ldg(a.temperature + row) : a.temperature_s;
    return T > 0.f ? T : 1.f;
}
__device__ unsigned int g_lm_logprob_status;

// x = z if a == b: a selection that keeps an array's elements in registers
// (written as a loop of ifs it becomes an indexed array in local memory, which
// every pass would have to fill).
__device__ __forceinline__ void select_if(float &x, float z, int a, int b) {
    asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, %3;\n\tselp.f32 %0, %1, %0, p;\n\t}" : "+f"(x) : "f"(z), "r"(a), "r"(b));
}

// A bounded wait whose outcome the whole warp shares.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, &g_lm_logprob_status));
}

// ------------------------------------------------------------ the products
// One persistent CTA an SM.  Warp 0 fetches tiles of 64 columns of H by TMA
// into a ring of stages, warp 1 issues the products, and warps 2 to 5 reduce
// the finished scores from one half of tensor memory while the next tile's
// products fill the other half (warps 2 to 9 where the scores are many: four
// for each quarter of the lanes, a quarter of the columns each).
//
// ROWS = false (few rows): the 128 lanes of tensor memory are vocabulary
// entries and the N columns are the hidden rows, so the weight is all that
// moves and nothing of the products is padding but N's remainder.  The
// vocabulary is cut into one run of rows a CTA, a multiple of 32, so that every
// SM moves the same bytes (whole tiles of 128 would leave a fifth of them idle
// at V = 32,000); a tile's copies are 32 rows each, and a run's last tile takes
// only the ones it needs.  A thread keeps one (m, Z) a hidden row over all its
// CTA's tiles; one part a CTA.
// ROWS = true: the lanes are 128 hidden rows and the columns N vocabulary
// entries; a thread reduces N / 2 of its row's scores by itself.  Tiles go
// through the hidden rows first, so that a weight tile is fetched from HBM once
// and from L2 by the other row blocks.  One part for every N / 2 entries of the
// vocabulary.
// The tensor cores add to their accumulator with truncation: a score of 320
// steps (H = 5,120) came out 9e-6 of itself too small, and 2,048
// log-probabilities were off by 2.4e-6 of themselves.  So the products of 512
// columns (1,024 where the products bound the kernel) at a time go to tensor
// memory and from there, rounded to nearest, into sums in registers: now 4e-7,
// for 7 % of the time.  (256 vocabulary entries a tile are 128 sums a thread, and 48 bytes of it
// are spilled.)
template <bool ROWS>
constexpr int kTcChunk = (ROWS ? 1024 : 512) / kTcK;  // steps of kTcK a chunk
template <bool ROWS>
constexpr int kTcThreads = ROWS ? 320 : 192;  // eight or four warps take the scores

template <int N, bool ROWS, int STAGES>
struct TcShape {
    static constexpr int A_BYTES = 128 * kTcK * 2, B_BYTES = N * kTcK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int SMEM = STAGES * STAGE + 1024;
    static constexpr int COLS = 2 * N < 32 ? 32 : 2 * N;
    // instruction descriptor: fp32 sums of bf16 products, both operands K-major, M = 128
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N / 8) << 17) | (8u << 24);
};

template <int N, bool ROWS, int STAGES>
__global__ void __launch_bounds__(kTcThreads<ROWS>, 1) lm_logprob_kernel(const __grid_constant__ CUtensorMap map_a,
                                                                   const __grid_constant__ CUtensorMap map_b,
                                                                   LmLogprobArgs a, int64_t tiles, int row_blocks, int64_t run) {
    using S = TcShape<N, ROWS, STAGES>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[STAGES], empty[STAGES], done[2], drained[2], last;
    __shared__ uint32_t tmem_slot;
    __shared__ float2 s_part[4][ROWS ? 1 : N];
    constexpr int NC = N / 2;  // a thread's columns of many rows' scores
    __shared__ __align__(16) float s_bias[ROWS ? 8 : 1][ROWS ? NC : 4];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kblocks = (int)((a.H + kTcK - 1) / kTcK);
    // this CTA's vocabulary rows (few hidden rows), or tiles
    const int64_t v_first = ROWS ? 0 : (int64_t)blockIdx.x * run;
    const int64_t v_end = ROWS || v_first + run > a.V ? a.V : v_first + run;
    const int64_t t_first = ROWS ? blockIdx.x : 0, t_step = ROWS ? gridDim.x : 1;
    const int64_t t_end = ROWS ? tiles : (v_end - v_first + 127) / 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&drained[i], ROWS ? 256 : 128);
        }
        mbar_init(&last, 1);
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(&tmem_slot, S::COLS);
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    pdl_launch_dependents();  // the joining kernel waits for this one's end before it reads
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t t = t_first; ok && t < t_end; t += t_step) {
                const int32_t va = ROWS ? (int32_t)(t % row_blocks) * 128 : (int32_t)(v_first + t * 128);
                const int groups = ROWS || v_end - va >= 128 ? 4 : (int)((v_end - va + 31) / 32);
                const int32_t vb = ROWS ? (int32_t)(t / row_blocks) * N : 0;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    if (!mbar_wait_bounded(&empty[s], ((it / STAGES) & 1u) ^ 1u, &g_lm_logprob_status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = ring + (size_t)s * S::STAGE;
                    if (ROWS) {
                        mbar_arrive_expect_tx(&full[s], S::STAGE);
                        tma_tile(st, &map_a, kb * kTcK, va, &full[s]);
                    } else {
                        mbar_arrive_expect_tx(&full[s], (uint32_t)(groups * (S::A_BYTES / 4) + S::B_BYTES));
                        for (int i = 0; i < groups; ++i)
                            tma_tile(st + i * (S::A_BYTES / 4), &map_a, kb * kTcK, va + 32 * i, &full[s]);
                    }
                    tma_tile(st + S::A_BYTES, &map_b, kb * kTcK, vb, &full[s]);
                }
            }
            // No copy may land, and no commit arrive, after the CTA is gone:
            // wait for the last use of each stage (the copies alone if a wait
            // above gave up).
            const uint32_t n = it < STAGES ? it : STAGES;
            for (uint32_t i = it - n; i < it; ++i)
                mbar_wait_bounded(ok ? &empty[i % STAGES] : &full[i % STAGES], (i / STAGES) & 1u,
                                  &g_lm_logprob_status);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0, j = 0;
            bool ok = true;
            for (int64_t t = t_first; ok && t < t_end; t += t_step) {
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const uint32_t b = j & 1u;
                    if (kb % kTcChunk<ROWS> == 0) {
                        if (!mbar_wait_bounded(&drained[b], ((j >> 1) & 1u) ^ 1u, &g_lm_logprob_status)) {
                            ok = false;
                            break;
                        }
                        mma_fence_after();
                    }
                    const uint32_t s = it % STAGES;
                    if (!mbar_wait_bounded(&full[s], (it / STAGES) & 1u, &g_lm_logprob_status)) {
                        ok = false;
                        break;
                    }
                    mma_fence_after();
                    const uint8_t *st = ring + (size_t)s * S::STAGE;
                    const uint64_t da = smem_tile(st), db = smem_tile(st + S::A_BYTES);
#pragma unroll
                    for (int k = 0; k < kTcK / 16; ++k)
                        mma_bf16(tmem + b * N, da + 2 * k, db + 2 * k, S::IDESC, kb % kTcChunk<ROWS> > 0 || k > 0);
                    mma_commit(&empty[s]);
                    if (kb % kTcChunk<ROWS> == kTcChunk<ROWS> - 1 || kb == kblocks - 1) {
                        mma_commit(&done[b]);
                        ++j;
                    }
                }
            }
            // the products are finished before tensor memory is freed
            mma_commit(&last);
            mbar_wait_bounded(&last, 0, &g_lm_logprob_status);
        }
    } else {
        const int quarter = warp & 3;  // a warp reads the lanes of its number modulo 4
        const uint32_t lane_at = (uint32_t)quarter << 21;
        const Cap cap = make_cap(a.cap);
        const int chunks = (kblocks + kTcChunk<ROWS> - 1) / kTcChunk<ROWS>;
        uint32_t j = 0;
        if constexpr (ROWS) {
            const int half = (warp - 2) >> 2;
            float *bias = s_bias[warp - 2];
            bool ok = true;
            for (int64_t t = t_first; ok && t < t_end; t += t_step) {
                const int64_t row = (t % row_blocks) * 128 + quarter * 32 + lane;
                const int64_t v0 = (t / row_blocks) * N + half * NC;
                const bool in = row < a.M;
                const float c2 = in ? kLog2eH / row_temp(a, row) : 1.f;
                const int64_t want = in ? __ldg(a.tokens + row) - v0 : -1;
                const int32_t *mrow = a.mask && in ? a.mask + row * a.mstride : nullptr;
                if (a.bias) {
                    __syncwarp();  // the last tile's values have been read
#pragma unroll
                    for (int i = 0; i < NC; i += 32)
                        bias[i + lane] = v0 + i + lane < a.V ? __ldg(a.bias + v0 + i + lane) : 0.f;
                    __syncwarp();
                }
                float z[NC];
                for (int c = 0; c < chunks; ++c, ++j) {
                    const uint32_t b = j & 1u;
                    ok = ok && warp_wait(&done[b], (j >> 1) & 1u);
                    if (!ok) break;
                    mma_fence_after();
                    const uint32_t at = tmem + lane_at + b * N + half * NC;
#pragma unroll
                    for (int q = 0; q < NC; q += 16) {
                        uint32_t r[16];
                        __syncwarp();
                        TmemLoad<16>::ld(at + q, r);
                        tmem_wait_ld();
                        if (c == 0) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) z[q + i] = __uint_as_float(r[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                split_pair(add2(pair_of(z[q + i], z[q + i + 1]),
                                                pair_of(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))),
                                           z[q + i], z[q + i + 1]);
                        }
                    }
                    mma_fence_before();
                    mbar_arrive(&drained[b]);
                }
                float2 st = make_float2(-INFINITY, 0.f);
                // 32 scores of the row at a time
#pragma unroll
                for (int c = 0; c < NC; c += 32) {
                    const int64_t left = a.V - (v0 + c);
                    if (left <= 0 || !ok) break;
                    float *x = z + c;
                    uint32_t bits = left < 32 ? (1u << left) - 1u : 0xFFFFFFFFu;
                    if (mrow) bits &= (uint32_t)__ldg(mrow + ((v0 + c) >> 5));
                    if (a.bias) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(bias + c + q);
                            split_pair(add2(pair_of(x[q], x[q + 1]), pair_of(f.x, f.y)), x[q], x[q + 1]);
                            split_pair(add2(pair_of(x[q + 2], x[q + 3]), pair_of(f.z, f.w)), x[q + 2], x[q + 3]);
                        }
                    }
                    if (a.cap > 0.f) soft_cap<32>(x, cap);
                    if (bits != 0xFFFFFFFFu) {
#pragma unroll
                        for (int q = 0; q < 32; ++q) x[q] = (bits >> q) & 1u ? x[q] : -INFINITY;
                    }
                    float sum = x[0], top = x[0];  // a sum is NaN if a score is
#pragma unroll
                    for (int q = 1; q < 32; ++q) top = fmaxf(top, x[q]);
                    unsigned long long all = pair_of(x[0], x[1]);
#pragma unroll
                    for (int q = 2; q < 32; q += 2) all = add2(all, pair_of(x[q], x[q + 1]));
                    float s1;
                    split_pair(all, sum, s1);
                    sum += s1;
                    if (sum != sum) {  // a NaN (counts as -inf), or both infinities
#pragma unroll
                        for (int q = 0; q < 32; ++q) x[q] = fmaxf(x[q], -INFINITY);
                        top = x[0];
#pragma unroll
                        for (int q = 1; q < 32; ++q) top = fmaxf(top, x[q]);
                    }
                    const int64_t w = want - c;
                    if (w >= 0 && w < 32) {
                        float found = -INFINITY;
#pragma unroll
                        for (int q = 0; q < 32; ++q) select_if(found, x[q], (int)w, q);
                        a.tok[row] = found;
                    }
                    if (top > -INFINITY) {
                        if (top > st.x) st = lm_join(st, make_float2(top, 0.f), c2);
                        const unsigned long long neg = pair_of(-st.x, -st.x), cc = pair_of(c2, c2);
                        unsigned long long acc = pair_of(st.y, 0.f);
#pragma unroll
                        for (int q = 0; q < 32; q += 2) {
                            float e0, e1;
                            split_pair(mul2(add2(pair_of(x[q], x[q + 1]), neg), cc), e0, e1);
                            acc = add2(acc, pair_of(ex2_approx(e0), ex2_approx(e1)));
                        }
                        float s0;
                        split_pair(acc, s0, s1);
                        st.y = s0 + s1;
                    }
                }
                if (in && v0 < a.V) a.part[((t / row_blocks) * 2 + half) * a.M + row] = st;
            }
        } else {
            float2 st[N];
#pragma unroll
            for (int q = 0; q < N; ++q) st[q] = make_float2(-INFINITY, 0.f);
            bool ok = true;
            for (int64_t t = t_first; ok && t < t_end; t += t_step) {
                const int64_t w0 = v_first + t * 128 + quarter * 32, v = w0 + lane;
                const float bias = a.bias && v < v_end ? __ldg(a.bias + v) : 0.f;
                float z[N];
                for (int c = 0; c < chunks; ++c, ++j) {
                    const uint32_t b = j & 1u;
                    ok = warp_wait(&done[b], (j >> 1) & 1u);
                    if (!ok) break;
                    mma_fence_after();
                    uint32_t r[N];
                    __syncwarp();
                    TmemLoad<N>::ld(tmem + lane_at + b * N, r);
                    tmem_wait_ld();
                    mma_fence_before();
                    mbar_arrive(&drained[b]);
#pragma unroll
                    for (int q = 0; q < N; ++q)
                        z[q] = c == 0 ? __uint_as_float(r[q]) : z[q] + __uint_as_float(r[q]);
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < N; ++q) z[q] += bias;
                if (a.cap > 0.f) soft_cap<N>(z, cap);
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    if (q >= a.M) break;
                    float x = fmaxf(z[q], -INFINITY);
                    if (v >= v_end) x = -INFINITY;  // lanes past the run hold what was there before
                    if (a.mask && w0 < v_end &&
                        !(((uint32_t)__ldg(a.mask + q * a.mstride + (w0 >> 5)) >> lane) & 1u))
                        x = -INFINITY;
                    if (v < v_end && __ldg(a.tokens + q) == v) a.tok[q] = x;
                    if (x > -INFINITY) st[q] = lm_join(st[q], make_float2(x, 1.f), kLog2eH / row_temp(a, q));
                }
            }
            if (ok) {
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    if (q >= a.M) break;
                    const float c2 = kLog2eH / row_temp(a, q);
                    float2 x = st[q];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        float2 y;
                        y.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, o);
                        y.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, o);
                        x = lm_join(x, y, c2);
                    }
                    if (lane == 0) s_part[quarter][q] = x;
                }
            }
        }
    }
    __syncthreads();
    if constexpr (!ROWS) {
        if (threadIdx.x < N && (int64_t)threadIdx.x < a.M) {
            const float c2 = kLog2eH / row_temp(a, threadIdx.x);
            float2 x = s_part[0][threadIdx.x];
            for (int w = 1; w < 4; ++w) x = lm_join(x, s_part[w][threadIdx.x], c2);
            a.part[(int64_t)blockIdx.x * a.M + threadIdx.x] = x;
        }
    }
    if (warp == 1) tmem_free(tmem, S::COLS);
}

// A row's parts: 8 rows a CTA, 64 threads a row (a pass over 2,048 parts is 32
// loads a thread, four under way together), then a tree over them.
constexpr int kJoinX = 8, kJoinY = 64;
__global__ void __launch_bounds__(kJoinX *kJoinY) lm_logprob_join_kernel(LmLogprobArgs a, int64_t parts) {
    __shared__ float2 sh[kJoinY][kJoinX];
    pdl_wait_primary();
    const int64_t row = (int64_t)blockIdx.x * kJoinX + threadIdx.x;
    const float T = row < a.M ? row_temp(a, row) : 1.f, c2 = kLog2eH / T;
    float2 s = make_float2(-INFINITY, 0.f);
    if (row < a.M) {
        const float2 *part = a.part + row;
        int64_t p = threadIdx.y;
        for (; p + 3 * kJoinY < parts; p += 4 * kJoinY) {
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(p + i * kJoinY) * a.M];
            s = lm_join(s, lm_join(lm_join(v[0], v[1], c2), lm_join(v[2], v[3], c2), c2), c2);
        }
        for (; p < parts; p += kJoinY) s = lm_join(s, part[p * a.M], c2);
    }
    sh[threadIdx.y][threadIdx.x] = s;
#pragma unroll
    for (int o = kJoinY / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.y < o)
            sh[threadIdx.y][threadIdx.x] = lm_join(sh[threadIdx.y][threadIdx.x], sh[threadIdx.y + o][threadIdx.x], c2);
    }
    if (threadIdx.y != 0 || row >= a.M) return;
    s = sh[0][threadIdx.x];
    const int64_t i = a.tokens[row];
    float r = __int_as_float(0x7FC00000);
    if (i >= 0 && i < a.V && s.x > -INFINITY && s.x < INFINITY) {
        const float z = a.tok[row];
        r = z > -INFINITY ? (z - s.x) / T - logf(s.y) : -INFINITY;
    }
    a.out[row] = r;
}

}  // namespace

// The row-block form needs full blocks to be worth its padding; up to 32 rows
// are columns instead.
constexpr int64_t kLmFew = 32;
// One block of hidden rows: smaller tiles spread the vocabulary more evenly.  100
// rows x 128,256 x 4,096: 200 us, 79 % of the copy rate for the weight alone (one
// row 162 us).
constexpr int64_t kLmMid = 128;

namespace {

template <int N, bool ROWS, int STAGES>
int launch_products(const LmLogprobArgs &args, int64_t *parts, cudaStream_t st) {
    using S = TcShape<N, ROWS, STAGES>;
    const void *fn = reinterpret_cast<const void *>(&lm_logprob_kernel<N, ROWS, STAGES>);
    CUtensorMap ma, mb;
    if (!make_map(&ma, ROWS ? args.hidden : args.weight, args.H, ROWS ? args.M : args.V,
                  ROWS ? args.hstride : args.wstride, ROWS ? 128 : 32) ||
        !make_map(&mb, ROWS ? args.weight : args.hidden, args.H, ROWS ? args.V : args.M,
                  ROWS ? args.wstride : args.hstride, N))
        return -1;
    if (prepare_kernel(fn, S::SMEM, 1) != 0) return -1;
    int row_blocks = ROWS ? (int)((args.M + 127) / 128) : 1;
    int64_t tiles = ROWS ? row_blocks * ((args.V + N - 1) / N) : (args.V + 127) / 128;
    const int64_t sms = sm_count();
    int64_t run = ((args.V + sms - 1) / sms + 31) / 32 * 32;
    const int64_t grid = ROWS ? (tiles < sms ? tiles : sms) : (args.V + run - 1) / run;
    *parts = ROWS ? (args.V + N / 2 - 1) / (N / 2) : grid;
    LmLogprobArgs a = args;
    void *params[] = {&ma, &mb, &a, &tiles, &row_blocks, &run};
    return cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(kTcThreads<ROWS>), params, S::SMEM, st) == cudaSuccess ? 0 : -1;
}

}  // namespace

// The most parts a form writes: half a tile of the vocabulary, or a CTA an SM.
int64_t lm_logprob_parts(int64_t M, int64_t V) {
    if (M <= kLmFew) return 256;
    return M <= kLmMid ? (V + 63) / 64 : (V + 127) / 128;
}

int lm_logprob_launch(const LmLogprobArgs &args, cudaStream_t st) {
    int64_t parts = 0;
    int r;
    if (args.M <= 16)
        r = launch_products<16, false, 11>(args, &parts, st);
    else if (args.M <= kLmFew)
        r = launch_products<32, false, 10>(args, &parts, st);
    else if (args.M <= kLmMid)
        r = launch_products<128, true, 6>(args, &parts, st);
    else
        r = launch_products<256, true, 4>(args, &parts, st);
    if (r != 0) return -1;
    LmLogprobArgs a = args;
    void *params[] = {&a, &parts};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + kJoinX - 1) / kJoinX));
    cfg.blockDim = dim3(kJoinX, kJoinY);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&lm_logprob_join_kernel), params) == cudaSuccess
               ? 0
               : -1;
}

unsigned int *lm_logprob_status_ptr() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_lm_logprob_status) != cudaSuccess) return nullptr;
    return reinterpret_cast<unsigned int *>(p);
}

}  // namespace tsa
