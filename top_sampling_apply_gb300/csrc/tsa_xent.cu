// The cross entropy of the head's scores with its gradients, without the
// scores.  With z = h W^T + b, z <- cap tanh(z / cap), l = ln sum_j exp(z_j):
//     row = l - z_t + c l^2,   loss = sum over rows of w row,
//     g_j = w ((1 + 2 c l) exp(z_j - l) - [j = t]) (1 - (z_j / cap)^2),
//     dH = G W,  dW = G^T H,  db = sum over rows of G.
// The rows that count are brought together first, so that skipped ones cost
// nothing and whatever they hold stays out of the products.  A first pass over
// the scores gives their log-sum-exps; then the vocabulary goes by in pieces: a
// piece's scores again, turned into its part of G in bf16, and that part's
// products.  That is 8 M V H operations where 6 would do if the scores were kept.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <numeric>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_tcgen05.cuh"

namespace tsa {

namespace {

// The rows that count, one after another in their order, each filled up to whole
// tiles of columns with zeros; their targets and weights (without weights each
// has 1 / (number of them)); zeros up to a multiple of 128 rows (128 at least),
// and in the outputs of skipped rows.  A warp a row.  Every CTA counts for itself
// the rows before its own, and all: M / 256 loads a thread, against a launch
// of their own for a prefix sum.
constexpr int kXentPrep = 8;

__device__ __forceinline__ bool xent_live(const XentArgs &a, int64_t m, float &w) {
    const int64_t t = a.targets[m];
    w = a.row_weight ? a.row_weight[m] : 1.f;
    return t >= 0 && t < a.V && w != 0.f;
}

__global__ void __launch_bounds__(32 * kXentPrep) xent_prepare_kernel(const XentArgs a) {
    __shared__ int s_all[kXentPrep], s_before[kXentPrep];
    __shared__ uint32_t s_top[kXentPrep];
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t m0 = (int64_t)blockIdx.x * kXentPrep, m = m0 + warp;
    int all = 0, before = 0;
    uint32_t top = 0;
    for (int64_t i = threadIdx.x; i < a.M; i += 32 * kXentPrep) {
        float w;
        if (xent_live(a, i, w)) {
            ++all;
            before += i < m0;
            top = max(top, __float_as_uint(fabsf(w)));
        }
    }
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) s_all[warp] = all, s_before[warp] = before, s_top[warp] = top;
    __syncthreads();
    all = before = 0, top = 0;
#pragma unroll
    for (int i = 0; i < kXentPrep; ++i) all += s_all[i], before += s_before[i], top = max(top, s_top[i]);
    const int64_t n = all, end = n < 1 ? 128 : (n + 127) / 128 * 128;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.count[0] = (int32_t)n;
        a.scale[0] = n < 1 ? 1.f : a.row_weight ? __uint_as_float(top) : 1.f / (float)n;
    }
    const int64_t vecs = a.H / 8, wide = xent_width(a.H) / 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 *rows = reinterpret_cast<uint4 *>(a.hidden_c);
    if (m0 >= a.M) {  // the CTAs behind the last row
        const int64_t i = n + m - (a.M + kXentPrep - 1) / kXentPrep * kXentPrep;
        if (i >= end) return;
        for (int64_t v = lane; v < wide; v += 32) rows[i * wide + v] = zero;
        if (lane == 0) a.tokens[i] = -1;
        return;
    }
    float w = 0.f;
    const bool one = lane < kXentPrep && m0 + lane < a.M && xent_live(a, m0 + lane, w);
    const uint32_t vote = __ballot_sync(0xFFFFFFFFu, one);
    if (m >= a.M) return;
    if (m >= n && lane == 0) a.weight_c[m] = a.row_loss_c[m] = 0.f;  // as a place, it has no row
    if (vote >> warp & 1u) {
        const int64_t at = before + __popc(vote & ((1u << warp) - 1u));
        const uint4 *from = reinterpret_cast<const uint4 *>(a.hidden + m * a.hstride);
        for (int64_t v = lane; v < wide; v += 32) rows[at * wide + v] = v < vecs ? from[v] : zero;
        if (lane == warp) {
            a.rows[at] = (int32_t)m;
            a.tokens[at] = a.targets[m];
            a.weight_c[at] = a.row_weight ? w : 1.f / (float)n;
        }
        return;
    }
    if (a.dh)
        for (int64_t v = lane; v < vecs; v += 32) reinterpret_cast<uint4 *>(a.dh + m * a.dhstride)[v] = zero;
    if (lane == 0) a.row_loss[m] = a.lse[m] = 0.f;
}

// A first pass over the scores of some of the rows that count.
struct XentPass {
    int64_t first, M;  // M at most
};

// The losses of a pass's rows from their parts, and what their gradients need;
// places up to the next multiple of 128 have none.  8 rows a CTA, 64 threads a
// row, then a tree over them.
constexpr int kXentJoinX = 8, kXentJoinY = 64;
__global__ void __launch_bounds__(kXentJoinX *kXentJoinY) xent_loss_kernel(const XentArgs a, const XentPass s,
                                                                           int64_t parts) {
    __shared__ float2 sh[kXentJoinY][kXentJoinX];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t n = a.count[0], at = (int64_t)blockIdx.x * kXentJoinX + threadIdx.x, i = s.first + at;
    const int64_t M = n - s.first < s.M ? n - s.first : s.M;  // the pass's rows
    float2 x = make_float2(-INFINITY, 0.f);
    if (at < M) {
        const float2 *part = a.part + at;
        int64_t p = threadIdx.y;
        for (; p + 3 * kXentJoinY < parts; p += 4 * kXentJoinY) {
            float2 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = part[(p + q * kXentJoinY) * M];
            x = lm_join(x, lm_join(lm_join(v[0], v[1], kLog2eH), lm_join(v[2], v[3], kLog2eH), kLog2eH), kLog2eH);
        }
        for (; p < parts; p += kXentJoinY) x = lm_join(x, part[p * M], kLog2eH);
    }
    sh[threadIdx.y][threadIdx.x] = x;
#pragma unroll
    for (int o = kXentJoinY / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.y < o)
            sh[threadIdx.y][threadIdx.x] = lm_join(sh[threadIdx.y][threadIdx.x], sh[threadIdx.y + o][threadIdx.x], kLog2eH);
    }
    if (threadIdx.y != 0 || i >= (n < 1 ? 128 : (n + 127) / 128 * 128)) return;
    if (i >= n) {
        a.coef[i] = make_float4(0.f, 0.f, INFINITY, 0.f);
        return;
    }
    if (at >= M) return;  // the next pass's
    x = sh[0][threadIdx.x];
    const float ln = logf(x.y), l = x.x < INFINITY ? x.x + ln : x.x, c = a.z_loss;
    // the score less the sum's reference is exact where they are near
    float loss = x.x > -INFINITY && x.x < INFINITY ? ln - (a.tok[at] - x.x) : __int_as_float(0x7FC00000);
    if (c != 0.f) loss += c * l * l;
    a.row_loss_c[i] = loss;
    a.row_loss[a.rows[i]] = loss;
    a.lse[a.rows[i]] = l;
    const float w = a.row_weight ? a.weight_c[i] / a.scale[0] : 1.f;
    a.coef[i] = make_float4(c != 0.f ? w * fmaf(2.f * c, l, 1.f) : w, w, l, 1.f);
}

__device__ unsigned int g_xent_status;

__device__ __forceinline__ bool xent_wait(uint64_t *bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, &g_xent_status);
}
__device__ __forceinline__ bool xent_warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, xent_wait(bar, parity));
}

// The rows that the products go over: those that count, up to whole tiles.
__device__ __forceinline__ int32_t xent_end(const XentArgs &a) {
    const int32_t n = a.count[0];
    return n < 1 ? 128 : (n + 127) / 128 * 128;
}

// Both kernels are one persistent CTA an SM in the form of lm_head_logprob's
// products: warp 0 fetches tiles of 64 K columns by TMA into a ring of stages,
// warp 1 issues the products of 128 x N tiles, warps 2 to 9 take finished sums
// from one half of tensor memory while the next tile's products fill the other
// half: four warps for each quarter of the lanes, half of the columns each.
// Results leave through 4 KB of shared memory a warp and TMA, so that
// whole lines are written.  1,024 rows x 32,000 x 4,096: a pass over the scores
// 164 to 168 us, 1.6 PFLOP/s, both products 309 us, 1.7 PFLOP/s, the tensor
// pipe busy for 76 to 83 % of the time; in a long run the power limit binds.
constexpr int kXentThreads = 320;
constexpr int kXentSlab = 32 * 128;  // 32 rows of 64 bf16
constexpr uint32_t kAcrossA = 1u << 15, kAcrossB = 1u << 16;  // instruction descriptor: M or N contiguous instead of K

// P CTAs work on a tile together.  Two of a cluster take 256 rows, each its 128 and
// half of the columns' operand, which then passes through L2 and shared memory
// once for both: a third of the traffic less.  These kernels run at the GPU's power
// limit, where what is not moved is time.
template <int N, int P>
struct XentShape {
    static constexpr int A_BYTES = 128 * kTcK * 2, B_BYTES = N / P * kTcK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = 192 * 1024 / STAGE;
    static constexpr int SMEM = STAGES * STAGE + 8 * kXentSlab + 1024;
    static constexpr int NC = N / 2;  // a thread's columns
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N / 8) << 17) | ((8u * P) << 24);
};

// (`full`, `drained` and `last` of the pair's first CTA alone are used.)
template <int STAGES>
struct XentBars {
    uint64_t full[STAGES], empty[STAGES], done[2], drained[2], last;
    uint32_t tmem;
};
template <int P, int STAGES>
__device__ __forceinline__ void xent_setup(XentBars<STAGES> &s, uint32_t cols) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.done[i], 1);
            mbar_init(&s.drained[i], 8 * P);
        }
        mbar_init(&s.last, 1);
        mbar_init_fence();
    }
    __syncthreads();
    if constexpr (P > 1) cluster_sync();  // the barriers are there before the other CTA's arrivals
    if ((threadIdx.x >> 5) == 1) tmem_alloc_by<P>(&s.tmem, cols);
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
}
template <int P>
__device__ __forceinline__ void xent_close(uint32_t tmem, uint32_t cols) {
    __syncthreads();
    if constexpr (P > 1) cluster_sync();  // nothing of this CTA is read or arrived at any more
    if ((threadIdx.x >> 5) == 1) tmem_free_by<P>(tmem, cols);
}
// This warp has read its sums: to the CTA that issues.
template <int P>
__device__ __forceinline__ void xent_drained(uint64_t *bar, int lane) {
    mma_fence_before();
    __syncwarp();
    if (lane != 0) return;
    if constexpr (P == 1)
        mbar_arrive(bar);
    else
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(dsmem_addr(bar, 0)) : "memory");
}
// The issuing warp's wait for them.
template <int P>
__device__ __forceinline__ bool xent_wait_drained(uint64_t *bar, uint32_t parity) {
    const bool ok = xent_warp_wait(bar, parity);
    if constexpr (P > 1) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    mma_fence_after();
    return ok;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's way round the ring, together: a stage, its barriers, and their
// phase.  One lane issues, from operands that are the same in all of them
// (a copy or product costs a thread on its own twice as much).
template <int STAGES, int P>
struct XentRing {
    XentBars<STAGES> &bars;
    uint8_t *ring;
    uint32_t bytes, s, phase, turns;
    bool ok, ready;
    __device__ __forceinline__ XentRing(XentBars<STAGES> &b, uint8_t *r, uint32_t stage_bytes, bool fill)
        : bars(b), ring(r), bytes(stage_bytes), s(0), phase(fill ? 1 : 0), turns(0), ok(true), ready(false) {}
    __device__ __forceinline__ uint8_t *stage() const { return ring + s * bytes; }
    __device__ __forceinline__ uint64_t *full() const { return &bars.full[s]; }
    __device__ __forceinline__ uint64_t *empty() const { return &bars.empty[s]; }
    __device__ __forceinline__ bool wait_empty() { return ok = xent_warp_wait(empty(), phase); }
    // What arrives at the issuing CTA's barrier: the copies of both, which its own producer announces.
    __device__ __forceinline__ uint32_t filled() const { return P == 1 ? smem_u32(full()) : dsmem_addr(full(), 0); }
    __device__ __forceinline__ void expect(uint32_t rank) const {
        if (rank == 0) mbar_arrive_expect_tx(full(), P * bytes);
    }
    // With a look at the next stage, whose answer comes while this one's products are issued.
    __device__ __forceinline__ bool wait_full() {
        ok = ok && (ready || xent_warp_wait(full(), phase));
        mma_fence_after();
        const bool wraps = s + 1 == STAGES;
        seen = mbar_test_wait(&bars.full[wraps ? 0 : s + 1], wraps ? phase ^ 1u : phase);
        return ok;
    }
    __device__ __forceinline__ void next() {
        if (++s == STAGES) s = 0, phase ^= 1u, ++turns;
        ready = __all_sync(0xFFFFFFFFu, seen);
    }
    // No copy may land, and no commit arrive, after the CTA is gone: the last
    // use of every stage is waited for, its copies alone if a wait ran out (a pair's
    // second CTA does not see those: its waits run out long after they have landed).
    __device__ __forceinline__ void finish() {
        for (int i = 0; i < STAGES; ++i) {
            if (turns > 0 || i < (int)s) {
                const uint32_t use = i < (int)s ? turns : turns - 1;
                xent_warp_wait(ok ? &bars.empty[i] : &bars.full[i], use & 1u);
            }
        }
    }
    bool seen = false;
};

// A thread's 64 results in bf16 as its row of the warp's slab, with the
// 128-byte swizzle of the maps that they are stored through.
__device__ __forceinline__ void slab_row(uint8_t *slab, int lane, const float *x) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack_bf16(x[8 * q + 2 * i], x[8 * q + 2 * i + 1]);
        *reinterpret_cast<uint4 *>(slab + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}
__device__ __forceinline__ void slab_store(const CUtensorMap *map, uint8_t *slab, int lane, int32_t x, int32_t y) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store(map, slab, x, y);
}
__device__ __forceinline__ void slab_wait(int lane) {
    if (lane == 0) tma_store_read();
    __syncwarp();
}

// Sums over the warp's lanes of 32 values a lane: lane i gets the sum of the
// i-th (31 exchanges instead of 5 for each).
__device__ __forceinline__ float lane_sums(float (&x)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? x[j + o] : x[j], send = up ? x[j] : x[j + o];
            x[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    }
    return x[0];
}

// Scores of a tile, in chunks of 1,024 columns (the tensor cores cut what they
// add).  Lanes are rows; tiles go through the rows first.  SUMS: a pass's parts of
// the log-sum-exps, one a half tile of the vocabulary; else, from the same
// scores once more, a piece's part of G.
constexpr int kXentChunk = 1024 / kTcK;

template <int N, int P, bool SUMS>
__global__ void __launch_bounds__(kXentThreads, 1)
    xent_scores_kernel(const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_g, const XentArgs a, int64_t v0, int32_t width,
                       const XentPass pass) {
    using S = XentShape<N, P>;
    constexpr int STAGES = S::STAGES, NC = S::NC;
    extern __shared__ uint8_t raw[];
    __shared__ XentBars<STAGES> s;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int kblocks = (int)((a.H + kTcK - 1) / kTcK);
    const uint32_t rank = P == 1 ? 0 : cluster_ctarank();
    xent_setup<P>(s, 2 * N);
    pdl_launch_dependents();
    pdl_wait_primary();
    // the pass's rows, or all up to whole tiles
    const int32_t row0 = SUMS ? (int32_t)pass.first : 0;
    const int32_t rows = SUMS ? (int32_t)max((int64_t)0, min(a.count[0] - pass.first, pass.M)) : xent_end(a);
    const int32_t row_blocks = (rows + 128 * P - 1) / (128 * P), t_first = blockIdx.x / P, t_step = gridDim.x / P;
    const int32_t left = (int32_t)(a.V - v0 < width ? a.V - v0 : width);  // the piece's entries
    const int32_t tiles = row_blocks * ((left + N - 1) / N);  // (the products take whole tiles of G, and none behind them)
    const uint32_t tmem = s.tmem;

    if (warp == 0) {
        XentRing<STAGES, P> r(s, ring, S::STAGE, true);
        for (int32_t t = t_first; r.ok && t < tiles; t += t_step) {
            const int32_t ya = row0 + (t % row_blocks * P + rank) * 128, yb = t / row_blocks * N + rank * (N / P);
            for (int kb = 0; kb < kblocks; ++kb, r.next()) {
                if (!r.wait_empty()) break;
                if (elect_one()) {
                    r.expect(rank);
                    tma_tile_by<P>(r.stage(), &map_h, kb * kTcK, ya, r.filled());
                    tma_tile_by<P>(r.stage() + S::A_BYTES, &map_w, kb * kTcK, yb, r.filled());
                }
                __syncwarp();
            }
        }
        r.finish();
    } else if (warp == 1 && rank == 0) {  // (a pair's first CTA issues for both)
        XentRing<STAGES, P> r(s, ring, S::STAGE, false);
        uint32_t j = 0;
        for (int32_t t = t_first; r.ok && t < tiles; t += t_step) {
            for (int kb = 0; kb < kblocks; ++kb) {
                const uint32_t b = j & 1u;
                if (kb % kXentChunk == 0) r.ok = xent_wait_drained<P>(&s.drained[b], ((j >> 1) & 1u) ^ 1u);
                if (!r.wait_full()) break;
                const bool end = kb % kXentChunk == kXentChunk - 1 || kb == kblocks - 1;
                const uint64_t da = smem_tile(r.stage()), db = smem_tile(r.stage() + S::A_BYTES);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTcK / 16; ++k)
                        mma_bf16_by<P>(tmem + b * N, da + 2 * k, db + 2 * k, S::IDESC, kb % kXentChunk > 0 || k > 0);
                    mma_commit_by<P>(r.empty());
                    if (end) mma_commit_by<P>(&s.done[b]);
                }
                if (end) ++j;
                r.next();
            }
        }
        if (elect_one()) mma_commit_own<P>(&s.last);  // the products are finished before tensor memory is freed
        xent_warp_wait(&s.last, 0);
    } else if (warp > 1) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t at = tmem + ((uint32_t)quarter << 21) + half * NC;
        const Cap cap = make_cap(a.cap);
        const int chunks = (kblocks + kXentChunk - 1) / kXentChunk;
        uint8_t *slab = ring + (size_t)STAGES * S::STAGE + (warp - 2) * kXentSlab;
        uint32_t j = 0;
        bool ok = true;
        for (int32_t t = t_first; ok && t < tiles; t += t_step) {
            const int32_t first = (t % row_blocks * P + rank) * 128 + quarter * 32;  // the warp's rows
            const int32_t c0 = t / row_blocks * N + half * NC;                      // and columns in the piece
            // (a pair's second 128 rows may be beyond the last)
            const bool in_row = SUMS ? first + lane < rows : first < rows;
            const float4 k = !SUMS && in_row ? a.coef[first + lane] : make_float4(0.f, 0.f, INFINITY, 0.f);
            const int64_t want = in_row ? a.tokens[row0 + first + lane] - v0 - c0 : -1;
            float z[NC];
            for (int c = 0; c < chunks; ++c, ++j) {
                const uint32_t b = j & 1u;
                ok = ok && xent_warp_wait(&s.done[b], (j >> 1) & 1u);
                if (!ok) break;
                mma_fence_after();
#pragma unroll
                for (int q = 0; q < NC; q += 16) {
                    uint32_t r[16];
                    __syncwarp();
                    TmemLoad<16>::ld(at + b * N + q, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        if (c == 0) {
                            z[q + i] = __uint_as_float(r[i]);
                            z[q + i + 1] = __uint_as_float(r[i + 1]);
                        } else {
                            split_pair(add2(pair_of(z[q + i], z[q + i + 1]),
                                            pair_of(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))),
                                       z[q + i], z[q + i + 1]);
                        }
                    }
                }
                xent_drained<P>(&s.drained[b], lane);
            }
            if (!ok) break;
            if (!SUMS && !in_row) continue;
            if (a.bias) {  // the warp's entries, by way of its slab
                slab_wait(lane);
                float *bias = reinterpret_cast<float *>(slab);
#pragma unroll
                for (int i = 0; i < NC; i += 32)
                    bias[i + lane] = c0 + i + lane < left ? __ldg(a.bias + v0 + c0 + i + lane) : 0.f;
                __syncwarp();
#pragma unroll
                for (int q = 0; q < NC; q += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(bias + q);
                    split_pair(add2(pair_of(z[q], z[q + 1]), pair_of(f.x, f.y)), z[q], z[q + 1]);
                    split_pair(add2(pair_of(z[q + 2], z[q + 3]), pair_of(f.z, f.w)), z[q + 2], z[q + 3]);
                }
                __syncwarp();
            }
            if constexpr (SUMS) {
                float2 st = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int c = 0; c < NC; c += 32) {
                    const int32_t in = left - (c0 + c);
                    if (in <= 0) break;
                    float *x = z + c;
                    if (a.cap > 0.f) soft_cap<32>(x, cap);
                    float top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        x[q] = q < in ? fmaxf(x[q], -INFINITY) : -INFINITY;  // NaN counts as -inf
                        top = fmaxf(top, x[q]);
                    }
                    const int64_t w = want - c;
                    if (w >= 0 && w < 32) {
                        float found = -INFINITY;
#pragma unroll
                        for (int q = 0; q < 32; ++q) found = w == q ? x[q] : found;
                        a.tok[first + lane] = found;
                    }
                    if (top > -INFINITY) {
                        if (top > st.x) st = lm_join(st, make_float2(top, 0.f), kLog2eH);
                        const unsigned long long neg = pair_of(-st.x, -st.x), cc = pair_of(kLog2eH, kLog2eH);
                        unsigned long long acc = pair_of(st.y, 0.f);
#pragma unroll
                        for (int q = 0; q < 32; q += 2) {
                            float e0, e1;
                            split_pair(mul2(add2(pair_of(x[q], x[q + 1]), neg), cc), e0, e1);
                            acc = add2(acc, pair_of(ex2_approx(e0), ex2_approx(e1)));
                        }
                        float s0, s1;
                        split_pair(acc, s0, s1);
                        st.y = s0 + s1;
                    }
                }
                if (in_row && c0 < left) a.part[(int64_t)(t / row_blocks * 2 + half) * rows + first + lane] = st;
                continue;
            }
            const float neg = -k.z * kLog2eH;
            // A place's entries in the piece: none behind the last row, where the products are 0 but a bias of +inf would
            // make NaN of them.
            const int32_t here = k.w > 0.f ? left - c0 : 0;
            // A score of NaN has no slope, and no part in a row's gradient, but where the row has no finite score at all.
            const float flat = neg < INFINITY ? 0.f : __int_as_float(0x7FC00000);
#pragma unroll
            for (int g0 = 0; g0 < NC; g0 += 64) {
#pragma unroll
                for (int h0 = 0; h0 < 64; h0 += 32) {
                    float *x = z + g0 + h0;
                    if (a.cap > 0.f) soft_cap<32>(x, cap);
                    const int32_t in = here - (g0 + h0);
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const float y = fmaxf(x[q], -INFINITY);  // NaN counts as -inf
                        float p = k.x * ex2_approx(fmaf(y, kLog2eH, neg));
                        if (want - (g0 + h0) == q) p -= k.y;
                        if (a.cap > 0.f) {
                            const float share = y * cap.inv;
                            p = y > -INFINITY ? p * fmaf(-share, share, 1.f) : flat;
                        }
                        x[q] = q < in ? p : 0.f;
                    }
                    if (a.db) {
                        float col[32];
#pragma unroll
                        for (int q = 0; q < 32; ++q) col[q] = x[q];
                        const float sum = lane_sums(col, lane);
                        a.db_part[(int64_t)(first / 32) * width + c0 + g0 + h0 + lane] = sum;
                    }
                }
                slab_wait(lane);
                slab_row(slab, lane, z + g0);
                slab_store(&map_g, slab, lane, c0 + g0, first);
            }
        }
        if (lane == 0) tma_store_done();
    }
    xent_close<P>(tmem, 2 * N);
}

// db of a piece: 32 columns a CTA, the rows' parts over 32 rows of threads.
__global__ void __launch_bounds__(1024) xent_bias_kernel(const XentArgs a, int64_t v0, int32_t width) {
    __shared__ float sh[32][33];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int32_t c = blockIdx.x * 32 + threadIdx.x, parts = xent_end(a) / 32;
    float s = 0.f;
    if (c < width && v0 + c < a.V)
        for (int32_t p = threadIdx.y; p < parts; p += 32) s += a.db_part[(int64_t)p * width + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = warp_sum_f32(sh[threadIdx.x][threadIdx.y]);  // column threadIdx.y
    const int64_t v = v0 + blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && v < a.V && v < v0 + width) a.db[v] = s * a.scale[0];
}

// The two products of a piece of G, as units of 128 x 256 results:
//     dW[v, h] = sum_m G[m, v] H[m, h],  dH[m, h] (+)= sum_v G[m, v] W[v, h],
// G without the largest row weight, which the results are multiplied by: rounded
// to bf16 with it, weights that are all the same (a mean's 1 / n) would shift
// every gradient by one and the same share, of up to 2^-9.
// G, H and W are taken as they lie: the operands of dW, and W, have K across
// their rows, which the tensor cores read just as well.  A CTA first takes its
// share of the dH units (long K: a piece of the vocabulary, or a part of it),
// then a run of the dW units whose length evens out what the first left uneven.
// dH is added up over the pieces in fp32, each unit by the one CTA that holds it.
struct XentUnits {
    int32_t rb, hb, dh, dw, all, kh, kw;  // row and column blocks; dH and dW units; K steps of a piece and of a unit each
    int32_t w0, w1;                       // this CTA's dW units
    int32_t group, groups, tall;          // this CTA's pair, pairs, and their rows
    __device__ __forceinline__ void plan(const XentArgs &a, int32_t left, int32_t end, int32_t P) {
        group = blockIdx.x / P, groups = gridDim.x / P, tall = 128 * P;
        rb = (end + tall - 1) / tall;
        hb = (int32_t)((a.H + 255) / 256);
        dh = a.dh ? rb * hb * a.splits : 0;
        dw = a.dw ? (left + tall - 1) / tall * hb : 0;
        all = (left + kTcK - 1) / kTcK;
        kh = (all + a.splits - 1) / a.splits;
        kw = end / kTcK;
        // the first `more` CTAs have a dH unit more, and `fewer` dW units each
        const int64_t ctas = groups, b = group, cost = kw + 4;  // a unit's results take about four steps
        const int64_t more = dh % ctas;
        int64_t fewer = 0;
        if (more > 0) {
            fewer = (((int64_t)dh * kh + (int64_t)dw * cost) / ctas - (dh / ctas + 1) * kh) / cost;
            if (fewer < 0) fewer = 0;
            if (fewer > dw / ctas) fewer = dw / ctas;
        }
        const int64_t rest = dw - more * fewer;
        if (b < more) {
            w0 = (int32_t)(b * fewer);
            w1 = (int32_t)(w0 + fewer);
        } else {
            w0 = (int32_t)(more * fewer + (b - more) * rest / (ctas - more));
            w1 = (int32_t)(more * fewer + (b - more + 1) * rest / (ctas - more));
        }
    }
    // This CTA's i-th unit, if it has one: its kind, its first row (of dH or dW)
    // and column, its first K step and their number.  dH units go through the
    // row blocks first, so that the CTAs share columns of W.
    struct Unit {
        bool is_dh;
        int32_t y, x, split, k0, ks;
    };
    __device__ __forceinline__ bool get(int32_t i, Unit &u) const {
        const int32_t b = group, ctas = groups;
        const int32_t own = b < dh % ctas ? dh / ctas + 1 : dh / ctas;
        u.is_dh = i < own;
        if (u.is_dh) {
            const int32_t t = b + i * ctas, tile = t % (rb * hb);
            u.split = t / (rb * hb);
            u.y = tile % rb * tall;
            u.x = tile / rb * 256;
            u.k0 = u.split * kh;
            u.ks = max(0, min(kh, all - u.k0));
            return true;
        }
        const int32_t t = w0 + i - own;
        u.y = t / hb * tall;
        u.x = t % hb * 256;
        u.split = u.k0 = 0;
        u.ks = kw;
        return t < w1;
    }
};

// Eight results of dH: on top of those of earlier pieces, into the fp32 sums or
// rounded to the gradient.
__device__ __forceinline__ void dh_results(const float *z, float *acc, bool add, uint16_t *to) {
    float4 p = make_float4(z[0], z[1], z[2], z[3]), r = make_float4(z[4], z[5], z[6], z[7]);
    if (add) {
        const float4 s = reinterpret_cast<const float4 *>(acc)[0], t = reinterpret_cast<const float4 *>(acc)[1];
        p.x += s.x, p.y += s.y, p.z += s.z, p.w += s.w;
        r.x += t.x, r.y += t.y, r.z += t.z, r.w += t.w;
    }
    if (!to) {
        reinterpret_cast<float4 *>(acc)[0] = p;
        reinterpret_cast<float4 *>(acc)[1] = r;
        return;
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(p.x, p.y), pack_bf16(p.z, p.w), pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
}

// The tensor cores cut what they add, a step of 16 by 2^-23 of the sum so far on average, always towards zero.  Sums
// over rows turn from one sign to the other (p h of all rows, -h of the entry's own), and what was cut on the way up stays:
// so a sum in tensor memory ends after 8,192 of K, 512 steps, and those are added in fp32.  What is lost is then 2^-15 of
// a part's largest sum, whatever K is.  65,536 rows x 256 x 128 in the order of their targets, hidden rows of mean 1: dW was
// off by 0.55 % of itself with one sum for all rows where exact sums of the same G give 0.39 %, and 1.0e-4 of the sum
// of absolute terms too small in the mean; by 0.42 % against 0.40 and 2.6e-5 so.  Up to 8,192 rows nothing is to be seen.
//
// LONG: units of more than 8,192 of K, whose sums are in registers until they leave; those of shorter units go
// from tensor memory to where they are stored 64 at a time (16 x 8,192 x 1,024 43 us, 45 by way of registers; 343 x
// 32,000 x 2,048 203 and 206).
constexpr int kXentSums = 8192 / kTcK;

template <int P, bool LONG>
__global__ void __launch_bounds__(kXentThreads, 1)
    xent_products_kernel(const __grid_constant__ CUtensorMap map_gk, const __grid_constant__ CUtensorMap map_gm,
                         const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h,
                         const __grid_constant__ CUtensorMap map_dw, const XentArgs a, int64_t v0, int32_t width,
                         int w_blocks) {
    using S = XentShape<256, P>;
    constexpr int STAGES = S::STAGES, NC = S::NC, BOX = 64 * 128;
    extern __shared__ uint8_t raw[];
    __shared__ XentBars<STAGES> s;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = P == 1 ? 0 : cluster_ctarank();
    xent_setup<P>(s, 512);
    pdl_launch_dependents();
    pdl_wait_primary();
    const int32_t n = a.count[0], end = xent_end(a);
    const float scale = a.scale[0];
    const int32_t left = (int32_t)(a.V - v0 < width ? a.V - v0 : width);
    XentUnits units;
    units.plan(a, left, end, P);
    const uint32_t tmem = s.tmem;
    XentUnits::Unit u;

    if (warp == 0) {
        XentRing<STAGES, P> r(s, ring, S::STAGE, true);
        for (int32_t x = 0; r.ok && units.get(x, u); ++x) {
            for (int kb = u.k0; kb < u.k0 + u.ks; ++kb, r.next()) {
                if (!r.wait_empty()) break;
                if (elect_one()) {
                    uint8_t *st = r.stage(), *sb = st + S::A_BYTES;
                    const int32_t ya = u.y + rank * 128, xb = u.x + rank * (256 / P);
                    r.expect(rank);
                    if (!u.is_dh) {
                        tma_blocks_by<P>(st, &map_gm, kb * kTcK, ya / kTcK, r.filled());
                        tma_blocks_by<P>(sb, &map_h, kb * kTcK, xb / kTcK, r.filled());
                    } else {
                        tma_tile_by<P>(st, &map_gk, kb * kTcK, ya, r.filled());
                        if (w_blocks) {
                            tma_blocks_by<P>(sb, &map_w, kb * kTcK, xb / kTcK, r.filled());
                        } else {
#pragma unroll
                            for (int q = 0; q < 4 / P; ++q)
                                tma_tile_by<P>(sb + q * BOX, &map_w, xb + 64 * q, kb * kTcK, r.filled());
                        }
                    }
                }
                __syncwarp();
            }
        }
        r.finish();
    } else if (warp == 1 && rank == 0) {  // (a pair's first CTA issues for both)
        XentRing<STAGES, P> r(s, ring, S::STAGE, false);
        uint32_t j = 0;
        for (int32_t x = 0; r.ok && units.get(x, u); ++x) {
            const uint32_t idesc = S::IDESC | kAcrossB | (u.is_dh ? 0u : kAcrossA), step = u.is_dh ? 2 : 128;
            for (int kb = 0; kb < u.ks; ++kb, r.next()) {
                const uint32_t b = j & 1u;
                if (kb % kXentSums == 0) r.ok = xent_wait_drained<P>(&s.drained[b], ((j >> 1) & 1u) ^ 1u);
                if (!r.wait_full()) break;
                const bool end = kb % kXentSums == kXentSums - 1 || kb == u.ks - 1;
                const uint64_t da = u.is_dh ? smem_tile(r.stage()) : smem_tile_across(r.stage(), BOX);
                const uint64_t db = smem_tile_across(r.stage() + S::A_BYTES, BOX);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTcK / 16; ++k)
                        mma_bf16_by<P>(tmem + b * 256, da + step * k, db + 128 * k, idesc, kb % kXentSums > 0 || k > 0);
                    mma_commit_by<P>(r.empty());
                    if (end) mma_commit_by<P>(&s.done[b]);
                }
                if (end) ++j;
            }
        }
        if (elect_one()) mma_commit_own<P>(&s.last);
        xent_warp_wait(&s.last, 0);
    } else if (warp > 1) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t at = tmem + ((uint32_t)quarter << 21) + half * NC;
        uint8_t *slab = ring + (size_t)STAGES * S::STAGE + (warp - 2) * kXentSlab;
        uint32_t j = 0;
        bool ok = true;
        for (int32_t i = 0; ok && units.get(i, u); ++i) {
            const int32_t y0 = u.y + rank * 128 + quarter * 32, h0 = u.x + half * NC;
            const bool used = u.is_dh || y0 < left;
            const uint32_t b = j & 1u;  // (of a single sum)
            float z[LONG ? NC : 64];
            if constexpr (LONG) {
#pragma unroll
                for (int q = 0; q < NC; ++q) z[q] = 0.f;
                for (int k0 = 0; k0 < u.ks; k0 += kXentSums, ++j) {
                    ok = xent_warp_wait(&s.done[j & 1u], (j >> 1) & 1u);
                    if (!ok) break;
                    mma_fence_after();
#pragma unroll
                    for (int q = 0; q < NC; q += 16) {
                        if (!used || h0 + q >= a.H) break;
                        uint32_t r[16];
                        __syncwarp();
                        TmemLoad<16>::ld(at + (j & 1u) * 256 + q, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            split_pair(add2(pair_of(z[q + i], z[q + i + 1]),
                                            pair_of(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))),
                                       z[q + i], z[q + i + 1]);
                    }
                    xent_drained<P>(&s.drained[j & 1u], lane);
                }
            } else if (u.ks > 0) {  // (a part of a short last piece may be empty)
                ok = xent_warp_wait(&s.done[b], (j >> 1) & 1u);
                mma_fence_after();
                ++j;
            }
            if (!ok) break;
            const int32_t m = y0 + lane;
            const bool mine = u.is_dh && m < n, last = a.splits == 1 && v0 + left >= a.V;
            float *acc = mine ? a.acc + ((int64_t)u.split * a.padded + m) * a.H + h0 : nullptr;
            uint16_t *to = mine && last ? a.dh + (int64_t)a.rows[m] * a.dhstride + h0 : nullptr;
#pragma unroll
            for (int g = 0; g < NC; g += 64) {
                if (!used || h0 + g >= a.H) break;
                float *x = z + (LONG ? g : 0);
                if constexpr (!LONG) {
#pragma unroll
                    for (int q = 0; q < 64; q += 16) {
                        uint32_t r[16];
                        __syncwarp();
                        TmemLoad<16>::ld(at + b * 256 + g + q, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[q + i] = u.ks > 0 ? __uint_as_float(r[i]) * scale : 0.f;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 64; ++q) x[q] *= scale;
                }
                if (!u.is_dh) {
                    slab_wait(lane);
                    slab_row(slab, lane, x);
                    slab_store(&map_dw, slab, lane, h0 + g, y0);
                } else if (mine) {
#pragma unroll
                    for (int q = 0; q < 64; q += 8) {
                        if (h0 + g + q < a.H) dh_results(x + q, acc + g + q, v0 > 0, last ? to + g + q : nullptr);
                    }
                }
            }
            if (!LONG && u.ks > 0) xent_drained<P>(&s.drained[b], lane);
        }
        if (lane == 0) tma_store_done();
    }
    xent_close<P>(tmem, 512);
}

// dH from the parts of a split K.
__global__ void __launch_bounds__(128) xent_join_kernel(const XentArgs a) {
    const int32_t m = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait_primary();
    if (m >= a.count[0]) return;
    const float *acc = a.acc + (int64_t)m * a.H;
    uint16_t *to = a.dh + (int64_t)a.rows[m] * a.dhstride;
    for (int64_t h = threadIdx.x * 4; h < a.H; h += 512) {
        float4 s = *reinterpret_cast<const float4 *>(acc + h);
        for (int i = 1; i < a.splits; ++i) {
            const float4 p = *reinterpret_cast<const float4 *>(acc + (int64_t)i * a.padded * a.H + h);
            s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
        }
        *reinterpret_cast<uint2 *>(to + h) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

}  // namespace

// Parts of the K of dH's units (a piece of the vocabulary): as many as keep a
// unit under half of what an SM has to do, down to 16 steps.
int xent_splits(int64_t M, int64_t H, int64_t V) {
    const int64_t pad = xent_padded(M), piece = xent_piece(M, V), hb = (H + 255) / 256;
    const int64_t left = piece < V ? piece : V, k = (left + kTcK - 1) / kTcK;
    const int64_t steps = pad / 128 * hb * k + (left + 127) / 128 * hb * (pad / kTcK + 4);
    const int64_t half = steps / 304 < 16 ? 16 : steps / 304;
    const int64_t n = (k + half - 1) / half;
    return (int)(n < 64 ? n : 64);
}

// The width of a piece of the vocabulary.  Its part of G takes up to 64 MB, half
// of L2, so that the products find much of it there, but it has 4,096 entries at
// least (of more than 8,192 rows), as dH's fp32 sums are read and written once a
// piece; and where that leaves a choice, its tiles are a multiple of the SMs (16
// blocks of rows: 57 tiles of 256 entries are six turns of 152 SMs, 63 would be 6.6).
int64_t xent_piece(int64_t M, int64_t V) {
    const int64_t blocks = xent_padded(M) / 128, all = (V + 255) / 256;
    int64_t fit = ((int64_t)64 << 20) / (2 * 128 * 256) / blocks;
    fit = fit < 16 ? 16 : fit > kXentMaxPiece / 256 ? kXentMaxPiece / 256 : fit;
    if (fit >= all) return all * 256;
    const int64_t turn = 152 / std::gcd((int64_t)152, blocks);
    return (fit < turn ? fit : fit / turn * turn) * 256;
}

unsigned int *xent_status_ptr() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_xent_status) != cudaSuccess) return nullptr;
    return reinterpret_cast<unsigned int *>(p);
}

namespace {

// A launch that may begin while the kernel before it drains; it waits for that
// one's end before it reads memory.  Clusters of P CTAs.
int launch(const void *fn, dim3 grid, dim3 block, size_t smem, void **params, cudaStream_t st, int P = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)P;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, params) == cudaSuccess ? 0 : -1;
}

// CTAs of a persistent launch: as many as there are SMs, whole pairs.
unsigned persistent(int64_t tiles, int P) {
    const int64_t groups = sm_count() / P;
    return (unsigned)((tiles < groups ? tiles : groups) * P);
}

template <int N, int P, bool SUMS>
int launch_scores(const XentArgs &args, int64_t v0, int64_t piece, XentPass pass, cudaStream_t st) {
    using S = XentShape<N, P>;
    const void *fn = reinterpret_cast<const void *>(&xent_scores_kernel<N, P, SUMS>);
    const int64_t pad = xent_padded(args.M), left = args.V - v0 < piece ? args.V - v0 : piece;
    CUtensorMap mh, mw, mg;
    if (!make_map(&mh, args.hidden_c, args.H, pad, xent_width(args.H), 128) ||
        !make_map(&mw, args.weight + v0 * args.wstride, args.H, left, args.wstride, N / P) ||
        !make_map(&mg, SUMS ? args.hidden_c : args.grad, SUMS ? args.H : piece, pad, SUMS ? xent_width(args.H) : piece, 32) ||
        prepare_kernel(fn, S::SMEM, 1) != 0)
        return -1;
    XentArgs a = args;
    int32_t width = (int32_t)piece;
    const int64_t rows = SUMS ? pass.M : pad;
    const unsigned grid = persistent((rows + 128 * P - 1) / (128 * P) * ((left + N - 1) / N), P);
    void *params[] = {&mh, &mw, &mg, &a, &v0, &width, &pass};
    return launch(fn, dim3(grid), dim3(kXentThreads), S::SMEM, params, st, P);
}

template <int P, bool LONG>
int launch_products(const XentArgs &args, int64_t v0, int64_t piece, cudaStream_t st) {
    using S = XentShape<256, P>;
    const void *fn = reinterpret_cast<const void *>(&xent_products_kernel<P, LONG>);
    const int64_t pad = xent_padded(args.M), left = args.V - v0 < piece ? args.V - v0 : piece;
    const int64_t wide = xent_width(args.H);
    const uint16_t *weight = args.weight + v0 * args.wstride;
    int w_blocks = args.H % kTcK == 0;  // else the last block would reach beyond the last row
    CUtensorMap gk, gm, mw, mh, dw;
    if (!make_map(&gk, args.grad, piece, pad, piece, 128) || !make_map_blocks(&gm, args.grad, piece, pad, piece, 64, 2) ||
        !(w_blocks ? make_map_blocks(&mw, weight, args.H, left, args.wstride, 64, 4 / P)
                   : make_map(&mw, weight, args.H, left, args.wstride, 64)) ||
        !make_map_blocks(&mh, args.hidden_c, wide, pad, wide, 64, 4 / P) ||
        !make_map(&dw, args.dw ? args.dw + v0 * args.dwstride : args.hidden_c, args.H, args.dw ? left : pad,
                  args.dw ? args.dwstride : wide, 32) ||
        prepare_kernel(fn, S::SMEM, 1) != 0)
        return -1;
    XentArgs a = args;
    int32_t width = (int32_t)piece;
    void *params[] = {&gk, &gm, &mw, &mh, &dw, &a, &v0, &width, &w_blocks};
    return launch(fn, dim3(persistent(sm_count(), P)), dim3(kXentThreads), S::SMEM, params, st, P);
}

// Whether pairs of CTAs take the rows, 256 at a time; an odd block of 128 (and how
// many blocks count is known on the GPU alone: skipped rows are left out) then
// costs two.  In a long run, single CTAs and pairs: 256 rows x 32,000 x 2,048 178
// and 182 us, 343 rows 211 and 230, 512 rows 249 and 238, 640 x 64,000 x 2,048 562
// and 562, 1,100 x 32,000 x 4,096 1,067 and 975, 2,048 x 128,256 x 5,120 7,190 and 6,640.
bool xent_pairs(int64_t M) { return xent_padded(M) / 128 >= 8; }

}  // namespace

int xent_launch(const XentArgs &args, cudaStream_t st) {
    XentArgs a = args;
    void *one[] = {&a};
    const int64_t pad = xent_padded(a.M), piece = xent_piece(a.M, a.V);
    const bool pairs = xent_pairs(a.M);
    // K steps of the longest unit: all rows for dW, a part of a piece for dH
    const int64_t steps = ((a.V < piece ? a.V : piece) + kTcK - 1) / kTcK, part = (steps + a.splits - 1) / a.splits;
    const bool sums = (a.dw && pad / kTcK > kXentSums) || (a.dh && part > kXentSums);
    if (cudaLaunchKernel(reinterpret_cast<const void *>(&xent_prepare_kernel),
                         dim3((unsigned)((a.M + kXentPrep - 1) / kXentPrep + 128 / kXentPrep)), dim3(32 * kXentPrep), one, 0,
                         st) != cudaSuccess)
        return -1;
    for (int64_t m = 0; m < a.M; m += kXentPass) {
        const bool more = a.M - m > kXentPass;
        XentPass pass = {m, more ? kXentPass : a.M - m};
        int64_t parts = xent_parts(a.M, a.V);
        // One block of rows: smaller tiles spread the vocabulary more evenly.  In a long run, tiles of 128 and 256 entries: 16
        // rows x 8,192 x 1,024 45 and 51 us, 100 x 128,256 x 4,096 899 and 942; but 200 x 32,000 x 2,048 182 and 173, 880
        // rows 401 and 356.
        if ((pairs        ? launch_scores<256, 2, true>(a, 0, (a.V + 255) / 256 * 256, pass, st)
             : pad == 128 ? launch_scores<128, 1, true>(a, 0, (a.V + 127) / 128 * 128, pass, st)
                          : launch_scores<256, 1, true>(a, 0, (a.V + 255) / 256 * 256, pass, st)) != 0)
            return -1;
        void *params[] = {&a, &pass, &parts};
        const int64_t places = more ? kXentPass : pad - m;
        if (launch(reinterpret_cast<const void *>(&xent_loss_kernel), dim3((unsigned)(places / kXentJoinX)),
                   dim3(kXentJoinX, kXentJoinY), 0, params, st) != 0)
            return -1;
    }
    for (int64_t v0 = 0; (a.dh || a.dw || a.db) && v0 < a.V; v0 += piece) {
        const XentPass none = {0, 0};
        if ((pairs        ? launch_scores<256, 2, false>(a, v0, piece, none, st)
             : pad == 128 ? launch_scores<128, 1, false>(a, v0, piece, none, st)
                          : launch_scores<256, 1, false>(a, v0, piece, none, st)) != 0)
            return -1;
        int32_t width = (int32_t)piece;
        void *params[] = {&a, &v0, &width};
        if (a.db && launch(reinterpret_cast<const void *>(&xent_bias_kernel), dim3((unsigned)((piece + 31) / 32)),
                           dim3(32, 32), 0, params, st) != 0)
            return -1;
        if ((a.dh || a.dw) && (pairs  ? sums ? launch_products<2, true>(a, v0, piece, st) : launch_products<2, false>(a, v0, piece, st)
                               : sums ? launch_products<1, true>(a, v0, piece, st)
                                      : launch_products<1, false>(a, v0, piece, st)) != 0)
            return -1;
    }
    if (a.dh && a.splits > 1 &&
        launch(reinterpret_cast<const void *>(&xent_join_kernel), dim3((unsigned)a.M), dim3(128), 0, one, st) != 0)
        return -1;
    return weighted_sum_launch(a.row_loss_c, a.weight_c, 0.f, a.M, a.loss, st);
}

}  // namespace tsa
