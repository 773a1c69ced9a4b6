// Row losses over vocabulary logits: what the clipped policy loss and the
// preference loss share.
//
// With x_j = l_j / T over a row's allowed tokens, every quantity follows from
// three sums against the row's largest allowed logit m:
//     e_j = exp((l_j - m) / T) = 2^((l_j - m) c2),  c2 = log2(e) / T,
//     Z = sum e_j,   t = sum e_j (l_j - m) c2,
//     ln p_j = (l_j - m) / T - ln Z,   p_j = e_j / Z,
//     H = -sum p_j ln p_j = ln Z - ln(2) t / Z,
// and a gradient on the logits is
//     g_j = a (1{j = i} - p_j) + b p_j (ln p_j + H)
// for two numbers a and b a row (b = 0 without an entropy term).
//
// The subtraction l - m comes before the product with c2: it is exact or
// rounds once at the difference's own size, so rows far from 0 (and masks of
// the type's lowest value) lose nothing.  NaN logits count as -inf, and a
// +inf logit makes the row's sums NaN, as in the selective log-softmax.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_sample_common.cuh"

namespace tsa {
namespace loss_detail {

using sample_detail::mask_vec;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eL = 1.4426950408889634f;
// An exponent this low underflows to 0 like -inf does, and stays finite in
// the entropy's products (0 times -inf would be NaN).
constexpr float kLowExp = -1.0e4f;

// ------------------------------------------------------------ element types
template <int DT> struct Pack;
template <> struct Pack<0> {
    __device__ static __forceinline__ uint4 vec(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    __device__ static __forceinline__ void store1(void *p, int64_t i, float x) { static_cast<float *>(p)[i] = x; }
    // NaN to -inf, everything else as it is
    __device__ static __forceinline__ void clean(uint4 &v) {
        v.x = __float_as_uint(fmaxf(__uint_as_float(v.x), -INFINITY));
        v.y = __float_as_uint(fmaxf(__uint_as_float(v.y), -INFINITY));
        v.z = __float_as_uint(fmaxf(__uint_as_float(v.z), -INFINITY));
        v.w = __float_as_uint(fmaxf(__uint_as_float(v.w), -INFINITY));
    }
    __device__ static __forceinline__ float vmax(const uint4 &v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};
template <> struct Pack<1> {
    __device__ static __forceinline__ uint32_t two(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static __forceinline__ uint4 vec(const float *x) {
        return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
    }
    __device__ static __forceinline__ void store1(void *p, int64_t i, float x) {
        static_cast<__half *>(p)[i] = __float2half_rn(x);
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ void clean(uint4 &v) {
        v.x = max2(v.x, 0xFC00FC00u);
        v.y = max2(v.y, 0xFC00FC00u);
        v.z = max2(v.z, 0xFC00FC00u);
        v.w = max2(v.w, 0xFC00FC00u);
    }
    __device__ static __forceinline__ float vmax(const uint4 &v) {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(Elem<1>::h2f(m & 0xFFFFu), Elem<1>::h2f(m >> 16));
    }
};
template <> struct Pack<2> {
    __device__ static __forceinline__ uint32_t two(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static __forceinline__ uint4 vec(const float *x) {
        return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
    }
    __device__ static __forceinline__ void store1(void *p, int64_t i, float x) {
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ void clean(uint4 &v) {
        v.x = max2(v.x, 0xFF80FF80u);
        v.y = max2(v.y, 0xFF80FF80u);
        v.z = max2(v.z, 0xFF80FF80u);
        v.w = max2(v.w, 0xFF80FF80u);
    }
    __device__ static __forceinline__ float vmax(const uint4 &v) {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
};

// One logit by a plain load (the gradient may be written over the logits, so
// no read here goes through the read-only path), NaN as -inf.
__device__ __forceinline__ float load_clean(const void *rp, int dt, int64_t i) {
    float x;
    if (dt == 0)
        x = static_cast<const float *>(rp)[i];
    else if (dt == 1)
        x = __half2float(static_cast<const __half *>(rp)[i]);
    else
        x = __bfloat162float(static_cast<const __nv_bfloat16 *>(rp)[i]);
    return fmaxf(x, -INFINITY);
}
__device__ __forceinline__ bool allowed_bit(const int32_t *mrow, int64_t i) {
    return ((uint32_t)__ldg(mrow + (i >> 5)) >> (uint32_t)(i & 31)) & 1u;
}

// ------------------------------------------------------------ running sums
// m: the largest logit seen (-inf: none); Z, t: the sums above against it.
struct RowStat {
    float m, Z, t;
};
// e and the exponent of one logit against m (m finite or +inf).
__device__ __forceinline__ float expo(float x, float m, float c2) { return __fmul_rn(__fsub_rn(x, m), c2); }

// Both parts against the larger maximum: the part with the smaller one is
// scaled by 2^d.  An empty part has Z = t = 0 and m = -inf; its exponent is
// -inf or NaN, and the lower bound makes the factor 0.  merge(a, b) and
// merge(b, a) have the same bits (on equal maxima the factor is 1 and the
// sums commute), so all lanes of a butterfly agree.
__device__ __forceinline__ RowStat merge(const RowStat &a, const RowStat &b, float c2) {
    const bool up = b.m > a.m;
    const RowStat hi = up ? b : a, lo = up ? a : b;
    const bool tie = hi.m == lo.m;
    const float d = tie ? 0.f : fmaxf((lo.m - hi.m) * c2, kLowExp);
    const float f = tie ? 1.f : ex2_approx(d);
    RowStat r;
    r.m = hi.m;
    r.Z = fmaf(lo.Z, f, hi.Z);
    r.t = fmaf(fmaf(lo.Z, d, lo.t), f, hi.t);
    return r;
}
__device__ __forceinline__ RowStat warp_merge(RowStat s, float c2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        RowStat b;
        b.m = __shfl_xor_sync(0xFFFFFFFFu, s.m, o);
        b.Z = __shfl_xor_sync(0xFFFFFFFFu, s.Z, o);
        b.t = __shfl_xor_sync(0xFFFFFFFFu, s.t, o);
        s = merge(s, b, c2);
    }
    return s;
}

// ------------------------------------------------------------ arguments
struct RowScalars {  // what a finished row writes and what its gradient needs
    float a, b;      // the two numbers of the gradient
};

// Whether a row takes part at all: its weight is not 0 and its token is one
// of the vocabulary.  Other rows' logits are not read.
__device__ __forceinline__ bool row_named(const RowLossArgs &r, int64_t row, float *w, int64_t *tok) {
    *w = r.weight ? __ldg(r.weight + row) : r.weight_s;
    *tok = __ldg(r.tokens + row);
    return *w != 0.f && *tok >= 0 && *tok < r.V;
}
__device__ __forceinline__ float row_temperature(const RowLossArgs &r, int64_t row) {
    const float T = r.temperature ? __ldg(r.temperature + row) : r.temperature_s;
    return T > 0.f ? T : 1.f;
}
// The token's logit: -inf where the mask excludes it.
__device__ __forceinline__ float token_logit(const RowLossArgs &r, const void *rp, const int32_t *mrow, int dt,
                                             int64_t tok) {
    if (mrow && !allowed_bit(mrow, tok)) return -INFINITY;
    return load_clean(rp, dt, tok);
}

// The loss of one row from its log-probability lp and entropy H, and its
// derivative c by lp.  min() takes the unclipped branch on a tie, where both
// branches have the same value; an advantage of 0 gives 0 even if the ratio
// overflows.
__device__ __forceinline__ float policy_row(const RowLossArgs &r, int64_t row, float lp, float H, float *c) {
    const float A = __ldg(r.advantage + row);
    const float ratio = expf(lp - __ldg(r.old_logprob + row));
    float loss = 0.f, d = 0.f;
    if (A != 0.f) {
        const float s1 = ratio * A, s2 = fminf(fmaxf(ratio, r.clip_lo), r.clip_hi) * A;
        // written so that a NaN ratio stays NaN
        const bool clipped = s1 > s2;
        loss = clipped ? -s2 : -s1;
        d = clipped ? 0.f : -s1;
    }
    if (r.ref_logprob) {
        const float u = __ldg(r.ref_logprob + row) - lp;
        const float e1 = expm1f(u);
        loss += r.kl * (e1 - u);
        d -= r.kl * e1;
    }
    *c = d;
    return loss - r.ent * H;
}

// ------------------------------------------------------------ the row, twice
// One CTA a row: the sums in one read, the gradient in a second one, which
// comes from L2 while the rows in flight fit there (152 rows of 128,256 bf16
// logits are 39 MB).  Every row length, alignment and stride; rows that fit a
// cluster's registers take row_loss_kernel instead.
constexpr int kStreamThreads = 512;
constexpr int kStreamU = 4;  // 16-byte vectors in flight a thread

__device__ __forceinline__ void stat_block(RowStat &s, RowStat *sh, float c2, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    s = warp_merge(s, c2);
    if (lane == 0) sh[warp] = s;
    __syncthreads();
    s = lane < warps ? sh[lane] : RowStat{-INFINITY, 0.f, 0.f};
    s = warp_merge(s, c2);
}

// Fills row outputs (by one thread) and returns the gradient's numbers.
template <int MODE, bool ENT>
__device__ __forceinline__ RowScalars finish_row(const RowLossArgs &r, int64_t row, const RowStat &s, float xt,
                                                 float T, float w, bool writer) {
    RowScalars g = {0.f, 0.f};
    const float Z = s.m == INFINITY ? __int_as_float(0x7FC00000) : s.Z;
    const float lnZ = logf(Z);
    const bool live = xt > -INFINITY;
    const float lp = live ? (xt - s.m) / T - lnZ : (s.m > -INFINITY ? -INFINITY : __int_as_float(0x7FC00000));
    if (MODE == 0) {
        const float H = ENT ? lnZ - kLn2 * (s.t / Z) : 0.f;
        float c = 0.f;
        const float loss = live ? policy_row(r, row, lp, H, &c) : 0.f;
        if (live) {
            const float wt = w / T;
            g.b = ENT ? wt * r.ent : 0.f;
            g.a = wt * c;
        }
        if (writer) {
            r.row_loss[row] = loss;
            r.logprob[row] = lp;
            if (ENT && r.entropy) r.entropy[row] = live ? H : 0.f;
        }
    } else if (writer) {
        r.logprob[row] = lp;
        r.row_m[row] = s.m;
        r.row_z[row] = Z;
        r.coef[row] = 0.f;
    }
    return g;
}
template <int MODE>
__device__ __forceinline__ void skip_row(const RowLossArgs &r, int64_t row) {
    r.logprob[row] = 0.f;
    if (MODE == 0) {
        r.row_loss[row] = 0.f;
        if (r.entropy) r.entropy[row] = 0.f;
    } else {
        r.row_m[row] = 0.f;
        r.row_z[row] = 1.f;
        r.coef[row] = 0.f;
    }
}

// One gradient element from e_j and its exponent y: k1 e + k2 e y, with
// k1 = (-a + b (H - ln Z)) / Z and k2 = b ln(2) / Z (ln p = ln(2) y - ln Z).
struct GradCoef {
    float k1, k2;
};
template <bool ENT>
__device__ __forceinline__ GradCoef grad_coef(const RowScalars &g, const RowStat &s) {
    // every product rounded by itself, wherever the compiler places this
    const float iz = __fdiv_rn(1.f, s.Z);
    GradCoef k;
    k.k1 = __fmul_rn(-g.a, iz);
    k.k2 = 0.f;
    if (ENT) {
        k.k2 = __fmul_rn(__fmul_rn(g.b, kLn2), iz);
        k.k1 = __fadd_rn(k.k1, __fmul_rn(k.k2, -__fmul_rn(s.t, iz)));  // b (H - ln Z) / Z
    }
    return k;
}

// The element of a logit x; `a` is added at the token.  Products and sums are
// kept apart (no fused multiply-add with `a`), so that an element has the same
// bits in the vector and the element-wise path.
template <bool ENT>
__device__ __forceinline__ float grad_el(float x, float m, float c2, const GradCoef &k) {
    float y = expo(x, m, c2);
    if (ENT) y = fmaxf(y, kLowExp);
    const float e = ex2_approx(y);
    return __fmul_rn(e, ENT ? fmaf(k.k2, y, k.k1) : k.k1);
}

template <int DT, int MODE, bool GRAD, bool ENT>
__global__ void __launch_bounds__(kStreamThreads) row_loss_stream_kernel(RowLossArgs r) {
    using E = Elem<DT>;
    constexpr int AE = E::AE;
    __shared__ RowStat sh[kStreamThreads / 32];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint8_t *rp = static_cast<const uint8_t *>(r.logits) + (size_t)row * r.stride * E::SIZE;
    uint8_t *gp = GRAD ? static_cast<uint8_t *>(r.grad) + (size_t)row * r.gstride * E::SIZE : nullptr;
    const int32_t *mrow = r.mask ? r.mask + (size_t)row * r.mstride : nullptr;
    const int32_t V = (int32_t)r.V;
    const Slice32 g = make_slice32<AE, E::SIZE>(rp, V, 0, 1);
    const bool same = GRAD && ((reinterpret_cast<uintptr_t>(rp) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0;
    float w;
    int64_t tok;
    const bool named = row_named(r, row, &w, &tok);
    if (!named) {
        if (tid == 0) skip_row<MODE>(r, row);
        if (GRAD) {
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            if (same) {
                for (int32_t v = tid; v < g.nvec; v += kStreamThreads)
                    __stcs(reinterpret_cast<uint4 *>(gp + (size_t)(g.head + v * AE) * E::SIZE), z);
                if (tid < g.head) Pack<DT>::store1(gp, tid, 0.f);
                if (tid < g.tail) Pack<DT>::store1(gp, g.head + g.nvec * AE + tid, 0.f);
            } else {
                for (int32_t i = tid; i < V; i += kStreamThreads) Pack<DT>::store1(gp, i, 0.f);
            }
        }
        return;
    }
    const float T = row_temperature(r, row), c2 = kLog2eL / T;
    const float xt = token_logit(r, rp, mrow, DT, tok);
    auto fetch = [&](int32_t v, uint4 &x) {  // a cleaned, masked vector
        const int32_t e = g.head + v * AE;
        // a plain load: the gradient may be written over the logits
        x = *reinterpret_cast<const uint4 *>(rp + (size_t)e * E::SIZE);
        if (mrow) {
            const uint32_t lo = (uint32_t)__ldg(mrow + (e >> 5));
            const uint32_t hi = ((e & 31) + AE > 32) ? (uint32_t)__ldg(mrow + (e >> 5) + 1) : 0u;
            mask_vec<DT>(x, __funnelshift_r(lo, hi, (uint32_t)(e & 31)) & ((1u << AE) - 1u));
        }
        Pack<DT>::clean(x);
    };
    auto fetch1 = [&](int32_t i) {
        return mrow && !allowed_bit(mrow, i) ? -INFINITY : load_clean(rp, DT, i);
    };
    RowStat s = {-INFINITY, 0.f, 0.f};
    auto add1 = [&](float x) {
        if (x > -INFINITY) s = merge(s, RowStat{x, x == INFINITY ? __int_as_float(0x7FC00000) : 1.f, 0.f}, c2);
    };
    if (tid < g.head) add1(fetch1(tid));
    if (tid < g.tail) add1(fetch1(g.head + g.nvec * AE + tid));
    for (int32_t v0 = tid; v0 < g.nvec; v0 += kStreamThreads * kStreamU) {
        uint4 x[kStreamU];
        float bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kStreamU; ++u) {
            const int32_t v = v0 + u * kStreamThreads;
            if (v < g.nvec)
                fetch(v, x[u]);
            else {
                float none[AE];
#pragma unroll
                for (int k = 0; k < AE; ++k) none[k] = -INFINITY;
                x[u] = Pack<DT>::vec(none);
            }
        }
#pragma unroll
        for (int u = 0; u < kStreamU; ++u) bm = fmaxf(bm, Pack<DT>::vmax(x[u]));
        if (bm > s.m) s = merge(s, RowStat{bm, 0.f, 0.f}, c2);
        if (s.m > -INFINITY) {
#pragma unroll
            for (int u = 0; u < kStreamU; ++u) {
                float f[AE];
                E::unpack(x[u], f);
#pragma unroll
                for (int k = 0; k < AE; ++k) {
                    float y = expo(f[k], s.m, c2);
                    if (ENT) y = fmaxf(y, kLowExp);
                    const float e = ex2_approx(y);
                    s.Z += e;
                    if (ENT) s.t = fmaf(e, y, s.t);
                }
            }
        }
    }
    stat_block(s, sh, c2, kStreamThreads / 32);
    if (s.m == INFINITY) s.Z = __int_as_float(0x7FC00000);
    const RowScalars gs = finish_row<MODE, ENT>(r, row, s, xt, T, w, tid == 0);
    if (!GRAD) return;
    // a row that does not count (its token masked) has a = b = 0: zeros
    const bool live = xt > -INFINITY;
    const GradCoef k = live ? grad_coef<ENT>(gs, s) : GradCoef{0.f, 0.f};
    const float m = live ? s.m : 0.f;
    auto grad1 = [&](float x) { return grad_el<ENT>(x, m, c2, k); };
    auto store_el = [&](int32_t i) {
        float f = live ? grad1(fetch1(i)) : 0.f;
        if (i == tok && live) f = __fadd_rn(f, gs.a);
        Pack<DT>::store1(gp, i, f);
    };
    if (!same) {
        for (int32_t i = tid; i < V; i += kStreamThreads) store_el(i);
        return;
    }
    if (tid < g.head) store_el(tid);
    if (tid < g.tail) store_el(g.head + g.nvec * AE + tid);
    for (int32_t v = tid; v < g.nvec; v += kStreamThreads) {
        float f[AE];
        if (live) {
            uint4 x;
            fetch(v, x);
            E::unpack(x, f);
            const int32_t e0 = g.head + v * AE;
#pragma unroll
            for (int q = 0; q < AE; ++q) {
                f[q] = grad1(f[q]);
                if (e0 + q == (int32_t)tok) f[q] = __fadd_rn(f[q], gs.a);
            }
        } else {
#pragma unroll
            for (int q = 0; q < AE; ++q) f[q] = 0.f;
        }
        __stcs(reinterpret_cast<uint4 *>(gp + (size_t)(g.head + v * AE) * E::SIZE), Pack<DT>::vec(f));
    }
}

// ------------------------------------------------------------ the row, once
// A cluster of C CTAs takes a row: 512 threads with eight 16-byte vectors each
// are 64 KB a CTA, so that a row of 128,256 logits takes four CTAs in 16 bits
// and eight in fp32.  Clusters are persistent.  A row's share comes by one bulk
// copy into shared memory, goes to registers at once, and the next row's copy
// starts as soon as every warp has read it, so that HBM works while the
// maximum, the sums and the gradient are formed from the registers.  The warps
// send their (m, Z, t) to every CTA of the cluster (asynchronous stores that
// count on the receiver's barrier); one warp a CTA joins them and finishes the
// row for the others.
//
// The issue slots are the scarce part: reading and writing a bf16 logit at
// 6.7 TB/s leaves 22 instructions an element.  So 16-bit maxima and the NaN
// test work on pairs, sums and products on packed fp32 pairs, addresses are
// one base and constants, and a row's scalars are computed by one warp.
constexpr int kRowVecs = 8, kRowThreads = 512;

// e and, with an entropy, the bounded exponents of two logits.
template <bool ENT>
__device__ __forceinline__ void exp_pair(float a, float b, unsigned long long negm, unsigned long long c2,
                                         unsigned long long &e, unsigned long long &y) {
    y = mul2(add2(pair_of(a, b), negm), c2);
    float p, q;
    split_pair(y, p, q);
    if (ENT) {
        p = fmaxf(p, kLowExp);
        q = fmaxf(q, kLowExp);
        y = pair_of(p, q);
    }
    e = pair_of(ex2_approx(p), ex2_approx(q));
}

// A CTA's share of one row: this thread's first vector's element, the CTA's
// vectors, and its one element of the misaligned head (first CTA) or tail
// (last CTA), -1 for none.  2^lg CTAs share the row's vectors.
struct RowPlace {
    int32_t first, nv, ie;
};
template <int DT>
__device__ __forceinline__ RowPlace place_row(const RowLossArgs &r, int64_t row, uint32_t rank, int lg) {
    using E = Elem<DT>;
    const uintptr_t at = reinterpret_cast<uintptr_t>(r.logits) + (size_t)row * r.stride * E::SIZE;
    const int32_t V = (int32_t)r.V, tid = (int32_t)threadIdx.x;
    const int32_t head = min((int32_t)((0u - (uint32_t)at) & 15u) / E::SIZE, V);
    const int32_t nvec = (V - head) / E::AE, tail = (V - head) & (E::AE - 1);
    const int32_t c0 = (int32_t)((rank * (uint32_t)nvec) >> lg), c1 = (int32_t)(((rank + 1) * (uint32_t)nvec) >> lg);
    RowPlace p;
    p.first = head + (c0 + tid) * E::AE;
    p.nv = c1 - c0;
    p.ie = -1;
    if (rank == 0 && tid < head) p.ie = tid;
    if (rank + 1 == 1u << lg && tid >= 8 && tid - 8 < tail) p.ie = V - tail + (tid - 8);
    return p;
}
// The largest of the warp's values (no NaN among them), on every lane.
__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(x));
    return m;
}

__device__ __forceinline__ void send_stat(float4 *slot, uint64_t *bar, uint32_t rank, float m, float Z, float t) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %3}, [%4];" ::"r"(
            dsmem_addr(slot, rank)),
        "f"(m), "f"(Z), "f"(t), "r"(dsmem_addr(bar, rank))
        : "memory");
}
__device__ __forceinline__ void arrive_one(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
constexpr size_t kRowSmem = (size_t)kRowThreads * kRowVecs * 16;

template <int DT, int MODE, bool GRAD, bool ENT>
__global__ void __launch_bounds__(kRowThreads, 2) row_loss_kernel(RowLossArgs r, int lg, unsigned int *status) {
    using E = Elem<DT>;
    constexpr int AE = E::AE, U = kRowVecs, THREADS = kRowThreads, WARPS = THREADS / 32;
    extern __shared__ __align__(128) uint4 buf[];  // the CTA's vectors of a row, padded with -inf
    __shared__ float4 stats[2][8 * WARPS];         // every warp of the cluster, for this row and the next
    __shared__ uint64_t full, empty, joined[2];
    __shared__ float4 finished;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t C = 1u << lg, rank = C > 1 ? cluster_ctarank() : 0u;
    const int64_t step = gridDim.x >> lg;
    int64_t row = blockIdx.x >> lg;
    const uint4 none = DT == 0 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                       : DT == 1 ? make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u)
                                 : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    if (tid == 0) {
        mbar_init(&full, 1);
        mbar_init(&empty, WARPS);
        mbar_init(&joined[0], 1);
        mbar_init(&joined[1], 1);
        mbar_init_fence();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) buf[tid + u * THREADS] = none;
    fence_proxy_async_smem();
    if (C > 1)
        cluster_sync();  // every CTA's barriers stand before another CTA counts on them
    else
        __syncthreads();
    const bool fixed = ((size_t)r.stride * E::SIZE) % 16 == 0;  // every row lies alike
    auto logits_at = [&](int64_t b) { return static_cast<const uint8_t *>(r.logits) + (size_t)b * r.stride * E::SIZE; };
    auto zero_row = [&](int64_t b) {
        if (rank == 0 && tid == 0) skip_row<MODE>(r, b);
        if (!GRAD) return;
        const RowPlace q = place_row<DT>(r, b, rank, lg);
        uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)b * r.gstride * E::SIZE;
        if (((reinterpret_cast<uintptr_t>(logits_at(b)) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0) {
            for (int v = tid; v < q.nv; v += THREADS)
                __stcs(reinterpret_cast<uint4 *>(gp + (size_t)(q.first + (v - tid) * AE) * E::SIZE),
                       make_uint4(0u, 0u, 0u, 0u));
        } else {
            for (int i = tid; i < q.nv * AE; i += THREADS) Pack<DT>::store1(gp, q.first - tid * AE + i, 0.f);
        }
        if (q.ie >= 0) Pack<DT>::store1(gp, q.ie, 0.f);
    };
    auto fetch = [&](int64_t b, const RowPlace &q) {  // by thread 0: the CTA's share of a row
        mbar_arrive_expect_tx(&full, (uint32_t)q.nv * 16u);
        if (q.nv > 0)
            bulk_g2s(buf, logits_at(b) + (size_t)(q.first - tid * AE) * E::SIZE, (uint32_t)q.nv * 16u, &full);
    };
    float w;
    int64_t tok;
    while (row < r.B && !row_named(r, row, &w, &tok)) {
        zero_row(row);
        row += step;
    }
    RowPlace p = place_row<DT>(r, row < r.B ? row : 0, rank, lg);
    if (row < r.B && tid == 0) fetch(row, p);
    bool ok = true;  // a wait that ran out ends all waiting; the status word tells
    for (uint32_t turn = 0; row < r.B; ++turn) {
        const uint32_t half = turn & 1u;
        if (tid == 0) mbar_arrive_expect_tx(&joined[half], (uint32_t)(WARPS << lg) * 16u);
        const uint8_t *rp = logits_at(row);
        const int32_t *mrow = r.mask ? r.mask + (size_t)row * r.mstride : nullptr;
        const float T = row_temperature(r, row), c2 = kLog2eL / T;
        const float xt = token_logit(r, rp, mrow, DT, tok);
        float xe = -INFINITY;
        if (p.ie >= 0 && (!mrow || allowed_bit(mrow, p.ie))) xe = load_clean(rp, DT, p.ie);
        // the next row that counts
        int64_t next = row + step, tok_next = -1;
        float w_next = 0.f;
        while (next < r.B && !row_named(r, next, &w_next, &tok_next)) next += step;
        const RowPlace pn = fixed || next >= r.B ? p : place_row<DT>(r, next, rank, lg);
        const int nu = (p.nv + THREADS - 1) / THREADS;

        ok = ok && mbar_wait_bounded(&full, turn & 1u, status);
        uint4 x[U];
        // The token's logit belongs to the row, so it may raise a warp's
        // reference; and a warp has then read it before it sends its sums,
        // after which another CTA may write a gradient over it.
        float mx = fmaxf(xe, xt);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < nu) {
                x[u] = buf[tid + u * THREADS];
                if (mrow && tid + u * THREADS < p.nv) {
                    const int32_t e = p.first + u * THREADS * AE;
                    const uint32_t lo = (uint32_t)__ldg(mrow + (e >> 5));
                    const uint32_t hi = ((e & 31) + AE > 32) ? (uint32_t)__ldg(mrow + (e >> 5) + 1) : 0u;
                    mask_vec<DT>(x[u], __funnelshift_r(lo, hi, (uint32_t)(e & 31)) & ((1u << AE) - 1u));
                }
                Pack<DT>::clean(x[u]);
                mx = fmaxf(mx, Pack<DT>::vmax(x[u]));
            }
        }
        if (pn.nv < p.nv) {  // shared memory past the next row's share is padding again
            __syncthreads();
            if (tid < p.nv - pn.nv) buf[pn.nv + tid] = none;
        }
        mx = warp_max(mx);
        if (lane == 0) arrive_one(&empty);
        if (tid == 0) {
            ok = ok && mbar_wait_bounded(&empty, turn & 1u, status);
            if (next < r.B) {
                fence_proxy_async_smem();
                fetch(next, pn);
            }
        }
        __syncwarp();
        float sz = 0.f, st = 0.f;
        if (mx > -INFINITY) {
            const unsigned long long negm = pair_of(-mx, -mx), cc = pair_of(c2, c2);
            unsigned long long Z = pair_of(0.f, 0.f), t = Z;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < nu) {
                    float f[AE];
                    E::unpack(x[u], f);
#pragma unroll
                    for (int q = 0; q < AE; q += 2) {
                        unsigned long long e, y;
                        exp_pair<ENT>(f[q], f[q + 1], negm, cc, e, y);
                        Z = add2(Z, e);
                        if (ENT) t = fma2(e, y, t);
                    }
                }
            }
            if (p.ie >= 0) {
                unsigned long long e, y;
                exp_pair<ENT>(xe, -INFINITY, negm, cc, e, y);
                Z = add2(Z, e);
                if (ENT) t = fma2(e, y, t);
            }
            float a, b;
            split_pair(Z, a, b);
            sz = warp_sum_f32(a + b);
            if (ENT) {
                split_pair(t, a, b);
                st = warp_sum_f32(a + b);
            }
        }
        // These slots were last read two rows ago: a warp sends a row's sums
        // only after its CTA has finished the row before, for which it had
        // every other CTA's sums of that row.
        if (lane < (int)C) send_stat(&stats[half][(int)rank * WARPS + warp], &joined[half], (uint32_t)lane, mx, sz, st);
        if (warp == 0) {
            ok = ok && mbar_wait_bounded(&joined[half], (turn >> 1) & 1u, status);
            if (GRAD || rank == 0) {
                const int n = WARPS << lg;
                RowStat s = {-INFINITY, 0.f, 0.f};
                for (int i = lane; i < n; i += 32) s.m = fmaxf(s.m, stats[half][i].x);
                s.m = warp_max(s.m);
                for (int i = lane; i < n; i += 32) {
                    const float4 v = stats[half][i];
                    const float d = v.x == s.m ? 0.f : fmaxf((v.x - s.m) * c2, kLowExp), f = ex2_approx(d);
                    s.Z = fmaf(v.y, f, s.Z);
                    if (ENT) s.t = fmaf(fmaf(v.y, d, v.z), f, s.t);
                }
                s.Z = s.m == INFINITY ? __int_as_float(0x7FC00000) : warp_sum_f32(s.Z);
                if (ENT) s.t = warp_sum_f32(s.t);
                const RowScalars gs = finish_row<MODE, ENT>(r, row, s, xt, T, w, rank == 0 && lane == 0);
                if (GRAD && lane == 0) {
                    // a row that does not count (its token masked) gets zeros
                    const GradCoef kc = xt > -INFINITY ? grad_coef<ENT>(gs, s) : GradCoef{0.f, 0.f};
                    finished = make_float4(kc.k1, kc.k2, gs.a, s.m);
                }
            }
        }
        __syncthreads();
        if (GRAD) {
            const float4 fin = finished;
            const GradCoef k = {fin.x, fin.y};
            const float m = fin.w;
            const bool live = xt > -INFINITY;
            uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)row * r.gstride * E::SIZE;
            const bool same = ((reinterpret_cast<uintptr_t>(rp) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0;
            uint8_t *gv = gp + (size_t)p.first * E::SIZE;
            const unsigned long long negm = pair_of(-m, -m), cc = pair_of(c2, c2), k1 = pair_of(k.k1, k.k1),
                                     k2 = pair_of(k.k2, k.k2);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < nu) {
                    float f[AE];
                    E::unpack(x[u], f);
#pragma unroll
                    for (int q = 0; q < AE; q += 2) {
                        unsigned long long e, y;
                        exp_pair<ENT>(f[q], f[q + 1], negm, cc, e, y);
                        split_pair(mul2(e, ENT ? fma2(k2, y, k1) : k1), f[q], f[q + 1]);
                    }
                    if (!live) {
#pragma unroll
                        for (int q = 0; q < AE; ++q) f[q] = 0.f;
                    }
                    if (tid + u * THREADS < p.nv) {
                        if (same) {
                            __stcs(reinterpret_cast<uint4 *>(gv) + u * THREADS, Pack<DT>::vec(f));
                        } else {
#pragma unroll
                            for (int q = 0; q < AE; ++q) Pack<DT>::store1(gv, u * THREADS * AE + q, f[q]);
                        }
                    }
                }
            }
            if (p.ie >= 0) Pack<DT>::store1(gp, p.ie, live ? grad_el<ENT>(xe, m, c2, k) : 0.f);
            if (live) {
                // the token's element once more, by the thread that wrote it
                const int32_t rel = (int32_t)tok - (p.first - tid * AE);
                const bool mine = p.ie == (int32_t)tok ||
                                  (rel >= 0 && rel < p.nv * AE && (rel / AE) % THREADS == tid);
                if (mine) Pack<DT>::store1(gp, tok, __fadd_rn(grad_el<ENT>(xt, m, c2, k), fin.z));
            }
        }
        for (row += step; row < next; row += step) zero_row(row);
        row = next;
        w = w_next;
        tok = tok_next;
        p = pn;
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

// ------------------------------------------------------------ known sums
// The gradient of a row whose m, Z and coefficient are known:
// coef / T (1{j = i} - p_j), element by element; grid (slices of a row, rows).
// Rows are taken last to first: the sums' pass ended with the last ones,
// whose logits are the ones still in L2.
constexpr int kKnownThreads = 256;
constexpr int kKnownU = 4;

template <int DT>
__global__ void __launch_bounds__(kKnownThreads) row_grad_kernel(RowLossArgs r) {
    using E = Elem<DT>;
    constexpr int AE = E::AE;
    pdl_wait_primary();
    const int tid = threadIdx.x;
    const int64_t row = r.B - 1 - (int64_t)blockIdx.y - (int64_t)blockIdx.z * gridDim.y;
    if (row < 0) return;
    const uint8_t *rp = static_cast<const uint8_t *>(r.logits) + (size_t)row * r.stride * E::SIZE;
    uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)row * r.gstride * E::SIZE;
    const Slice32 g = make_slice32<AE, E::SIZE>(rp, (int32_t)r.V, blockIdx.x, gridDim.x);
    const bool same = ((reinterpret_cast<uintptr_t>(rp) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0;
    const float coef = r.coef[row];
    const bool live = coef != 0.f;
    const float T = row_temperature(r, row), c2 = kLog2eL / T, m = r.row_m[row];
    const float a = coef / T;
    const GradCoef k = {-a / r.row_z[row], 0.f};
    const int64_t tok = r.tokens[row];
    auto store_el = [&](int32_t i) {
        float f = live ? grad_el<false>(load_clean(rp, DT, i), m, c2, k) : 0.f;
        if (live && i == tok) f = __fadd_rn(f, a);
        Pack<DT>::store1(gp, i, f);
    };
    if (!same) {
        for (int32_t i = g.lo + tid; i < g.hi; i += kKnownThreads) store_el(i);
        return;
    }
    if (g.lo == 0 && tid < g.head) store_el(tid);
    if (g.hi == (int32_t)r.V && tid < g.tail) store_el(g.hi - g.tail + tid);
    for (int32_t v0 = g.vc0 + tid; v0 < g.vc0 + g.nv; v0 += kKnownThreads * kKnownU) {
        uint4 x[kKnownU];
#pragma unroll
        for (int u = 0; u < kKnownU; ++u) {
            const int32_t v = v0 + u * kKnownThreads;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (live && v < g.vc0 + g.nv) {
                x[u] = *reinterpret_cast<const uint4 *>(rp + (size_t)(g.head + v * AE) * E::SIZE);
                Pack<DT>::clean(x[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kKnownU; ++u) {
            const int32_t v = v0 + u * kKnownThreads;
            if (v >= g.vc0 + g.nv) continue;
            const int32_t e0 = g.head + v * AE;
            if (live) {
                float f[AE];
                E::unpack(x[u], f);
#pragma unroll
                for (int q = 0; q < AE; ++q) {
                    f[q] = grad_el<false>(f[q], m, c2, k);
                    if (e0 + q == (int32_t)tok) f[q] = __fadd_rn(f[q], a);
                }
                x[u] = Pack<DT>::vec(f);
            }
            __stcs(reinterpret_cast<uint4 *>(gp + (size_t)e0 * E::SIZE), x[u]);
        }
    }
}

}  // namespace loss_detail
}  // namespace tsa
