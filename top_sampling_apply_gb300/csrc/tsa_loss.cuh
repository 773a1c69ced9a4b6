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
    // the larger of two words' values, NaN if one is; a word's value
    __device__ static __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
        float d;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(d);
    }
    __device__ static __forceinline__ float top(uint32_t w) { return __uint_as_float(w); }
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
    __device__ static __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ float top(uint32_t w) {
        float d;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(Elem<1>::h2f(w & 0xFFFFu)), "f"(Elem<1>::h2f(w >> 16)));
        return d;
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
    __device__ static __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static __forceinline__ float top(uint32_t w) {
        float d;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__uint_as_float(w << 16)), "f"(__uint_as_float(w & 0xFFFF0000u)));
        return d;
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

// What is to be known of a row before its sums are.  It is fetched rows ahead:
// read when a row is finished, the last three cost every row a trip to memory.
struct RowMeta {
    int64_t row, tok;  // row = B: there are no more
    float w, T, c2, xt;
    float old, adv, ref;
};
template <int DT, int MODE>
__device__ __forceinline__ RowMeta row_meta(const RowLossArgs &r, int64_t b, float w, int64_t tok) {
    RowMeta m = {b, tok, w, 1.f, 1.f, -INFINITY, 0.f, 0.f, 0.f};
    if (b < r.B) {
        if (MODE == 0) {
            m.old = __ldg(r.old_logprob + b);
            m.adv = __ldg(r.advantage + b);
            if (r.ref_logprob) m.ref = __ldg(r.ref_logprob + b);
        }
        m.T = row_temperature(r, b);
        m.c2 = kLog2eL / m.T;
        m.xt = token_logit(r, static_cast<const uint8_t *>(r.logits) + (size_t)b * r.stride * Elem<DT>::SIZE,
                           r.mask ? r.mask + (size_t)b * r.mstride : nullptr, DT, tok);
    }
    return m;
}

// The loss of one row from its log-probability lp and entropy H, and its
// derivative c by lp.  min() takes the unclipped branch on a tie, where both
// branches have the same value; an advantage of 0 gives 0 even if the ratio
// overflows.
__device__ __forceinline__ float policy_row(const RowLossArgs &r, const RowMeta &mt, float lp, float H, float *c) {
    const float A = mt.adv;
    const float ratio = expf(lp - mt.old);
    float loss = 0.f, d = 0.f;
    if (A != 0.f) {
        const float s1 = ratio * A, s2 = fminf(fmaxf(ratio, r.clip_lo), r.clip_hi) * A;
        // written so that a NaN ratio stays NaN
        const bool clipped = s1 > s2;
        loss = clipped ? -s2 : -s1;
        d = clipped ? 0.f : -s1;
    }
    if (r.ref_logprob && r.kl != 0.f) {  // 0 times a term that overflows would be NaN
        const float u = mt.ref - lp;
        const float e1 = expm1f(u);
        loss += r.kl * (e1 - u);
        d -= r.kl * e1;
    }
    *c = d;
    return loss - r.ent * H;
}

// ------------------------------------------------------------ a finished row
// Fills row outputs (by one thread) and returns the gradient's numbers.
template <int MODE, bool ENT>
__device__ __forceinline__ RowScalars finish_row(const RowLossArgs &r, const RowMeta &mt, const RowStat &s,
                                                 bool writer) {
    const int64_t row = mt.row;
    const float xt = mt.xt, T = mt.T;
    RowScalars g = {0.f, 0.f};
    const float Z = s.m == INFINITY ? __int_as_float(0x7FC00000) : s.Z;
    const float lnZ = logf(Z);
    const bool live = xt > -INFINITY;
    const float lp = live ? (xt - s.m) / T - lnZ : (s.m > -INFINITY ? -INFINITY : __int_as_float(0x7FC00000));
    if (MODE == 0) {
        const float H = ENT ? lnZ - kLn2 * (s.t / Z) : 0.f;
        float c = 0.f;
        const float loss = live ? policy_row(r, mt, lp, H, &c) : 0.f;
        if (live) {
            const float wt = mt.w / T;
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
    }
    return g;
}
template <int MODE>
__device__ __forceinline__ void skip_row(const RowLossArgs &r, int64_t row) {
    r.logprob[row] = 0.f;
    if (MODE == 0) {
        r.row_loss[row] = 0.f;
        if (r.entropy) r.entropy[row] = 0.f;
    }
    if (r.fin) r.fin[row] = make_float4(0.f, MODE == 0 ? 0.f : 1.f, 0.f, 0.f);
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

// ------------------------------------------------------------ the rows, streamed
// The sums of rows of any length, without a gradient.  One persistent CTA an SM
// takes rows as streams of 44 KB stages through a ring in shared memory, filled
// by bulk copies.  22 warps reduce the stages (m, Z, t, against a reference a
// warp) and go from one row to the next without a pause, a warp of its own
// joins a row's sums and finishes it meanwhile, and another one looks for the
// rows to come.  What a row costs by itself is spread over its whole length.
// Fewer rows than SMs are shared by the C CTAs of a cluster, of which only the
// finishing warps talk to one another.  512 x 128,256 fp32 with the entropies:
// 52 us, 5.1 TB/s.
constexpr int kRowVecs = 4;                               // 16-byte vectors a thread in a stage
constexpr int kRowWarps = 22, kRowUsers = 32 * kRowWarps; // the warps that work on stages
constexpr int kRowThreads = kRowUsers + 64;               // one more to copy, one to finish rows
constexpr int kRowStage = kRowUsers * kRowVecs;           // vectors a stage
constexpr int kRowSlots = 4;                              // stages in shared memory
constexpr int kRowRing = 16;                              // rows under way at most
constexpr int kRowMaxCluster = 8;

// A row's (or a warp's) reference as its exponents are formed from it.  Near 0
// the exponent is one fused multiply-add, l c2 - R with R = m c2 rounded; the
// rounding (at most 2^-10 for |R| < 2^14, known exactly by one more fma) scales
// every term alike and is taken out of the sums.  Far from 0 it is (l - m) c2.
struct Ref {
    unsigned long long c2, neg;  // pairs: c2, and -R or -m
    bool near;
};
__device__ __forceinline__ bool near_zero(float m, float c2) { return fabsf(m * c2) < 16384.f; }
__device__ __forceinline__ Ref make_ref(float m, float c2) {
    Ref r;
    r.near = near_zero(m, c2);
    const float n = r.near ? -__fmul_rn(m, c2) : -m;
    r.c2 = pair_of(c2, c2);
    r.neg = pair_of(n, n);
    return r;
}
// How far the near form's exponents lie above (l - m) c2, and 2 to minus that.
__device__ __forceinline__ float near_shift(float m, float c2, float *f) {
    if (!near_zero(m, c2)) {
        *f = 1.f;
        return 0.f;
    }
    const float d = fmaf(m, c2, -__fmul_rn(m, c2)), z = -kLn2 * d;
    *f = fmaf(z, fmaf(z, 0.5f, 1.f), 1.f);
    return d;
}
// e and, with an entropy, the bounded exponents of two logits.  ex2.approx is
// one instruction and off by 1.5e-7 of its value at most (6e-8 rms), on average
// 5e-8 too small (measured over [-20, 0)); c2's own rounding, 1.3e-8 of itself at T = 1,
// makes distant terms too large.  The two nearly cancel: a log-probability is off by
// 3e-7 to 6e-7 rms and by less than 2e-8 on average over rows of 8,192 to 128,256
// logits, where fp32 sums of expf give the same rms and 1e-8.
template <bool ENT, bool NEAR>
__device__ __forceinline__ void exp_pair(float a, float b, const Ref &r, unsigned long long &e, unsigned long long &y) {
    const unsigned long long x = pair_of(a, b);
    y = NEAR ? fma2(x, r.c2, r.neg) : mul2(add2(x, r.neg), r.c2);
    float p, q;
    split_pair(y, p, q);
    if (ENT) {
        p = fmaxf(p, kLowExp);
        q = fmaxf(q, kLowExp);
        y = pair_of(p, q);
    }
    e = pair_of(ex2_approx(p), ex2_approx(q));
}
// A gradient element of one logit, with the bits of the paired form.
template <bool ENT>
__device__ __forceinline__ float ref_grad(float x, const Ref &r, float k1, float k2) {
    unsigned long long e, y;
    if (r.near)
        exp_pair<ENT, true>(x, x, r, e, y);
    else
        exp_pair<ENT, false>(x, x, r, e, y);
    float a, b;
    const unsigned long long kk = pair_of(k1, k1);
    split_pair(mul2(e, ENT ? fma2(pair_of(k2, k2), y, kk) : kk), a, b);
    return a;
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
// By a warp: the mask words of `count` elements from `first` on go to L2, 128
// bytes a lane.
__device__ __forceinline__ void prefetch_mask(const RowLossArgs &r, int64_t row, int32_t first, int32_t count) {
    const int32_t w = (first >> 5) + (int32_t)(threadIdx.x & 31) * 32;
    if (w <= (first + count - 1) >> 5)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(r.mask + (size_t)row * r.mstride + w));
}
// The largest of the warp's values (no NaN among them), on every lane.
__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(x));
    return m;
}

// The same, NaN if one of them is.
__device__ __forceinline__ float warp_top(float x) {
    float m;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(x));
    return m;
}
__device__ __forceinline__ void send_stat(float4 *slot, uint64_t *bar, uint32_t rank, float m, float Z, float t) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %3}, [%4];" ::"r"(
            dsmem_addr(slot, rank)),
        "f"(m), "f"(Z), "f"(t), "r"(dsmem_addr(bar, rank))
        : "memory");
}
constexpr size_t kRowSmem = (size_t)kRowSlots * kRowStage * 16;

// A warp's running sums against its reference m: in the form that m calls for
// (see Ref).
struct WarpSums {
    float m, Z, t;  // m is the warp's, Z and t the thread's
};
// 2^d for d <= 0 from e^x's series at |x| <= ln(2) / 2 (its ninth term is 5e-9),
// rounded to nearest: the factor that brings a part of a row's sums to a larger
// reference.  By ex2.approx every such factor took another 5e-8 off, two or three
// times in a long row, and a sequence's log-ratio added that up: its reward
// was off by 2.5e-6 to 3.6e-6 of itself over 2,000 rows of 128,256 bf16 logits, and
// is by 0.9e-6 to 1.3e-6 now.
__device__ __forceinline__ float exp2_factor(float d) {
    const float n = rintf(d), r = d - n;
    float p = 1.525273380405984e-5f;
    p = fmaf(p, r, 1.5403530393381608e-4f);
    p = fmaf(p, r, 1.3333558146428443e-3f);
    p = fmaf(p, r, 9.618129107628477e-3f);
    p = fmaf(p, r, 5.550410866482158e-2f);
    p = fmaf(p, r, 2.402265069591007e-1f);
    p = fmaf(fmaf(p, r, kLn2), r, 1.f);
    return n > -126.f ? __int_as_float(__float_as_int(p) + ((int)n << 23)) : 0.f;
}
// A larger reference: Z and t are brought from the old one's form to the new one's.
template <bool ENT>
__device__ __forceinline__ void raise(WarpSums &s, float m, float c2) {
    if (s.m > -INFINITY) {
        float fo, fn;
        const float d0 = near_shift(s.m, c2, &fo), d1 = near_shift(m, c2, &fn);
        // from the old form to the old m, to the new m, to the new form
        const float d = fmaxf((s.m - m) * c2, kLowExp), f = exp2_factor(d) * fo * (2.f - fn);
        // y_new = y_old - d0 + (m_old - m_new) c2 + d1
        if (ENT) s.t = f * fmaf(s.Z, d - d0 + d1, s.t);
        s.Z *= f;
    }
    s.m = m;
}
// Z and t of the first nu of a thread's vectors.
template <int DT, bool ENT, bool NEAR, int U>
__device__ __forceinline__ void add_vecs(const uint4 (&x)[U], int nu, const Ref &ref, WarpSums &s) {
    constexpr int AE = Elem<DT>::AE;
    unsigned long long Z = pair_of(s.Z, 0.f), Z2 = pair_of(0.f, 0.f), t = pair_of(s.t, 0.f), e, y;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u < nu) {
            float f[AE];
            Elem<DT>::unpack(x[u], f);
#pragma unroll
            for (int q = 0; q < AE; q += 4) {
                exp_pair<ENT, NEAR>(f[q], f[q + 1], ref, e, y);
                Z = add2(Z, e);
                if (ENT) t = fma2(e, y, t);
                exp_pair<ENT, NEAR>(f[q + 2], f[q + 3], ref, e, y);
                Z2 = add2(Z2, e);
                if (ENT) t = fma2(e, y, t);
            }
        }
    }
    float a, b;
    split_pair(add2(Z, Z2), a, b);
    s.Z = a + b;
    if (ENT) {
        split_pair(t, a, b);
        s.t = a + b;
    }
}
// One more logit.
template <bool ENT>
__device__ __forceinline__ void add_one(float x, const Ref &ref, WarpSums &s) {
    unsigned long long e, y;
    if (ref.near)
        exp_pair<ENT, true>(x, -INFINITY, ref, e, y);
    else
        exp_pair<ENT, false>(x, -INFINITY, ref, e, y);
    float a, b, ignored;
    split_pair(e, a, ignored);
    split_pair(y, b, ignored);
    s.Z += a;
    if (ENT) s.t = fmaf(a, b, s.t);
}
// The warp's sums against its largest logit itself.
template <bool ENT>
__device__ __forceinline__ float4 against_top(const WarpSums &s, float c2) {
    float Z = warp_sum_f32(s.Z), t = ENT ? warp_sum_f32(s.t) : 0.f;
    if (s.m > -INFINITY) {
        float f;
        const float d = near_shift(s.m, c2, &f);
        if (ENT) t = f * fmaf(-d, Z, t);
        Z *= f;
    }
    return make_float4(s.m, Z, t, 0.f);
}
// k1, k2, a and m of a finished row, for exponents formed from m as Ref does;
// zeros for a row that does not count (its token masked).
template <bool ENT>
__device__ __forceinline__ float4 finished_coef(const RowScalars &g, const RowStat &s, float xt, float c2) {
    if (!(xt > -INFINITY)) return make_float4(0.f, 0.f, 0.f, 0.f);
    const GradCoef k = grad_coef<ENT>(g, s);
    float f;
    const float d = near_shift(s.m, c2, &f);
    return make_float4(f * fmaf(-d, k.k2, k.k1), f * k.k2, g.a, s.m);
}

// The largest logit of the warp among the first nu vectors of its threads, NaN
// if there is one; and the vectors with -inf in the place of NaN.
template <int DT, int U>
__device__ __forceinline__ float largest(const uint4 (&x)[U], int nu) {
    using P = Pack<DT>;
    uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
    for (int u = 1; u < U; ++u) {
        if (u < nu) {
            w[0] = P::top2(w[0], x[u].x);
            w[1] = P::top2(w[1], x[u].y);
            w[2] = P::top2(w[2], x[u].z);
            w[3] = P::top2(w[3], x[u].w);
        }
    }
    return warp_top(P::top(P::top2(P::top2(w[0], w[1]), P::top2(w[2], w[3]))));
}
template <int DT, int U>
__device__ __forceinline__ void clean_all(uint4 (&x)[U], int nu) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < nu) Pack<DT>::clean(x[u]);
}
template <int DT>
__device__ __forceinline__ uint4 none_vec() {
    return DT == 0   ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
           : DT == 1 ? make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u)
                     : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
}
// The mask bits of the vector whose first element is e, in two words.
template <int AE>
__device__ __forceinline__ void mask_words(const int32_t *mrow, int32_t e, bool in, uint32_t &lo, uint32_t &hi) {
    lo = in ? (uint32_t)__ldg(mrow + (e >> 5)) : 0u;
    hi = in && (e & 31) + AE > 32 ? (uint32_t)__ldg(mrow + (e >> 5) + 1) : 0u;
}
template <int AE>
__device__ __forceinline__ uint32_t mask_bits(uint32_t lo, uint32_t hi, int32_t e) {
    return __funnelshift_r(lo, hi, (uint32_t)(e & 31)) & ((1u << AE) - 1u);
}

// The gradient of a vector: k1 e + k2 e y, in place of the logits.
template <int DT, bool ENT, bool NEAR>
__device__ __forceinline__ void grad_vec(uint4 &x, const Ref &ref, float k1, float k2) {
    constexpr int AE = Elem<DT>::AE;
    const unsigned long long a = pair_of(k1, k1), b = pair_of(k2, k2);
    float f[AE];
    Elem<DT>::unpack(x, f);
#pragma unroll
    for (int q = 0; q < AE; q += 2) {
        unsigned long long e, y;
        exp_pair<ENT, NEAR>(f[q], f[q + 1], ref, e, y);
        split_pair(mul2(e, ENT ? fma2(b, y, a) : a), f[q], f[q + 1]);
    }
    x = Pack<DT>::vec(f);
}

// `stages`: a CTA's stages of a row, of nu * kRowUsers vectors each (the last
// ones may be short or empty).
template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kRowThreads, 1) row_loss_kernel(RowLossArgs r, int lg, int stages, int nu,
                                                                  unsigned int *status) {
    using E = Elem<DT>;
    constexpr int AE = E::AE, U = kRowVecs, S = kRowSlots, RING = kRowRing;
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ float4 sums[RING][kRowWarps];           // a row's (m, Z, t) by warp
    __shared__ float4 peers[RING][kRowMaxCluster];     // and by CTA of the cluster
    __shared__ RowMeta meta[RING];
    __shared__ uint64_t full[S], empty[S];             // a stage has come; every warp has read it
    __shared__ uint64_t known[RING], summed[RING], joined[RING], fin[RING];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t C = 1u << lg, rank = C > 1 ? cluster_ctarank() : 0u;
    const int64_t step = gridDim.x >> lg, first_row = blockIdx.x >> lg;
    const bool fixed = ((size_t)r.stride * E::SIZE) % 16 == 0;  // every row lies alike
    auto logits_at = [&](int64_t b) { return static_cast<const uint8_t *>(r.logits) + (size_t)b * r.stride * E::SIZE; };
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kRowWarps);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(&known[i], 1);
            mbar_init(&summed[i], kRowWarps);
            mbar_init(&joined[i], 1);
            mbar_init(&fin[i], 1);
        }
        mbar_init_fence();
    }
    if (C > 1)
        cluster_sync();  // every CTA's barriers stand before another CTA counts on them
    else
        __syncthreads();
    pdl_launch_dependents();  // the next kernel waits for this one's end before it reads
    const int stage = nu * kRowUsers;
    bool ok = true;  // a wait that ran out ends all waiting; the status word tells

    if (warp == kRowWarps) {
        // ---- copies
        RowMeta mine = {r.B, -1, 0.f, 1.f, 1.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t found = 0;
        bool fresh = false;
        int64_t base = first_row;
        uint32_t slot = 0, phase = 1, issued = 0;
        for (uint32_t k = 0;; ++k) {
            // the next row that counts: 32 rows looked at together
            while (found == 0 && base < r.B) {
                const int64_t b = base + lane * step;
                float w = 0.f;
                int64_t tok = -1;
                const bool named = b < r.B && row_named(r, b, &w, &tok);
                mine = {b, tok, w, 1.f, 1.f, 0.f, 0.f, 0.f, 0.f};
                found = __ballot_sync(0xFFFFFFFFu, named);
                fresh = true;
                base += 32 * step;
            }
            const int who = found ? __ffs((int)found) - 1 : 0;
            const int64_t row = found ? __shfl_sync(0xFFFFFFFFu, mine.row, who) : r.B;
            const RowPlace p = place_row<DT>(r, row < r.B ? row : 0, rank, lg);
            auto copy = [&](int s) {
                int cnt = p.nv - s * stage;
                cnt = cnt < 0 ? 0 : (cnt > stage ? stage : cnt);
                if (lane == 0) ok = ok && mbar_wait_bounded(&empty[slot], phase, status);
                if (lane == 0 && ok) {
                    mbar_arrive_expect_tx(&full[slot], (uint32_t)cnt * 16u);
                    if (cnt > 0)
                        bulk_g2s(ring + slot * kRowStage,
                                 logits_at(row) + (size_t)(p.first - tid * AE) * E::SIZE + (size_t)s * stage * 16u,
                                 (uint32_t)cnt * 16u, &full[slot]);
                    ++issued;
                }
                if (r.mask) prefetch_mask(r, row, p.first - tid * AE + s * stage * AE, cnt * AE);
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1u;
                }
            };
            if (row < r.B) copy(0);
            if (fresh && ((found >> lane) & 1u))  // the rest of what is known of 32 rows, under the copy
                mine = row_meta<DT, MODE>(r, mine.row, mine.w, mine.tok);
            fresh = false;
            found &= found - 1;
            // Rows k - 16 are done with: the stages hold back this warp to
            // five rows before the summing ones, and those stay within eight of
            // the finishing one.
            if (lane == who) {
                RowMeta m = mine;
                m.row = row;
                meta[k % RING] = m;
                mbar_arrive(&known[k % RING]);
            }
            __syncwarp();
            if (row >= r.B) break;
            for (int s = 1; s < stages; ++s) copy(s);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;  // the other warps' waits for this row run out too
        }
        // no copy may land after the CTA is gone, not even after a wait that ran out
        if (lane == 0)
            for (uint32_t i = issued < S ? 0u : issued - S; i < issued; ++i)
                mbar_wait_bounded(&full[i % S], (i / S) & 1u, status);
    } else if (warp == kRowWarps + 1) {
        // ---- finished rows
        for (uint32_t k = 0;; ++k) {
            const uint32_t i = k % RING, phase = (k / RING) & 1u;
            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_bounded(&known[i], phase, status));
            const RowMeta mt = meta[i];
            if (!ok || mt.row >= r.B) break;
            if (C > 1 && lane == 0) mbar_arrive_expect_tx(&joined[i], C * 16u);
            ok = ok && mbar_wait_bounded(&summed[i], phase, status);
            auto join = [&](const float4 v, bool in) {
                RowStat s;
                s.m = warp_max(in ? v.x : -INFINITY);
                const float d = in ? (v.x == s.m ? 0.f : fmaxf((v.x - s.m) * mt.c2, kLowExp)) : kLowExp;
                const float f = exp2_factor(d);
                s.Z = warp_sum_f32(in ? v.y * f : 0.f);
                s.t = ENT ? warp_sum_f32(in ? fmaf(v.y, d, v.z) * f : 0.f) : 0.f;
                return s;
            };
            RowStat s = join(lane < kRowWarps ? sums[i][lane] : make_float4(0.f, 0.f, 0.f, 0.f), lane < kRowWarps);
            if (C > 1) {
                if (lane < (int)C) send_stat(&peers[i][rank], &joined[i], (uint32_t)lane, s.m, s.Z, s.t);
                ok = ok && mbar_wait_bounded(&joined[i], phase, status);
                s = join(lane < (int)C ? peers[i][lane] : make_float4(0.f, 0.f, 0.f, 0.f), lane < (int)C);
            }
            if (s.m == INFINITY) s.Z = __int_as_float(0x7FC00000);
            if (rank == 0) {
                const RowScalars gs = finish_row<MODE, ENT>(r, mt, s, lane == 0);
                if (r.fin && lane == 0) {
                    if (MODE == 0)
                        r.fin[mt.row] = finished_coef<ENT>(gs, s, mt.xt, mt.c2);
                    else
                        r.fin[mt.row] = make_float4(0.f, s.Z, 0.f, s.m);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&fin[i]);
        }
    } else {
        // ---- stages
        RowPlace p = place_row<DT>(r, 0, rank, lg);
        uint32_t slot = 0, phase = 0;
        int64_t zero = first_row;  // the next row that either counts or is skipped
        for (uint32_t k = 0;; ++k) {
            const uint32_t i = k % RING;
            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_bounded(&known[i], (k / RING) & 1u, status));
            const int64_t row = ok ? meta[i].row : r.B;
            if (rank == 0)
                for (int64_t b = zero + (int64_t)tid * step; b < row; b += kRowUsers * step) skip_row<MODE>(r, b);
            if (row >= r.B) break;
            zero = row + step;
            const float c2 = meta[i].c2;
            if (!fixed) p = place_row<DT>(r, row, rank, lg);
            WarpSums sum = {-INFINITY, 0.f, 0.f};
            uint32_t lo[U], hi[U];
            auto words = [&](int s) {  // a stage's mask words, under the work on the one before
                const int32_t *mrow = r.mask + (size_t)row * r.mstride;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    mask_words<AE>(mrow, p.first + (s * stage + u * kRowUsers) * AE,
                                   u < nu && tid + u * kRowUsers < p.nv - s * stage, lo[u], hi[u]);
            };
            if (r.mask) words(0);
#pragma unroll 1
            for (int s = 0; s < stages; ++s) {
                const int cnt = p.nv - s * stage;
                const int32_t e0 = p.first + s * stage * AE;
                uint4 x[U];
                ok = ok && mbar_wait_bounded(&full[slot], phase, status);
                const uint4 *in = ring + slot * kRowStage + tid;
                if (cnt >= stage) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u < nu) x[u] = in[u * kRowUsers];
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        x[u] = none_vec<DT>();
                        if (u < nu && tid + u * kRowUsers < cnt) x[u] = in[u * kRowUsers];
                    }
                }
                if (r.mask) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u < nu) mask_vec<DT>(x[u], mask_bits<AE>(lo[u], hi[u], e0 + u * kRowUsers * AE));
                    if (s + 1 < stages) words(s + 1);
                }
                float top = largest<DT>(x, nu);
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&empty[slot]);  // a stage that has not come is not free
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1u;
                }
                if (top != top) {  // NaN counts as -inf
                    clean_all<DT>(x, nu);
                    top = largest<DT>(x, nu);
                }
                float xe = -INFINITY;  // the element outside the vectors
                if (s == 0) {
                    if (p.ie >= 0 && (!r.mask || allowed_bit(r.mask + (size_t)row * r.mstride, p.ie)))
                        xe = load_clean(logits_at(row), DT, p.ie);
                    top = warp_max(fmaxf(top, xe));
                }
                if (top > sum.m) raise<ENT>(sum, top, c2);
                if (sum.m > -INFINITY) {
                    const Ref ref = make_ref(sum.m, c2);
                    if (ref.near)
                        add_vecs<DT, ENT, true>(x, nu, ref, sum);
                    else
                        add_vecs<DT, ENT, false>(x, nu, ref, sum);
                    if (s == 0 && p.ie >= 0) add_one<ENT>(xe, ref, sum);
                }
            }
            const float4 total = against_top<ENT>(sum, c2);
            // rows are finished in order; half a ring behind at most
            if (k >= RING / 2)
                ok = ok && mbar_wait_bounded(&fin[(k - RING / 2) % RING], ((k - RING / 2) / RING) & 1u, status);
            if (lane == 0) {
                sums[i][warp] = total;
                mbar_arrive(&summed[i]);
            }
        }
    }
    __syncwarp();
    if (C > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

// ------------------------------------------------------------ the rows, held
// The policy loss with its gradient, for rows that eight CTAs can hold: a
// cluster of C CTAs of 512 threads keeps a row in registers, 8 vectors a
// thread (64 KB a CTA: four CTAs for 128,256 logits in 16 bits, eight in fp32).
// A CTA's share comes by one bulk copy into shared memory and goes to registers
// at once; the next row's copy starts as soon as every warp has read it.  The
// warps send their sums to every CTA of the cluster (asynchronous stores that
// count on the receiver's barrier).  HBM reads every logit once.  (Streaming a
// row a second time from L2 instead does not work: beside the gradient's stores
// L2 keeps too little of it.  4,096 x 128,256 bf16 took 434 us so.)
//
// Two CTAs share an SM, so that one's exchange passes under the other's
// arithmetic: 16 instructions an element, and 58 % of the issue slots are used;
// waiting at a row's barriers takes the most time beside them.  What a row needs
// once, one warp does for all, another one each row: one starts the next copy,
// one looks for the row after it, one joins the sums and finishes.  4,096 x
// 128,256 bf16, an eighth of the rows skipped: 325 us, 6.1 TB/s.  (It was 353 us
// before a row's token score and arguments were fetched rows ahead; at that time
// 366 us with 256 threads of 16 vectors, and 347 us with four CTAs of 256 threads
// an SM, which needs clusters of 16 for fp32.  Looking up the arguments of 32 rows
// at a time instead of one a row cost 4 us.)
//
// Two CTAs of 512 threads leave a thread 64 registers, and half of them are the
// row.  16 to 20 bytes a thread are spilled in every row's turn, 28 to 48 with an
// entropy: a part of what that costs (8,192 x 32,000 bf16: 226 us with it, 180
// without).
//
// A warp copies the mask words of its own part of the next row into shared
// memory under the gradient of this one (72 words in 16 bits, each read from
// memory once): 1,023 x 32,001 f16 with a mask and the entropies 43
// us, 52 when each vector's words were loaded under the row's wait (39 without
// a mask).
//
// Rows of up to 16 or 32 KB take CTAs of 128 or 256 threads instead, so that an
// SM has eight or four of them under way: the exchange of a row takes as long
// as a short row's arithmetic (10,000 x 8,192 bf16: 164 us with 512 threads, 67 us
// with 128).
constexpr int kHeldVecs = 8, kHeldThreads = 512;
constexpr int kHeldCluster = 8;
constexpr size_t held_smem(int threads) { return (size_t)threads * kHeldVecs * 16; }

// The first row from b on (by steps) that counts, B if none.
__device__ __forceinline__ int64_t find_row(const RowLossArgs &r, int64_t b, int64_t step, float *w, int64_t *tok) {
    while (b < r.B && !row_named(r, b, w, tok)) b += step;
    return b < r.B ? b : r.B;
}
template <int DT, bool ENT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_held_kernel(RowLossArgs r, int lg, unsigned int *status) {
    using E = Elem<DT>;
    constexpr int AE = E::AE, U = kHeldVecs, WARPS = THREADS / 32;
    extern __shared__ __align__(128) uint4 ring[];               // the CTA's vectors of a row
    __shared__ float4 stats[2][kHeldCluster * WARPS];            // the cluster's warps, this row and the next
    __shared__ RowMeta meta[4];
    __shared__ float4 finished;                                  // k1, k2, a and m
    __shared__ uint64_t full, empty, joined[2];
    constexpr int MW = AE + 1;                                   // words that 32 vectors' bits lie in
    __shared__ uint32_t words[WARPS][U * MW + 1];                // each warp's own mask words of a row; the
                                                                 // last one is read with its bits unused
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t C = 1u << lg, rank = C > 1 ? cluster_ctarank() : 0u;
    const int64_t step = gridDim.x >> lg;
    int64_t zero = blockIdx.x >> lg;  // the next row that is either counted or set to 0
    const bool fixed = ((size_t)r.stride * E::SIZE) % 16 == 0;  // every row lies alike
    RowPlace p = place_row<DT>(r, 0, rank, lg);
    auto logits_at = [&](int64_t b) { return static_cast<const uint8_t *>(r.logits) + (size_t)b * r.stride * E::SIZE; };
    auto fetch = [&](int64_t b) {  // by one thread: the CTA's share of a row
        const RowPlace q = fixed ? p : place_row<DT>(r, b, rank, lg);
        mbar_arrive_expect_tx(&full, (uint32_t)q.nv * 16u);
        if (q.nv > 0)
            bulk_g2s(ring, logits_at(b) + (size_t)(q.first - tid * AE) * E::SIZE, (uint32_t)q.nv * 16u, &full);
    };
    auto fetch_mask = [&](int64_t b) {  // by every warp: the mask words of its vectors; 0 beyond the row
        const RowPlace q = fixed ? p : place_row<DT>(r, b, rank, lg);
        const int32_t *mrow = r.mask + (size_t)b * r.mstride;
        const int32_t w0 = (q.first - lane * AE) >> 5;
        const uint32_t n = (uint32_t)(r.V + 31) >> 5;
#pragma unroll
        for (int i = 0; i < U * MW; i += 32) {
            const int k = i + lane;
            const uint32_t w = (uint32_t)(w0 + k / MW * (THREADS * AE / 32) + k % MW);
            if (k < U * MW) cp_async_4(&words[warp][k], mrow + (w < n ? w : 0u), w < n);
        }
        cp_async_commit();
    };
    if (tid == 0) {
        mbar_init(&full, 1);
        mbar_init(&empty, WARPS);
        mbar_init(&joined[0], 1);
        mbar_init(&joined[1], 1);
        mbar_init_fence();
    }
    __syncthreads();
    if (warp == 0) {
        float w = 0.f;
        int64_t tok = -1;
        const int64_t a = find_row(r, zero, step, &w, &tok);
        if (lane == 0 && a < r.B) {
            mbar_arrive_expect_tx(&joined[0], (uint32_t)(WARPS << lg) * 16u);
            fetch(a);
        }
        __syncwarp();
        const RowMeta ma = row_meta<DT, 0>(r, a, w, tok);
        const int64_t b = find_row(r, a < r.B ? a + step : r.B, step, &w, &tok);
        const RowMeta mb = row_meta<DT, 0>(r, b, w, tok);
        if (lane == 0) {
            meta[0] = ma;
            meta[1] = mb;
        }
    }
    if (C > 1)
        cluster_sync();  // every CTA's barriers stand before another CTA counts on them
    else
        __syncthreads();
    pdl_launch_dependents();  // the next kernel waits for this one's end before it reads
    bool ok = true;  // a wait that ran out ends all waiting; the status word tells
    if (r.mask && meta[0].row < r.B) fetch_mask(meta[0].row);
    for (uint32_t turn = 0;; ++turn) {
        const uint32_t half = turn & 1u;
        const RowMeta &mt = meta[turn & 3u];
        const int64_t row = mt.row;
        for (; zero < row; zero += step) {  // rows that do not count
            if (rank == 0 && tid == 0) skip_row<0>(r, zero);
            const RowPlace q = place_row<DT>(r, zero, rank, lg);
            uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)zero * r.gstride * E::SIZE;
            if (((reinterpret_cast<uintptr_t>(logits_at(zero)) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0) {
                for (int v = tid; v < q.nv; v += THREADS)
                    __stcs(reinterpret_cast<uint4 *>(gp + (size_t)(q.first + (v - tid) * AE) * E::SIZE),
                           make_uint4(0u, 0u, 0u, 0u));
            } else {
                for (int v = tid; v < q.nv * AE; v += THREADS) Pack<DT>::store1(gp, q.first - tid * AE + v, 0.f);
            }
            if (q.ie >= 0) Pack<DT>::store1(gp, q.ie, 0.f);
        }
        if (row >= r.B) break;
        zero = row + step;
        const float c2 = mt.c2;
        const int32_t *mrow = r.mask ? r.mask + (size_t)row * r.mstride : nullptr;
        if (!fixed) p = place_row<DT>(r, row, rank, lg);
        const int nu = (p.nv + THREADS - 1) / THREADS;
        float xe = -INFINITY;
        if (p.ie >= 0) {
            xe = load_clean(logits_at(row), DT, p.ie);
            if (mrow && !allowed_bit(mrow, p.ie)) xe = -INFINITY;
        }
        uint4 x[U];
        if (ok && !mbar_wait_bounded(&full, turn & 1u, status)) {
            ok = false;
            mbar_wait_bounded(&full, turn & 1u, status);  // the copy may not land after the CTA is gone
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = none_vec<DT>();
            if (u + 1 < nu || tid + u * THREADS < p.nv) x[u] = ring[tid + u * THREADS];
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&empty);
        if (mrow) {
            cp_async_wait<0>();
            __syncwarp();
            // 32 vectors a step are a whole number of words: one place and one shift for all
            const uint32_t *mw = words[warp] + ((p.first >> 5) - ((p.first - lane * AE) >> 5));
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < nu) mask_vec<DT>(x[u], mask_bits<AE>(mw[u * MW], mw[u * MW + 1], p.first));
        }
        float top = largest<DT>(x, nu);
        if (top != top) {  // NaN counts as -inf
            clean_all<DT>(x, nu);
            top = largest<DT>(x, nu);
        }
        top = warp_max(fmaxf(top, xe));
        if (warp == (int)(turn % WARPS) && lane == 0) {  // the next row's copy
            const int64_t next = meta[(turn + 1u) & 3u].row;
            if (next < r.B && ok) {
                mbar_arrive_expect_tx(&joined[half ^ 1u], (uint32_t)(WARPS << lg) * 16u);
                ok = mbar_wait_bounded(&empty, turn & 1u, status);
                if (ok) {
                    fence_proxy_async_smem();
                    fetch(next);
                }
            }
        }
        __syncwarp();
        WarpSums sum = {top, 0.f, 0.f};
        if (top > -INFINITY) {
            const Ref ref = make_ref(top, c2);
            if (ref.near)
                add_vecs<DT, ENT, true>(x, nu, ref, sum);
            else
                add_vecs<DT, ENT, false>(x, nu, ref, sum);
            if (p.ie >= 0) add_one<ENT>(xe, ref, sum);
        }
        const float4 total = against_top<ENT>(sum, c2);
        // These slots were last read two rows ago: a warp sends after its CTA
        // has finished the row before, for which every CTA had sent, and so
        // finished the row before that.
        if (lane < (int)C)
            send_stat(&stats[half][(int)rank * WARPS + warp], &joined[half], (uint32_t)lane, total.x, total.y, total.z);
        if (warp == (int)((turn + 3u) % WARPS)) {  // finish the row
            ok = ok && mbar_wait_bounded(&joined[half], (turn >> 1) & 1u, status);
            const int n = WARPS << lg;
            RowStat s = {-INFINITY, 0.f, 0.f};
            for (int i = lane; i < n; i += 32) s.m = fmaxf(s.m, stats[half][i].x);
            s.m = warp_max(s.m);
            for (int i = lane; i < n; i += 32) {
                const float4 v = stats[half][i];
                const float d = v.x == s.m ? 0.f : fmaxf((v.x - s.m) * c2, kLowExp), f = exp2_factor(d);
                s.Z = fmaf(v.y, f, s.Z);
                if (ENT) s.t = fmaf(fmaf(v.y, d, v.z), f, s.t);
            }
            s.Z = s.m == INFINITY ? __int_as_float(0x7FC00000) : warp_sum_f32(s.Z);
            if (ENT) s.t = warp_sum_f32(s.t);
            const RowScalars gs = finish_row<0, ENT>(r, mt, s, rank == 0 && lane == 0);
            if (lane == 0) finished = finished_coef<ENT>(gs, s, mt.xt, c2);
        }
        if (warp == (int)((turn + 6u) % WARPS)) {  // look two rows ahead
            const int64_t next = meta[(turn + 1u) & 3u].row;
            float w = 0.f;
            int64_t tok = -1;
            const int64_t b = find_row(r, next < r.B ? next + step : r.B, step, &w, &tok);
            const RowMeta m2 = row_meta<DT, 0>(r, b, w, tok);
            if (lane == 0) meta[(turn + 2u) & 3u] = m2;
        }
        __syncthreads();
        if (r.mask && meta[(turn + 1u) & 3u].row < r.B) fetch_mask(meta[(turn + 1u) & 3u].row);
        const float4 k = finished;
        const bool live = mt.xt > -INFINITY;
        const Ref ref = make_ref(live ? k.w : 0.f, c2);
        uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)row * r.gstride * E::SIZE;
        const bool same = ((reinterpret_cast<uintptr_t>(logits_at(row)) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0;
        uint8_t *gv = gp + (size_t)p.first * E::SIZE;
        if (live && ref.near && same) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < nu) {
                    grad_vec<DT, ENT, true>(x[u], ref, k.x, k.y);
                    if (u + 1 < nu || tid + u * THREADS < p.nv)
                        __stcs(reinterpret_cast<uint4 *>(gv) + u * THREADS, x[u]);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (tid + u * THREADS < p.nv) {
                    if (!live)
                        x[u] = make_uint4(0u, 0u, 0u, 0u);
                    else if (ref.near)
                        grad_vec<DT, ENT, true>(x[u], ref, k.x, k.y);
                    else
                        grad_vec<DT, ENT, false>(x[u], ref, k.x, k.y);
                    if (same) {
                        __stcs(reinterpret_cast<uint4 *>(gv) + u * THREADS, x[u]);
                    } else {
                        float f[AE];
                        E::unpack(x[u], f);
#pragma unroll
                        for (int j = 0; j < AE; ++j) Pack<DT>::store1(gv, u * THREADS * AE + j, f[j]);
                    }
                }
            }
        }
        if (p.ie >= 0) Pack<DT>::store1(gp, p.ie, live ? ref_grad<ENT>(xe, ref, k.x, k.y) : 0.f);
        if (live) {
            // the token's element once more, by the thread that wrote it
            const int32_t tok = (int32_t)mt.tok, rel = tok - (p.first - tid * AE);
            const bool mine = p.ie == tok || (rel >= 0 && rel < p.nv * AE && (rel / AE) % THREADS == tid);
            if (mine) Pack<DT>::store1(gp, tok, __fadd_rn(ref_grad<ENT>(mt.xt, ref, k.x, k.y), k.z));
        }
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another may still write to it
}

// ------------------------------------------------------------ known sums
// A sum with its rounding errors beside it (Knuth's two-sum), in fp32: about
// 48 bits, so that a sequence's log-ratio keeps the differences that cancel in
// it.  (FP64 does a few operations a cycle and SM here: with it these small
// sums took 6 and 11 us.)
struct Sum2 {
    float s, c;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
        s = t;
    }
    __device__ __forceinline__ void add_product(float a, float b) {
        const float p = __fmul_rn(a, b);
        add(p);
        c = __fadd_rn(c, fmaf(a, b, -p));
    }
    __device__ __forceinline__ void add(const Sum2 &o) {
        add(o.s);
        c = __fadd_rn(c, o.c);
    }
    // infinities and NaN as the plain sum has them
    __device__ __forceinline__ float value() const { return fabsf(s) < INFINITY ? __fadd_rn(s, c) : s; }
};
// Block sum in a fixed order; the result on every thread.
template <int THREADS>
__device__ __forceinline__ Sum2 block_sum(Sum2 v, Sum2 *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto down = [&]() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Sum2 w;
            w.s = __shfl_down_sync(0xFFFFFFFFu, v.s, o);
            w.c = __shfl_down_sync(0xFFFFFFFFu, v.c, o);
            v.add(w);
        }
    };
    down();
    __syncthreads();  // sh may hold an earlier sum
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = lane < THREADS / 32 ? sh[lane] : Sum2{0.f, 0.f};
    down();
    v.s = __shfl_sync(0xFFFFFFFFu, v.s, 0);
    v.c = __shfl_sync(0xFFFFFFFFu, v.c, 0);
    return v;
}

// The gradient of rows whose coefficients are known (k1, k2, a and m in `fin`),
// element by element; grid (slices of 32 KB of a row, rows).  Rows are taken
// last to first: the sums' pass ended with the last ones, whose logits are the
// ones still in L2.  The first CTA also writes a preference loss, the mean of
// the pairs' losses, in a fixed order.  3,400 rows of 128,256 bf16 logits and
// 1,140 skipped ones: 291 us, 7.0 TB/s.
constexpr int kKnownThreads = 256;
constexpr int kKnownU = 8;

template <int DT, bool ENT>
__global__ void __launch_bounds__(kKnownThreads) row_grad_kernel(RowLossArgs r, const float *pair_loss, int64_t pairs,
                                                                 float *loss) {
    using E = Elem<DT>;
    constexpr int AE = E::AE;
    __shared__ Sum2 sh[kKnownThreads / 32];
    pdl_wait_primary();
    const int tid = threadIdx.x;
    if (loss && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        Sum2 s = {0.f, 0.f};
        for (int64_t i = tid; i < pairs; i += kKnownThreads) s.add(pair_loss[i]);
        s = block_sum<kKnownThreads>(s, sh);
        if (tid == 0) *loss = pairs > 0 ? s.value() / (float)pairs : 0.f;
    }
    const int64_t row = r.B - 1 - (int64_t)blockIdx.y - (int64_t)blockIdx.z * gridDim.y;
    if (row < 0) return;
    const uint8_t *rp = static_cast<const uint8_t *>(r.logits) + (size_t)row * r.stride * E::SIZE;
    uint8_t *gp = static_cast<uint8_t *>(r.grad) + (size_t)row * r.gstride * E::SIZE;
    const int32_t V = (int32_t)r.V, head = min((int32_t)((0u - (uint32_t)(uintptr_t)rp) & 15u) / E::SIZE, V);
    const int32_t nvec = (V - head) / AE, tail = (V - head) & (AE - 1);
    const int32_t v0 = (int32_t)blockIdx.x * kKnownThreads * kKnownU + tid, left = nvec - v0;
    const bool same = ((reinterpret_cast<uintptr_t>(rp) ^ reinterpret_cast<uintptr_t>(gp)) & 15u) == 0;
    const int32_t e_first = head + v0 * AE;
    // one element outside the vectors, by the first CTA of a row
    const int32_t ie = blockIdx.x != 0 ? -1 : (tid < head ? tid : (tid >= 8 && tid - 8 < tail ? V - tail + tid - 8 : -1));
    const float4 k = r.fin[row];
    auto store = [&](int u, const uint4 &x) {
        if (same) {
            __stcs(reinterpret_cast<uint4 *>(gp + (size_t)e_first * E::SIZE) + u * kKnownThreads, x);
        } else {
            float f[AE];
            E::unpack(x, f);
#pragma unroll
            for (int q = 0; q < AE; ++q) Pack<DT>::store1(gp, e_first + u * kKnownThreads * AE + q, f[q]);
        }
    };
    if (k.x == 0.f && k.z == 0.f && (!ENT || k.y == 0.f)) {  // skipped, or nothing to change
#pragma unroll
        for (int u = 0; u < kKnownU; ++u)
            if (u * kKnownThreads < left) store(u, make_uint4(0u, 0u, 0u, 0u));
        if (ie >= 0) Pack<DT>::store1(gp, ie, 0.f);
        return;
    }
    uint4 x[kKnownU];
#pragma unroll
    for (int u = 0; u < kKnownU; ++u) {
        x[u] = none_vec<DT>();
        if (u * kKnownThreads < left)
            x[u] = *(reinterpret_cast<const uint4 *>(rp + (size_t)e_first * E::SIZE) + u * kKnownThreads);
    }
    const int32_t *mrow = r.mask ? r.mask + (size_t)row * r.mstride : nullptr;
    if (mrow) {
        uint32_t lo[kKnownU], hi[kKnownU];
#pragma unroll
        for (int u = 0; u < kKnownU; ++u)
            mask_words<AE>(mrow, e_first + u * kKnownThreads * AE, u * kKnownThreads < left, lo[u], hi[u]);
#pragma unroll
        for (int u = 0; u < kKnownU; ++u)
            mask_vec<DT>(x[u], mask_bits<AE>(lo[u], hi[u], e_first + u * kKnownThreads * AE));
    }
    const Ref ref = make_ref(k.w, kLog2eL / row_temperature(r, row));
    const float xe = ie >= 0 && (!mrow || allowed_bit(mrow, ie)) ? load_clean(rp, DT, ie) : -INFINITY;
    const int32_t tok = (int32_t)r.tokens[row], rel = tok - (head + (v0 - tid) * AE);
    const bool mine = tok == ie || (rel >= 0 && rel < kKnownThreads * kKnownU * AE && tok < V - tail &&
                                    (rel / AE) % kKnownThreads == tid);
    const float xt = mine ? load_clean(rp, DT, tok) : 0.f;  // before it may be written over
#pragma unroll
    for (int u = 0; u < kKnownU; ++u) {
        if (u * kKnownThreads < left) {
            Pack<DT>::clean(x[u]);
            if (ref.near)
                grad_vec<DT, ENT, true>(x[u], ref, k.x, k.y);
            else
                grad_vec<DT, ENT, false>(x[u], ref, k.x, k.y);
            store(u, x[u]);
        }
    }
    if (ie >= 0) Pack<DT>::store1(gp, ie, ref_grad<ENT>(xe, ref, k.x, k.y));
    // the token's element once more, by the thread that wrote it
    if (mine) Pack<DT>::store1(gp, tok, __fadd_rn(ref_grad<ENT>(xt, ref, k.x, k.y), k.z));
}

}  // namespace loss_detail
}  // namespace tsa
