// AdamW over many tensors in one launch, with 32-bit or 8-bit states.
//
//     m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2,
//     p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once: 28 bytes with fp32 everything, 10
// with bf16 parameters and gradients and 8-bit states.  The tensors' pointers
// travel in the launch's parameters (up to 512 tensors a launch; no table in
// device memory, nothing to copy, and the launch can be captured).
//
// 8-bit states keep three mantissa bits and an exponent relative to their
// block of 256 elements, so that decoding is an integer addition and a shift:
// a code c != 0 of a block with base b is the float with bits (c + 8 b) << 20.
// One warp handles one block (8 elements a lane), and the block's base comes
// from one warp-wide maximum.
//   - v is rounded stochastically.  A step changes v by about 1 - b2 of its
//     distance to g^2 (0.1 % for b2 = 0.999), and a code step is 6 to 12 %:
//     to nearest, v would stop growing at a few hundredths of E g^2.  A value
//     above 0 keeps code 1 at least, since v = 0 beside m != 0 would divide
//     by eps.
//   - m is rounded to nearest: a step renews 10 % of it, above half a code
//     step, and its sign and size only steer one update.
//   - bf16 parameters are rounded stochastically: updates are a few thousandths
//     of a bf16 step near the end of training.
// The random word of element i of tensor k is word i & 3 of the Philox block
// of counter (i >> 2, k, offset) under key seed, as sample's draw has it: its
// low half rounds v, its high half p.
//
// m' and v' are formed without fused multiply-adds, in the order written
// above: a value near a code's rounding point then takes the same code
// wherever the same fp32 arithmetic is used.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"

namespace tsa {

namespace {

constexpr int kAdThreads = 128;
constexpr int kAdPer = 8;                          // elements a lane: a warp is one block of 256
constexpr int kAdIter = kAdThreads * kAdPer;       // elements a CTA takes at a time
constexpr int kAdFew = 48, kAdMany = 512;          // tensors in a launch's parameters

template <int N>
struct AdamTable {
    AdamTensor t[N];
    uint32_t start[N + 1];  // first chunk of each tensor
    int32_t count;
    int32_t iters;          // kAdIter-element steps a chunk
};

// The tensor a chunk belongs to.
template <int N>
__device__ __forceinline__ int find_tensor(const AdamTable<N> &tab, uint32_t chunk) {
    int lo = 0, hi = tab.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.start[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
__device__ __forceinline__ bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Eight consecutive elements as they lie in memory (whole: 16-byte aligned and
// all there; else element by element, 0 past cnt), and as floats.
template <int DT>
struct Eight {
    uint4 w[DT == 0 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, int64_t i, int cnt, bool whole) {
        if (whole) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + i * (DT == 0 ? 4 : 2));
            w[0] = __ldcs(p);
            if constexpr (DT == 0) w[1] = __ldcs(p + 1);
            return;
        }
        uint32_t u[DT == 0 ? 8 : 4] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= cnt) continue;
            if constexpr (DT == 0)
                u[k] = static_cast<const uint32_t *>(base)[i + k];
            else
                u[k >> 1] |= (uint32_t)static_cast<const uint16_t *>(base)[i + k] << (16 * (k & 1));
        }
        w[0] = make_uint4(u[0], u[1], u[2], u[3]);
        if constexpr (DT == 0) w[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        Elem<DT>::unpack(w[0], x);
        if constexpr (DT == 0) {
            x[4] = __uint_as_float(w[1].x);
            x[5] = __uint_as_float(w[1].y);
            x[6] = __uint_as_float(w[1].z);
            x[7] = __uint_as_float(w[1].w);
        }
    }
};
__device__ __forceinline__ void store8_f32(void *base, int64_t i, int cnt, bool whole, const float (&x)[8]) {
    float *p = static_cast<float *>(base) + i;
    if (whole) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < cnt) p[k] = x[k];
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *base, int64_t i, int cnt, bool whole) {
    if (whole) return __ldcs(reinterpret_cast<const uint2 *>(base + i));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < cnt) w[k >> 2] |= (uint32_t)base[i + k] << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t *base, int64_t i, int cnt, bool whole, uint2 c) {
    if (whole) {
        __stcs(reinterpret_cast<uint2 *>(base + i), c);
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < cnt) base[i + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
}
// bf16 by adding 16 random bits below the kept ones; non-finite values as they
// are (a NaN keeps its quiet bit, which is among the kept ones).
__device__ __forceinline__ uint32_t bf16_stochastic(float x, uint32_t word) {
    const uint32_t b = __float_as_uint(x);
    return ((b & 0x7F800000u) == 0x7F800000u ? b : b + (word >> 16)) >> 16;
}
__device__ __forceinline__ float decode_v(uint32_t c, uint32_t b8) {
    return c ? __uint_as_float((c + b8) << 20) : 0.f;
}
__device__ __forceinline__ float decode_m(uint32_t c, uint32_t b8) {
    const uint32_t k = c & 127u;
    return k ? __uint_as_float(((k + b8) << 20) | ((c & 128u) << 24)) : 0.f;
}
__device__ __forceinline__ bool finite_bits(uint32_t mag) { return mag < 0x7F800000u; }
// The base of a block from its elements' magnitudes' bits: the warp's largest
// exponent less `span`, at least 0.  All 32 lanes call this.
__device__ __forceinline__ uint32_t block_base(const uint32_t (&mag)[8], uint32_t span) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, finite_bits(mag[k]) ? mag[k] : 0u);
    top = __reduce_max_sync(0xFFFFFFFFu, top) >> 23;
    return top > span ? top - span : 0u;
}

// ------------------------------------------------------------ 8-bit codes
// Two ways to read and write codes.  The general one handles code 0, values
// under a block's range and non-finite ones, element by element in integers:
// with them alone a step took 106 instructions an element, 70 of them on the
// half-rate integer pipe, and that bounded it (256 million bf16 parameters:
// 1,040 us).  With the others it takes 57, and 560 us, 4.6 TB/s: the issue slots
// still bound it, ten of the 57 being the random words.  Seven CTAs an SM leave 72
// registers a thread, and 16 to 72 bytes of them are spilled (the most with 16-bit
// parameters and gradients).
// The other one is for a warp whose 256 elements need none of that:
//   - exp_avg's codes from 9 on are the bytes of e4m3, so
//     the conversion instructions read and round (to nearest, ties to even)
//     two at once, on values scaled by a power of two;
//   - exp_avg_sq's are taken from the upper byte of the shifted float bits.
// A warp decides by votes, on the codes it read and on those it would write.

// Any of four codes under 9, or 127 (e4m3's NaN).  Codes under 8 are subnormal
// in e4m3, and 8 may have been rounded up from there, on a coarser grid.
__device__ __forceinline__ bool not_e4m3(uint32_t w) {
    const uint32_t x = w & 0x7F7F7F7Fu;
    return ((x + 0x77777777u) & ~(x + 0x01010101u) & 0x80808080u) != 0x80808080u;
}
__device__ __forceinline__ bool zero_byte(uint32_t w) { return ((w - 0x01010101u) & ~w & 0x80808080u) != 0u; }
__device__ __forceinline__ float two_to(uint32_t biased) { return __uint_as_float(biased << 23); }

// A code's value is 2^(b - 120) times its e4m3 value.
__device__ __forceinline__ void decode_m_fast(uint2 c, uint32_t b, float (&m)[8]) {
    const float sc = two_to(b + 7u);
    const unsigned long long s2 = pair_of(sc, sc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(h ? c.y : c.x));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        split_pair(mul2(pair_of(a.x, a.y), s2), m[4 * h], m[4 * h + 1]);
        split_pair(mul2(pair_of(d.x, d.y), s2), m[4 * h + 2], m[4 * h + 3]);
    }
}
__device__ __forceinline__ void decode_v_fast(uint2 c, uint32_t b, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
        v[q] = __uint_as_float(__byte_perm(q < 4 ? c.x : c.y, 0u, 0x4440u | (uint32_t)(q & 3)) * 0x100000u + (b << 23));
}
__device__ __forceinline__ uint2 encode_m_fast(const float (&m)[8], uint32_t b) {
    const float sc = two_to(247u - b);
    const unsigned long long s2 = pair_of(sc, sc);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float a, d, e, f;
        split_pair(mul2(pair_of(m[4 * h], m[4 * h + 1]), s2), a, d);
        split_pair(mul2(pair_of(m[4 * h + 2], m[4 * h + 3]), s2), e, f);
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
            : "=r"(w[h])
            : "f"(a), "f"(d), "f"(e), "f"(f));
    }
    return make_uint2(w[0], w[1]);
}
// Code c is byte 3 of 16 (bits + 16 r - (8 b << 20)), for v > 0 brought up to code 1.
__device__ __forceinline__ uint2 encode_v_fast(const float (&v)[8], uint32_t b, const uint32_t (&word)[8]) {
    const float low = __uint_as_float((8u * b + 1u) << 20);
    const uint32_t off = b << 27;
    uint32_t u[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
        u[q] = __float_as_uint(fmaxf(v[q], low)) * 16u + (__byte_perm(word[q], 0u, 0x4104u) - off);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __byte_perm(__byte_perm(u[4 * h], u[4 * h + 1], 0x0073u), __byte_perm(u[4 * h + 2], u[4 * h + 3], 0x0073u),
                           0x5410u);
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 encode_m_any(const float (&m)[8], uint32_t b, int cnt) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t mag = q < cnt ? __float_as_uint(m[q]) & 0x7FFFFFFFu : 0u;
        const int32_t r = (int32_t)((mag + 0x7FFFFu + ((mag >> 20) & 1u)) >> 20) - (int32_t)(8u * b);
        const uint32_t c = finite_bits(mag) ? (uint32_t)min(max(r, 0), 127) : 127u;
        w[q >> 2] |= (c | (m[q] < 0.f ? 128u : 0u)) << (8 * (q & 3));
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint2 encode_v_any(const float (&v)[8], uint32_t b, const uint32_t (&word)[8], int cnt) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t mag = q < cnt ? __float_as_uint(v[q]) & 0x7FFFFFFFu : 0u;
        const int32_t r = (int32_t)((mag + ((word[q] & 0xFFFFu) << 4)) >> 20) - (int32_t)(8u * b);
        const uint32_t c = finite_bits(mag) ? (uint32_t)min(max(r, 1), 255) : 255u;
        w[q >> 2] |= (mag ? c : 0u) << (8 * (q & 3));
    }
    return make_uint2(w[0], w[1]);
}
// The base of a block of finite values with an element that is not (those
// leave the base alone).
__device__ __forceinline__ uint32_t finite_base(const float (&x)[8], uint32_t span, int cnt) {
    uint32_t mag[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) mag[q] = q < cnt ? __float_as_uint(x[q]) & 0x7FFFFFFFu : 0u;
    return block_base(mag, span);
}

// The step's numbers as pairs.
struct AdamPairs {
    unsigned long long scale, b1, b1c, b2, b2c, rsc2, eps, rate, keep;
};
// m, v, p of eight elements by one step.  PLAIN: v' is a normal number.
template <bool PLAIN>
__device__ __forceinline__ void step8(const AdamPairs &a, const float (&g)[8], float (&p)[8], float (&m)[8],
                                      float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
        const unsigned long long gs = mul2(pair_of(g[q], g[q + 1]), a.scale);
        // the last sums one by one: a packed sum of packed products was fused
        float m0, m1, n0, n1;
        split_pair(mul2(a.b1, pair_of(m[q], m[q + 1])), m0, m1);
        split_pair(mul2(a.b1c, gs), n0, n1);
        m[q] = __fadd_rn(m0, n0);
        m[q + 1] = __fadd_rn(m1, n1);
        split_pair(mul2(a.b2, pair_of(v[q], v[q + 1])), m0, m1);
        split_pair(mul2(a.b2c, mul2(gs, gs)), n0, n1);
        v[q] = __fadd_rn(m0, n0);
        v[q + 1] = __fadd_rn(m1, n1);
        const unsigned long long mm = pair_of(m[q], m[q + 1]);
        // The root of v' and the reciprocal, each within 2^-22: the update, some
        // thousandths of p, is within 2^-20 of itself.  v' may lie below the
        // normal numbers (the square of a gradient of 1e-19), where it still
        // decides the step if eps does not; a v' of 0 counts as the least number
        // above it, so that 0 / 0 is 0.
        float r0, r1, d0, d1;
        if (PLAIN) {
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(v[q]));
            asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(v[q + 1]));
        } else {
            asm("sqrt.approx.f32 %0, %1;" : "=f"(r0) : "f"(fmaxf(v[q], 0x1p-149f)));
            asm("sqrt.approx.f32 %0, %1;" : "=f"(r1) : "f"(fmaxf(v[q + 1], 0x1p-149f)));
        }
        split_pair(fma2(pair_of(r0, r1), a.rsc2, a.eps), d0, d1);
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d0));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d1));
        split_pair(fma2(a.rate, mul2(mm, pair_of(d0, d1)), mul2(pair_of(p[q], p[q + 1]), a.keep)), p[q], p[q + 1]);
    }
}
__device__ __forceinline__ void words8(const AdamArgs &a, uint32_t row, uint32_t quad, uint32_t (&word)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 w = token_block(a.seed, a.offset, row, quad + h);
        word[4 * h] = w.x;
        word[4 * h + 1] = w.y;
        word[4 * h + 2] = w.z;
        word[4 * h + 3] = w.w;
    }
}
// Eight parameters as they are stored: fp32, or bf16 by adding 16 random bits
// below the kept ones.  An infinity stays one; a NaN might pass through the
// sign, so a sum over the elements looks for one.
template <int PD>
__device__ __forceinline__ void store_params(void *base, int64_t i, int cnt, bool whole, const float (&p)[8],
                                             const uint32_t (&word)[8]) {
    if constexpr (PD == 0) {
        store8_f32(base, i, cnt, whole, p);
    } else {
        uint32_t w[4];
        float s0, s1;
        split_pair(add2(add2(pair_of(p[0], p[1]), pair_of(p[2], p[3])), add2(pair_of(p[4], p[5]), pair_of(p[6], p[7]))),
                   s0, s1);
        const float any = s0 + s1;
        if (any == any) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = __byte_perm(__float_as_uint(p[2 * q]) + (word[2 * q] >> 16),
                                   __float_as_uint(p[2 * q + 1]) + (word[2 * q + 1] >> 16), 0x7632u);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = bf16_stochastic(p[2 * q], word[2 * q]) | (bf16_stochastic(p[2 * q + 1], word[2 * q + 1]) << 16);
        }
        uint16_t *d = static_cast<uint16_t *>(base) + i;
        if (whole) {
            __stcs(reinterpret_cast<uint4 *>(d), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt) d[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        }
    }
}
// The 8-bit states of eight elements, in the fast forms; false where v' (and
// so a gradient) is not finite.
__device__ __forceinline__ bool encode_fast(const float (&m)[8], const float (&v)[8], const uint32_t (&word)[8],
                                            uint2 &cm, uint2 &cv, uint32_t &bm, uint32_t &bv) {
    float tm = 0.f;
    uint32_t tv = 0u;
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
        tm = fmaxf(fmaxf(tm, fabsf(m[q])), fabsf(m[q + 1]));
        tv = max(max(tv, __float_as_uint(v[q])), __float_as_uint(v[q + 1]));
    }
    tv = __reduce_max_sync(0xFFFFFFFFu, tv);
    const uint32_t em = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tm)) >> 23;
    if (!finite_bits(tv)) return false;
    bm = em > 14u ? em - 14u : 0u;
    bv = (tv >> 23) > 30u ? (tv >> 23) - 30u : 0u;
    cm = encode_m_fast(m, bm);
    cv = encode_v_fast(v, bv, word);
    if (not_e4m3(cm.x) || not_e4m3(cm.y)) cm = encode_m_any(m, bm, 8);
    return true;
}

template <int PD, int GD, int BITS, int N>
__global__ void __launch_bounds__(kAdThreads, BITS == 8 ? 7 : 1) adamw_kernel(const __grid_constant__ AdamTable<N> tab,
                                                           const __grid_constant__ AdamArgs a) {
    const float scale = a.scale ? *a.scale : 1.f;
    if (!(fabsf(scale) < INFINITY)) return;
    const int k = find_tensor(tab, blockIdx.x);
    const AdamTensor t = tab.t[k];
    const int64_t n = t.n;
    const bool vec = aligned16(t.param) && aligned16(t.grad) &&
                     (BITS == 32 ? aligned16(t.m) && aligned16(t.v) : aligned8(t.m) && aligned8(t.v));
    const int lane = threadIdx.x & 31;
    const uint32_t row = a.first + (uint32_t)k;
    const AdamPairs c = {pair_of(scale, scale),     pair_of(a.b1, a.b1),   pair_of(a.b1c, a.b1c),
                         pair_of(a.b2, a.b2),       pair_of(a.b2c, a.b2c), pair_of(a.rsc2, a.rsc2),
                         pair_of(a.eps, a.eps),     pair_of(-a.rate, -a.rate), pair_of(a.keep, a.keep)};
    // the warp's blocks of 256 elements
    int64_t wb = (int64_t)(blockIdx.x - tab.start[k]) * tab.iters * kAdIter + (threadIdx.x >> 5) * 256;
    int64_t end = wb + (int64_t)tab.iters * kAdIter;
    if (end > n) end = n;
    // Lane j holds the exponents of the warp's j-th block (at most 16), read
    // before the first and written after the last: a byte written beside
    // bytes that are still to be read made each read wait for the write.
    const int64_t my_block = (wb >> 8) + (int64_t)lane * (kAdIter / 256);
    const bool have = BITS == 8 && lane < tab.iters && my_block * 256 < n;
    uint32_t em_all = have ? t.me[my_block] : 0u, ev_all = have ? t.ve[my_block] : 0u;
    int turn = 0;
#pragma unroll 1
    for (; wb < end; wb += kAdIter, ++turn) {
        const int64_t i = wb + lane * kAdPer;
        const bool full = wb + 256 <= n, whole = vec && full;
        const int cnt = full ? 8 : (n - i >= 8 ? 8 : (n > i ? (int)(n - i) : 0));
        float g[8], p[8], m[8], v[8];
        uint32_t word[8] = {};
        Eight<GD> eg;
        Eight<PD> ep;
        eg.load(t.grad, i, cnt, whole);
        ep.load(t.param, i, cnt, whole);
        if constexpr (BITS == 32) {
            Eight<0> em, ev;
            em.load(t.m, i, cnt, whole);
            ev.load(t.v, i, cnt, whole);
            if constexpr (PD == 2) words8(a, row, (uint32_t)(i >> 2), word);
            eg.floats(g);
            ep.floats(p);
            em.floats(m);
            ev.floats(v);
            step8<false>(c, g, p, m, v);
            store_params<PD>(t.param, i, cnt, whole, p, word);
            store8_f32(t.m, i, cnt, whole, m);
            store8_f32(t.v, i, cnt, whole, v);
        } else {
            uint2 cm = load_codes(static_cast<const uint8_t *>(t.m), i, cnt, whole);
            uint2 cv = load_codes(static_cast<const uint8_t *>(t.v), i, cnt, whole);
            uint32_t bm = __shfl_sync(0xFFFFFFFFu, em_all, turn), bv = __shfl_sync(0xFFFFFFFFu, ev_all, turn);
            words8(a, row, (uint32_t)(i >> 2), word);  // under the loads
            eg.floats(g);
            ep.floats(p);
            if (!__any_sync(0xFFFFFFFFu, not_e4m3(cm.x) || not_e4m3(cm.y))) {
                decode_m_fast(cm, bm, m);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) m[q] = decode_m(((q < 4 ? cm.x : cm.y) >> (8 * (q & 3))) & 255u, 8u * bm);
            }
            // beta2 and the base keep v' above 0 (and normal) where v is
            bool done = false;
            if (full && bv >= 32u && a.b2 >= 0x1p-16f &&
                !__any_sync(0xFFFFFFFFu, zero_byte(cv.x) || zero_byte(cv.y))) {
                decode_v_fast(cv, bv, v);
                step8<true>(c, g, p, m, v);
                store_params<PD>(t.param, i, cnt, whole, p, word);  // p and its random bits are done with
                done = encode_fast(m, v, word, cm, cv, bm, bv);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = decode_v(((q < 4 ? cv.x : cv.y) >> (8 * (q & 3))) & 255u, 8u * bv);
                step8<false>(c, g, p, m, v);
                store_params<PD>(t.param, i, cnt, whole, p, word);
            }
            if (!done) {
                bm = finite_base(m, 14u, cnt);
                bv = finite_base(v, 30u, cnt);
                cm = encode_m_any(m, bm, cnt);
                cv = encode_v_any(v, bv, word, cnt);
            }
            store_codes(static_cast<uint8_t *>(t.m), i, cnt, whole, cm);
            store_codes(static_cast<uint8_t *>(t.v), i, cnt, whole, cv);
            if (lane == turn) {
                em_all = bm;
                ev_all = bv;
            }
        }
    }
    if (have) {
        t.me[my_block] = (uint8_t)em_all;
        t.ve[my_block] = (uint8_t)ev_all;
    }
}

// 8-bit states to bf16: the code's bits are the upper half of the float.
template <int N>
__global__ void __launch_bounds__(kAdThreads) adamw_values_kernel(const __grid_constant__ AdamTable<N> tab) {
    const int k = find_tensor(tab, blockIdx.x);
    const AdamTensor &t = tab.t[k];
    const int64_t n = t.n;
    uint16_t *om = static_cast<uint16_t *>(t.param), *ov = static_cast<uint16_t *>(const_cast<void *>(t.grad));
    const bool vec = aligned16(om) && aligned16(ov) && aligned8(t.m) && aligned8(t.v);
    const int64_t first = (int64_t)(blockIdx.x - tab.start[k]) * tab.iters * kAdIter;
#pragma unroll 1
    for (int it = 0; it < tab.iters; ++it) {
        const int64_t i = first + (int64_t)it * kAdIter + threadIdx.x * kAdPer;
        if (i >= n) return;
        const int cnt = n - i < 8 ? (int)(n - i) : 8;
        const uint2 cm = load_codes(static_cast<const uint8_t *>(t.m), i, cnt, vec && cnt == 8);
        const uint2 cv = load_codes(static_cast<const uint8_t *>(t.v), i, cnt, vec && cnt == 8);
        const uint32_t mb = 8u * t.me[i >> 8], vb = 8u * t.ve[i >> 8];
        uint32_t wm[4], wv[4];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t x = __float_as_uint(decode_m(((q < 4 ? cm.x : cm.y) >> (8 * (q & 3))) & 255u, mb)) >> 16;
            const uint32_t y = __float_as_uint(decode_v(((q < 4 ? cv.x : cv.y) >> (8 * (q & 3))) & 255u, vb)) >> 16;
            wm[q >> 1] = q & 1 ? wm[q >> 1] | (x << 16) : x;
            wv[q >> 1] = q & 1 ? wv[q >> 1] | (y << 16) : y;
        }
        if (vec && cnt == 8) {
            __stcs(reinterpret_cast<uint4 *>(om + i), make_uint4(wm[0], wm[1], wm[2], wm[3]));
            __stcs(reinterpret_cast<uint4 *>(ov + i), make_uint4(wv[0], wv[1], wv[2], wv[3]));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < cnt) {
                    om[i + q] = (uint16_t)(wm[q >> 1] >> (16 * (q & 1)));
                    ov[i + q] = (uint16_t)(wv[q >> 1] >> (16 * (q & 1)));
                }
        }
    }
}

template <int N>
const void *adam_kernel(int pd, int gd, int bits) {
#define TSA_ADAM(P, G, Z) \
    if (pd == P && gd == G && bits == Z) return reinterpret_cast<const void *>(&adamw_kernel<P, G, Z, N>)
    TSA_ADAM(0, 0, 32);
    TSA_ADAM(0, 1, 32);
    TSA_ADAM(0, 2, 32);
    TSA_ADAM(2, 0, 32);
    TSA_ADAM(2, 1, 32);
    TSA_ADAM(2, 2, 32);
    TSA_ADAM(0, 0, 8);
    TSA_ADAM(0, 1, 8);
    TSA_ADAM(0, 2, 8);
    TSA_ADAM(2, 0, 8);
    TSA_ADAM(2, 1, 8);
    TSA_ADAM(2, 2, 8);
#undef TSA_ADAM
    return nullptr;
}

// A chunk's length in steps of 1,024 elements: one while that leaves the GPU
// few chunks, so that small lists spread over every SM.  Large lists take up
// to 4 with fp32 states (100 million parameters: 401 us, 7.0 TB/s; 8 steps 6 us
// more), which end more evenly, and up to 16 with 8-bit ones (256 million with the
// values' call: 802 us; 32 steps 2 us more), where a warp keeps its blocks'
// exponents over a chunk.
int chunk_iters(int64_t total, int most) {
    const int64_t steps = (total + kAdIter - 1) / kAdIter;
    int n = 1;
    while (n < most && steps >= 152 * 8 * 2 * n) n *= 2;
    return n;
}

template <int N>
int launch_table(const AdamTensor *tensors, int64_t count, const void *fn, const AdamArgs *args, int iters,
                 cudaStream_t st) {
    AdamTable<N> tab;
    const int64_t per = (int64_t)iters * kAdIter;
    int64_t i = 0;
    while (i < count) {
        // as many tensors as the table and a grid hold; one tensor's chunks fit a grid
        tab.count = 0;
        tab.iters = iters;
        tab.start[0] = 0;
        AdamArgs a = args ? *args : AdamArgs{};
        a.first = (uint32_t)i;
        while (i < count && tab.count < N) {
            const int64_t chunks = (tensors[i].n + per - 1) / per;
            if (tab.count > 0 && (int64_t)tab.start[tab.count] + chunks > 0x7FFFFFFFll) break;
            tab.t[tab.count] = tensors[i];
            tab.start[tab.count + 1] = tab.start[tab.count] + (uint32_t)chunks;
            ++tab.count;
            ++i;
        }
        const uint32_t grid = tab.start[tab.count];
        if (grid == 0) continue;
        void *params[] = {&tab, &a};
        if (cudaLaunchKernel(fn, dim3(grid), dim3(kAdThreads), params, 0, st) != cudaSuccess) return -1;
    }
    return 0;
}

int64_t total_of(const AdamTensor *tensors, int64_t count) {
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) n += tensors[i].n;
    return n;
}

}  // namespace

int adamw_launch(const AdamTensor *tensors, int64_t count, int param_dtype, int grad_dtype, int bits,
                 const AdamArgs &args, cudaStream_t st) {
    const int iters = chunk_iters(total_of(tensors, count), bits == 8 ? 16 : 4);
    if (count <= kAdFew)
        return launch_table<kAdFew>(tensors, count, adam_kernel<kAdFew>(param_dtype, grad_dtype, bits), &args, iters,
                                    st);
    return launch_table<kAdMany>(tensors, count, adam_kernel<kAdMany>(param_dtype, grad_dtype, bits), &args, iters,
                                 st);
}

int adamw_values_launch(const AdamTensor *tensors, int64_t count, cudaStream_t st) {
    const int iters = chunk_iters(total_of(tensors, count), 4);
    if (count <= kAdFew)
        return launch_table<kAdFew>(tensors, count, reinterpret_cast<const void *>(&adamw_values_kernel<kAdFew>),
                                    nullptr, iters, st);
    return launch_table<kAdMany>(tensors, count, reinterpret_cast<const void *>(&adamw_values_kernel<kAdMany>),
                                 nullptr, iters, st);
}

}  // namespace tsa
