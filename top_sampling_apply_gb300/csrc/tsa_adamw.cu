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

constexpr int kAdThreads = 256;
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

template <int DT>
__device__ __forceinline__ float load1(const void *base, int64_t i) {
    if constexpr (DT == 0) return static_cast<const float *>(base)[i];
    if constexpr (DT == 1) return __half2float(static_cast<const __half *>(base)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[i]);
}
// Eight consecutive elements (k < cnt valid; the rest 0), as floats.
template <int DT>
__device__ __forceinline__ void load8(const void *base, int64_t i, int cnt, bool vec, float (&x)[8]) {
    using E = Elem<DT>;
    if (vec && cnt == 8) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + (size_t)i * E::SIZE);
        E::unpack(__ldcs(p), x);
        if constexpr (DT == 0) {
            const uint4 q = __ldcs(p + 1);
            x[4] = __uint_as_float(q.x);
            x[5] = __uint_as_float(q.y);
            x[6] = __uint_as_float(q.z);
            x[7] = __uint_as_float(q.w);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < cnt ? load1<DT>(base, i + k) : 0.f;
}
__device__ __forceinline__ void store8_f32(void *base, int64_t i, int cnt, bool vec, const float (&x)[8]) {
    float *p = static_cast<float *>(base) + i;
    if (vec && cnt == 8) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < cnt) p[k] = x[k];
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *base, int64_t i, int cnt, bool vec) {
    if (vec && cnt == 8) return __ldcs(reinterpret_cast<const uint2 *>(base + i));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < cnt) w[k >> 2] |= (uint32_t)base[i + k] << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t *base, int64_t i, int cnt, bool vec, uint2 c) {
    if (vec && cnt == 8) {
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

template <int PD, int GD, int BITS, int N>
__global__ void __launch_bounds__(kAdThreads) adamw_kernel(const __grid_constant__ AdamTable<N> tab,
                                                           const __grid_constant__ AdamArgs a) {
    const float scale = a.scale ? *a.scale : 1.f;
    if (!(fabsf(scale) < INFINITY)) return;
    const int k = find_tensor(tab, blockIdx.x);
    const AdamTensor &t = tab.t[k];
    const int64_t n = t.n;
    const bool vec = aligned16(t.param) && aligned16(t.grad) &&
                     (BITS == 32 ? aligned16(t.m) && aligned16(t.v) : aligned8(t.m) && aligned8(t.v));
    const int64_t first = (int64_t)(blockIdx.x - tab.start[k]) * tab.iters * kAdIter;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int it = 0; it < tab.iters; ++it) {
        // the warp's 256 elements; whole warps leave together
        const int64_t wb = first + (int64_t)it * kAdIter + (threadIdx.x >> 5) * 256;
        if (wb >= n) return;
        const int64_t i = wb + lane * kAdPer;
        const int cnt = i >= n ? 0 : (n - i < 8 ? (int)(n - i) : 8);
        float g[8], p[8], m[8], v[8];
        load8<GD>(t.grad, i, cnt, vec, g);
        load8<PD>(t.param, i, cnt, vec, p);
        if constexpr (BITS == 32) {
            load8<0>(t.m, i, cnt, vec, m);
            load8<0>(t.v, i, cnt, vec, v);
        } else {
            const uint2 cm = load_codes(static_cast<const uint8_t *>(t.m), i, cnt, vec);
            const uint2 cv = load_codes(static_cast<const uint8_t *>(t.v), i, cnt, vec);
            const uint32_t mb = 8u * t.me[wb >> 8], vb = 8u * t.ve[wb >> 8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                m[q] = decode_m(((q < 4 ? cm.x : cm.y) >> (8 * (q & 3))) & 255u, mb);
                v[q] = decode_v(((q < 4 ? cv.x : cv.y) >> (8 * (q & 3))) & 255u, vb);
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float gs = __fmul_rn(g[q], scale);
            m[q] = __fadd_rn(__fmul_rn(a.b1, m[q]), __fmul_rn(a.b1c, gs));
            v[q] = __fadd_rn(__fmul_rn(a.b2, v[q]), __fmul_rn(a.b2c, __fmul_rn(gs, gs)));
            float root;
            asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[q]));
            // within 2^-21 of the quotient, times an update of some thousandths of p
            const float upd = __fdividef(m[q], fmaf(root, a.rsc2, a.eps));
            p[q] = fmaf(-a.rate, upd, p[q] * a.keep);
        }
        uint32_t word[8];
        if constexpr (BITS == 8 || PD == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 w = token_block(a.seed, a.offset, a.first + (uint32_t)k, (uint32_t)(i >> 2) + h);
                word[4 * h] = w.x;
                word[4 * h + 1] = w.y;
                word[4 * h + 2] = w.z;
                word[4 * h + 3] = w.w;
            }
        }
        if constexpr (PD == 0) {
            store8_f32(t.param, i, cnt, vec, p);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = bf16_stochastic(p[2 * q], word[2 * q]) | (bf16_stochastic(p[2 * q + 1], word[2 * q + 1]) << 16);
            uint16_t *d = static_cast<uint16_t *>(t.param) + i;
            if (vec && cnt == 8) {
                __stcs(reinterpret_cast<uint4 *>(d), make_uint4(w[0], w[1], w[2], w[3]));
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < cnt) d[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
            }
        }
        if constexpr (BITS == 32) {
            store8_f32(t.m, i, cnt, vec, m);
            store8_f32(t.v, i, cnt, vec, v);
        } else {
            uint32_t mag[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) mag[q] = q < cnt ? __float_as_uint(m[q]) & 0x7FFFFFFFu : 0u;
            const uint32_t bm = block_base(mag, 14u);
            uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int32_t r = (int32_t)((mag[q] + 0x7FFFFu + ((mag[q] >> 20) & 1u)) >> 20) - (int32_t)(8u * bm);
                const uint32_t c = finite_bits(mag[q]) ? (uint32_t)min(max(r, 0), 127) : 127u;
                cm[q >> 2] |= (c | (m[q] < 0.f ? 128u : 0u)) << (8 * (q & 3));
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) mag[q] = q < cnt ? __float_as_uint(v[q]) & 0x7FFFFFFFu : 0u;
            const uint32_t bv = block_base(mag, 30u);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int32_t r = (int32_t)((mag[q] + ((word[q] & 0xFFFFu) << 4)) >> 20) - (int32_t)(8u * bv);
                uint32_t c = finite_bits(mag[q]) ? (uint32_t)min(max(r, 1), 255) : 255u;
                cv[q >> 2] |= (mag[q] ? c : 0u) << (8 * (q & 3));
            }
            store_codes(static_cast<uint8_t *>(t.m), i, cnt, vec, make_uint2(cm[0], cm[1]));
            store_codes(static_cast<uint8_t *>(t.v), i, cnt, vec, make_uint2(cv[0], cv[1]));
            if (lane == 0) {
                t.me[wb >> 8] = (uint8_t)bm;
                t.ve[wb >> 8] = (uint8_t)bv;
            }
        }
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
        const uint2 cm = load_codes(static_cast<const uint8_t *>(t.m), i, cnt, vec);
        const uint2 cv = load_codes(static_cast<const uint8_t *>(t.v), i, cnt, vec);
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

// A chunk's length: 2,048 elements while that leaves the GPU few chunks, so
// that small lists spread over every SM, and up to 8,192 for large ones, which
// then pay the tensor search once in four steps.
int chunk_iters(int64_t total) {
    const int64_t steps = (total + kAdIter - 1) / kAdIter;
    return steps >= 152 * 8 * 4 ? 4 : (steps >= 152 * 8 * 2 ? 2 : 1);
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
    const int iters = chunk_iters(total_of(tensors, count));
    if (count <= kAdFew)
        return launch_table<kAdFew>(tensors, count, adam_kernel<kAdFew>(param_dtype, grad_dtype, bits), &args, iters,
                                    st);
    return launch_table<kAdMany>(tensors, count, adam_kernel<kAdMany>(param_dtype, grad_dtype, bits), &args, iters,
                                 st);
}

int adamw_values_launch(const AdamTensor *tensors, int64_t count, cudaStream_t st) {
    const int iters = chunk_iters(total_of(tensors, count));
    if (count <= kAdFew)
        return launch_table<kAdFew>(tensors, count, reinterpret_cast<const void *>(&adamw_values_kernel<kAdFew>),
                                    nullptr, iters, st);
    return launch_table<kAdMany>(tensors, count, reinterpret_cast<const void *>(&adamw_values_kernel<kAdMany>),
                                 nullptr, iters, st);
}

}  // namespace tsa
