// The root-mean-square norm that makes the head's hidden rows, with the
// residual's addition and rows in 8 bits, and its backward pass:
//     s = round(x + r),  q = (mean s^2 + eps)^(-1/2),  y = s q w,
//     scale = max |y| / 127,  code = rint(y / scale);
//     f = w dy,  h = s q:  dx = q (f - h mean(f h)) + gr,  dw = sum over rows of dy h.
// Every kernel reads its rows once and holds them in registers between the
// row's sum and the results; what bounds it is HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tsa_device.cuh"
#include "tsa_host.h"

namespace tsa {

namespace {

constexpr int kNormElems = 16;  // a thread's elements of a long row
// Most threads a row: 512 keep 128 registers each, enough to hold the next row
// too; rows of more than 8,192 elements take up to 1,024 threads.
constexpr int norm_threads(bool big) { return big ? 1024 : 512; }
static_assert(kNormElems * norm_threads(true) == kNormMaxH, "the longest row fits");

__device__ unsigned int g_norm_status;

// W elements of a row at `i`: a 16-byte vector, or single elements where a
// row does not start on 16 bytes.  Plain loads: an output may be an input's
// own memory, and every element is read by the thread that writes it.
template <int DT, int W>
struct Part {
    // What a load brings, before it is unpacked: 16 bytes, or an element.
    using Raw = std::conditional_t<(W > 1), uint4, std::conditional_t<DT == 0, uint32_t, uint16_t>>;
    static __device__ __forceinline__ Raw fetch(const void *p, int64_t i) {
        return *reinterpret_cast<const Raw *>(static_cast<const uint8_t *>(p) + i * Elem<DT>::SIZE);
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float *x) {
        if constexpr (W > 1)
            Elem<DT>::unpack(r, x);
        else if constexpr (DT == 0)
            x[0] = __uint_as_float(r);
        else if constexpr (DT == 1)
            x[0] = __half2float(__ushort_as_half(r));
        else
            x[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ void load(const void *p, int64_t i, float *x) { unpack(fetch(p, i), x); }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float *x) {
        if constexpr (W > 1) {
            uint4 v;
            if constexpr (DT == 0) {
                v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            } else {
                uint32_t *u = &v.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (DT == 1) {
                        const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                        u[j] = *reinterpret_cast<const uint32_t *>(&h);
                    } else {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                        u[j] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p) + i * Elem<DT>::SIZE) = v;
        } else if constexpr (DT == 0) {
            static_cast<float *>(p)[i] = x[0];
        } else if constexpr (DT == 1) {
            static_cast<__half *>(p)[i] = __float2half_rn(x[0]);
        } else {
            static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x[0]);
        }
    }
    // x rounded to the type, as the row then holds it
    static __device__ __forceinline__ float held(float x) {
        if constexpr (DT == 0) return x;
        if constexpr (DT == 1) return __half2float(__float2half_rn(x));
        return __bfloat162float(__float2bfloat16_rn(x));
    }
    // W elements of a weight of the rows' type or of fp32
    static __device__ __forceinline__ void weight(const void *p, bool f32, int64_t i, float *x) {
        if (DT == 0 || !f32) {
            load(p, i, x);
        } else {
            const float *w = static_cast<const float *>(p) + i;
            if constexpr (W > 1) {
                const float4 a = *reinterpret_cast<const float4 *>(w), b = *reinterpret_cast<const float4 *>(w + 4);
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
                x[4 % W] = b.x, x[5 % W] = b.y, x[6 % W] = b.z, x[7 % W] = b.w;
            } else {
                x[0] = w[0];
            }
        }
    }
    static __device__ __forceinline__ void store_codes(int8_t *p, int64_t i, const float *x) {
        if constexpr (W > 1) {
            uint32_t u[W / 4];
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
                u[j] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) u[j] |= ((uint32_t)__float2int_rn(x[4 * j + k]) & 0xFFu) << (8 * k);
            }
            if constexpr (W == 8)
                *reinterpret_cast<uint2 *>(p + i) = make_uint2(u[0], u[1]);
            else
                *reinterpret_cast<uint32_t *>(p + i) = u[0];
        } else {
            p[i] = (int8_t)__float2int_rn(x[0]);
        }
    }
};

// A row's sum over the blockDim.x threads that share it (a multiple of 32),
// the same in all of them.  `turn` alternates between two halves of the
// scratch, so that one barrier a sum is enough.
__device__ __forceinline__ float row_sum(float v, float (*sh)[32], int turn) {
    v = warp_sum_f32(v);
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5, first = threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) sh[turn][first + (threadIdx.x >> 5)] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += sh[turn][first + i];
    return s;
}
// The row's largest bit pattern: of absolute values the largest, and a NaN
// above them.
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (*sh)[32], int turn) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5, first = threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) sh[turn][first + (threadIdx.x >> 5)] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int i = 0; i < warps; ++i) s = max(s, sh[turn][first + i]);
    return s;
}

// A row's scale from its largest absolute value, and what a value is rounded to
// its code from.  A largest value under 2^-100 would overflow the reciprocal:
// such rows are brought up by 2^64 first.  A row that is not finite has codes 0
// under a scale of NaN.
struct Codes {
    float scale, up, f;
    bool finite;
    __device__ __forceinline__ explicit Codes(float most) {
        finite = most < INFINITY;
        up = most < 0x1p-100f ? 0x1p64f : 1.f;
        f = finite && most > 0.f ? 127.f / (most * up) : 0.f;
        scale = finite ? most / 127.f : __int_as_float(0x7FC00000);
    }
    __device__ __forceinline__ float of(float x) const { return finite ? x * up * f : 0.f; }
};

// NORM = false: the rows themselves in 8 bits.
template <int DT, int W, int E, bool NORM, bool Q>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a) {
    using P = Part<DT, W>;
    constexpr int NV = E / W;
    __shared__ float sh_sum[2][32];
    __shared__ uint32_t sh_max[2][32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = row < a.N;
    const int step = blockDim.x * W, c0 = threadIdx.x * W;
    const int H = (int)a.H;
    float v[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = 0.f;
        if (in && c0 + i * step < H) P::load(a.x, row * a.xs + c0 + i * step, v[i]);
    }
    if constexpr (NORM) {
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (in && c < H) {
                    float r[W];
                    P::load(a.r, row * a.rs + c, r);
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] = P::held(v[i][j] + r[j]);
                    if (a.res) P::store(a.res, row * a.ress + c, v[i]);
                }
            }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) s = fmaf(v[i][j], v[i][j], s);
        }
        s = row_sum(s, sh_sum, 0);
        const float rstd = 1.f / sqrtf(s / (float)H + a.eps);
        if (in && threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
                float w[W];
                P::weight(a.w, a.w_f32, c, w);
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = v[i][j] * rstd * w[j];
                if (!Q && in) P::store(a.out, row * a.os + c, v[i]);
            }
        }
    }
    if constexpr (Q) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) top = max(top, __float_as_uint(fabsf(v[i][j])));
        }
        const Codes k(__uint_as_float(row_max(top, sh_max, 0)));
        if (in && threadIdx.x == 0) a.scale[row] = k.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = k.of(v[i][j]);
                P::store_codes(static_cast<int8_t *>(a.out), row * a.os + c, v[i]);
            }
        }
    }
}

// Rows go round the CTAs, so that a thread keeps its columns' part of dw in
// registers; a part a CTA (and row of threads) goes to the workspace.  What bounds
// it is a row's latency: 1,216 x 1,001 bf16 take 9.4 us, four turns of 304 CTAs and
// the launch that adds the parts.  BIG, for rows of more than 8,192 elements, is
// for those that the ring has no two stages for: the compiler spills 172 to 304
// bytes a thread of rows of vectors and 756 to 1,028 of rows of single elements
// (4,096 x 12,344 f32 with a residual's gradient 246 us, x 12,345 642).
template <int DT, int W, int E, bool BIG>
__global__ void __launch_bounds__(norm_threads(BIG)) norm_back_kernel(NormBackArgs a) {
    // whether the registers hold the next row too, and the weights
    constexpr bool AHEAD = !BIG && (W > 1 || E == 8), KEEP = E == 8;
    using P = Part<DT, W>;
    constexpr int NV = E / W;
    __shared__ float sh[2][32];
    const int step = blockDim.x * W, c0 = threadIdx.x * W;
    const int H = (int)a.H;
    float acc[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[i][j] = 0.f;
    typename P::Raw rx[NV], rg[NV], rr[NV];
    float next = 0.f;
    const auto fetch = [&](int64_t row) {
        if (row >= a.N) return;
        next = a.rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
                rx[i] = P::fetch(a.x, row * a.xs + c);
                rg[i] = P::fetch(a.g, row * a.gs + c);
                if (a.gr) rr[i] = P::fetch(a.gr, row * a.grs + c);
            }
        }
    };
    int turn = 0;
    const int64_t stride = (int64_t)gridDim.x * blockDim.y;
    float kept[KEEP ? NV : 1][W];
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c0 + i * step < H) P::weight(a.w, a.w_f32, c0 + i * step, kept[KEEP ? i : 0]);
    }
    if (AHEAD) fetch((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.N; r0 += stride, turn ^= 1) {
        const int64_t row = r0 + threadIdx.y;
        const bool in = row < a.N;
        if (!AHEAD) fetch(row);
        const float rstd = next;
        float h[NV][W], f[NV][W], add[NV][W], dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            P::unpack(rx[i], h[i]);
            P::unpack(rg[i], f[i]);
            P::unpack(rr[i], add[i]);
        }
        if (AHEAD) fetch(row + stride);  // under this row's sums
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
                float w[W];
                if (!KEEP) P::weight(a.w, a.w_f32, c, w);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    h[i][j] *= rstd;
                    acc[i][j] = fmaf(f[i][j], h[i][j], acc[i][j]);
                    f[i][j] *= KEEP ? kept[KEEP ? i : 0][j] : w[j];
                    dot = fmaf(f[i][j], h[i][j], dot);
                }
            }
        }
        const float mean = row_sum(dot, sh, turn) / (float)H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    f[i][j] = fmaf(rstd, fmaf(-h[i][j], mean, f[i][j]), a.gr ? add[i][j] : 0.f);
                P::store(a.dx, row * a.dxs + c, f[i]);
            }
        }
    }
    const int64_t part = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c0 + i * step + j < H) a.part[part * a.H + c0 + i * step + j] = acc[i][j];
}

// Many long rows: a persistent CTA goes through its rows with the next ones on
// their way into shared memory by bulk copies, and its columns' weights in
// registers.  A stage is free once every thread is past the barrier of the row
// after it, so that copies run STAGES - 1 rows ahead.  16,384 x 5,120 bf16 with a
// residual: forward 108 us, 6.2 TB/s (124 with a CTA a row), backward 116 us, 5.8
// TB/s (149 with the next row in registers, 214 without it).
//
// Rows that start anywhere (ODD: odd lengths, strides or bases, alike in every tensor) are taken 16 bytes at a time
// all the same.  The grid is a multiple of 152 = 8 * 19 CTAs, so that each of a CTA's rows starts as far into 16
// bytes as its first one does: its columns are shifted by that once, weights and the parts of dw with them, and only a
// row's first and last 16 bytes are cut.  By single elements from the ring 16,384 x 4,881 takes 255 us forward and 488
// backward, shifted 126 and 183.
template <int SIZE, bool ODD>  // bytes of an element; whether rows start anywhere
struct RowRing {
    uint8_t *mem;
    uint64_t *full;
    int *dead;  // a wait ran out: the CTA finishes without waiting
    int stages, rows;
    uint32_t bytes, pitch;  // of a row, and of its place
    int64_t n, first, step;  // rows in all, this CTA's first, and from one to the next
    // The i-th row of this CTA: `src` gives the rows of each input.
    template <class F>
    __device__ __forceinline__ void issue(int i, F src) const {
        const int64_t row = first + i * step;
        if (threadIdx.x != 0 || row >= n) return;
        const int s = i % stages;
        if constexpr (!ODD) {
            mbar_arrive_expect_tx(&full[s], bytes * rows);
            for (int j = 0; j < rows; ++j) bulk_g2s(mem + (size_t)(s * rows + j) * bytes, src(j, row), bytes, &full[s]);
            return;
        }
        uint32_t sum = 0;
        for (int j = 0; j < rows; ++j) {
            const uint8_t *p = src(j, row);
            const Span at = span(p, row);
            sum += at.hi - at.lo;
            uint8_t *to = mem + (size_t)(s * rows + j) * pitch;
            for (uint32_t b = at.skip; b < at.lo; b += SIZE) put(to + b, p + (b - at.skip));
            for (uint32_t b = at.hi; b < at.end; b += SIZE) put(to + b, p + (b - at.skip));
        }
        mbar_arrive_expect_tx(&full[s], sum);  // the waiting threads see the writes above, too
        for (int j = 0; j < rows; ++j) {
            const uint8_t *p = src(j, row);
            const Span at = span(p, row);
            bulk_g2s(mem + (size_t)(s * rows + j) * pitch + at.lo, p - at.skip + at.lo, at.hi - at.lo, &full[s]);
        }
    }
    // A row in its place, from `skip` to `end`, and the whole 16 bytes that are copied.  Those at the first row's start
    // and at the last one's end may hold memory that is not the tensor's: that row's part of them goes by elements.
    struct Span {
        uint32_t skip, end, lo, hi;
    };
    __device__ __forceinline__ Span span(const uint8_t *p, int64_t row) const {
        const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15), end = skip + bytes;
        return Span{skip, end, skip > 0 && row == 0 ? 16u : 0u, row == n - 1 ? end & ~15u : (end + 15) & ~15u};
    }
    __device__ __forceinline__ void put(uint8_t *to, const uint8_t *from) const {
        if constexpr (SIZE == 4)
            *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
        else
            *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
    }
    __device__ __forceinline__ const uint8_t *wait(int i) const {
        const int s = i % stages;
        if (*(volatile int *)dead == 0 && !mbar_wait_bounded(&full[s], (i / stages) & 1u, &g_norm_status)) *(volatile int *)dead = 1;
        return mem + (size_t)s * rows * pitch;
    }
    // No copy may land after the CTA is gone (they all have, unless a wait ran out).
    __device__ __forceinline__ void finish(int done) const {
        if (threadIdx.x != 0 || *(volatile int *)dead == 0) return;
        for (int i = done < stages ? 0 : done - stages; first + i * step < n && i < done + stages; ++i)
            mbar_wait_bounded(&full[i % stages], (i / stages) & 1u, &g_norm_status);
    }
};
// Bytes of a row's place: ODD rows start up to 15 bytes into it.
__host__ __device__ constexpr uint32_t ring_pitch(uint32_t bytes, bool odd) {
    return odd ? (bytes + 15) / 16 * 16 + 16 : bytes;
}
template <int SIZE, bool ODD>
__device__ __forceinline__ RowRing<SIZE, ODD> make_ring(uint8_t *raw, uint64_t *full, int *dead, int stages, int rows, int H,
                                                        int64_t n) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
        *dead = 0;
        mbar_init_fence();
    }
    __syncthreads();
    const uint32_t bytes = (uint32_t)(H * SIZE);
    return RowRing<SIZE, ODD>{raw, full, dead, stages, rows, bytes, ring_pitch(bytes, ODD), n, blockIdx.x, gridDim.x};
}
constexpr int kRingStages = 4;
// Threads and CTAs an SM that the registers are counted for: up to 384 with 80
// registers a thread, two CTAs and more; 512 with 128, which the backward pass
// needs (with 64 it spills: 8,192 x 8,192 139 us instead of 95); 1,024 with 64.
constexpr int ring_threads(int c) { return c == 0 ? 384 : c == 1 ? 512 : 1024; }

// 16 bytes of a row from column c on, of which the first may be before the row and the last behind it: what is not the
// row's reads as 0 and is not written.
template <int DT, bool ODD>
struct Cut {
    static constexpr int W = Elem<DT>::AE;
    using P = Part<DT, W>;
    using One = Part<DT, 1>;
    static __device__ __forceinline__ bool whole(int c, int H) { return !ODD || (c >= 0 && c + W <= H); }
    static __device__ __forceinline__ void load(const uint8_t *place, int shift, int c, int H, float *x) {
        P::load(place, c + shift, x);
        if (whole(c, H)) return;
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c + j < 0 || c + j >= H) x[j] = 0.f;
    }
    static __device__ __forceinline__ void weight(const void *w, bool f32, int c, int H, float *x) {
        if constexpr (!ODD) {
            P::weight(w, f32, c, x);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                x[j] = 0.f;
                if (c + j >= 0 && c + j < H) One::weight(w, f32, c + j, x + j);
            }
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t row, int c, int H, const float *x) {
        if (whole(c, H)) {
            P::store(p, row + c, x);
            return;
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c + j >= 0 && c + j < H) One::store(p, row + c + j, x + j);
    }
    static __device__ __forceinline__ void store_codes(int8_t *p, int64_t row, int c, int H, const float *x) {
        if (whole(c, H)) {
            P::store_codes(p, row + c, x);
            return;
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c + j >= 0 && c + j < H) One::store_codes(p, row + c + j, x + j);
    }
};

template <int DT, bool ODD, bool Q, int C>
__global__ void __launch_bounds__(ring_threads(C), C == 0 ? 2 : 1) norm_ring_kernel(NormArgs a, int stages) {
    constexpr int W = Elem<DT>::AE, NV = kNormElems / W;
    using P = Part<DT, W>;
    using R = Cut<DT, ODD>;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ uint64_t full[kRingStages];
    __shared__ int dead;
    __shared__ float sh_sum[2][32];
    __shared__ uint32_t sh_max[2][32];
    const int H = (int)a.H, step = blockDim.x * W;
    const auto ring = make_ring<Elem<DT>::SIZE, ODD>(raw, full, &dead, stages, a.r ? 2 : 1, H, a.N);
    const auto src = [&](int j, int64_t row) {
        return static_cast<const uint8_t *>(j == 0 ? a.x : a.r) + row * (j == 0 ? a.xs : a.rs) * Elem<DT>::SIZE;
    };
    for (int i = 0; i < stages - 1; ++i) ring.issue(i, src);
    const int shift = ODD ? (int)((reinterpret_cast<uintptr_t>(src(0, ring.first)) & 15) / Elem<DT>::SIZE) : 0;
    const int c0 = threadIdx.x * W - shift;
    float w[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (c0 + i * step < H) R::weight(a.w, a.w_f32, c0 + i * step, H, w[i]);
    int it = 0;
    for (int64_t row = ring.first; row < a.N; row += ring.step, ++it) {
        const uint8_t *in = ring.wait(it);
        float v[NV][W], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
                R::load(in, shift, c, H, v[i]);
                if (a.r) {
                    float r[W];
                    R::load(in + ring.pitch, shift, c, H, r);
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] = P::held(v[i][j] + r[j]);
                    if (a.res) R::store(a.res, row * a.ress, c, H, v[i]);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) s = fmaf(v[i][j], v[i][j], s);
            }
        }
        s = row_sum(s, sh_sum, it & 1);
        ring.issue(it + stages - 1, src);
        const float rstd = 1.f / sqrtf(s / (float)H + a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    v[i][j] = v[i][j] * rstd * w[i][j];
                    top = max(top, __float_as_uint(fabsf(v[i][j])));
                }
                if (!Q) R::store(a.out, row * a.os, c, H, v[i]);
            }
        }
        if constexpr (Q) {
            const Codes k(__uint_as_float(row_max(top, sh_max, it & 1)));
            if (threadIdx.x == 0) a.scale[row] = k.scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
                if (c < H) {
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] = k.of(v[i][j]);
                    R::store_codes(static_cast<int8_t *>(a.out), row * a.os, c, H, v[i]);
                }
            }
        }
    }
    ring.finish(it);
}

template <int DT, bool ODD, int C>
__global__ void __launch_bounds__(ring_threads(C), C == 0 ? 2 : 1) norm_back_ring_kernel(NormBackArgs a, int stages) {
    constexpr int W = Elem<DT>::AE, NV = kNormElems / W;
    using R = Cut<DT, ODD>;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ uint64_t full[kRingStages];
    __shared__ int dead;
    __shared__ float sh[2][32];
    const int H = (int)a.H, step = blockDim.x * W;
    const auto ring = make_ring<Elem<DT>::SIZE, ODD>(raw, full, &dead, stages, a.gr ? 3 : 2, H, a.N);
    const auto src = [&](int j, int64_t row) {
        const void *p = j == 0 ? a.x : j == 1 ? a.g : a.gr;
        return static_cast<const uint8_t *>(p) + row * (j == 0 ? a.xs : j == 1 ? a.gs : a.grs) * Elem<DT>::SIZE;
    };
    for (int i = 0; i < stages - 1; ++i) ring.issue(i, src);
    const int shift = ODD ? (int)((reinterpret_cast<uintptr_t>(src(0, ring.first)) & 15) / Elem<DT>::SIZE) : 0;
    const int c0 = threadIdx.x * W - shift;
    float w[NV][W], acc[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) acc[i][j] = 0.f;
        if (c0 + i * step < H) R::weight(a.w, a.w_f32, c0 + i * step, H, w[i]);
    }
    int it = 0;
    for (int64_t row = ring.first; row < a.N; row += ring.step, ++it) {
        const float rstd = a.rstd[row];
        const uint8_t *in = ring.wait(it);
        float h[NV][W], f[NV][W], dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
                R::load(in, shift, c, H, h[i]);
                R::load(in + ring.pitch, shift, c, H, f[i]);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    h[i][j] *= rstd;
                    acc[i][j] = fmaf(f[i][j], h[i][j], acc[i][j]);
                    f[i][j] *= w[i][j];
                    dot = fmaf(f[i][j], h[i][j], dot);
                }
            }
        }
        const float mean = row_sum(dot, sh, it & 1) / (float)H;
        // every thread is past the row before, whose stage the next copy takes
        ring.issue(it + stages - 1, src);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < H) {
                float add[W];
#pragma unroll
                for (int j = 0; j < W; ++j) add[j] = 0.f;
                if (a.gr) R::load(in + 2 * ring.pitch, shift, c, H, add);
#pragma unroll
                for (int j = 0; j < W; ++j) f[i][j] = fmaf(rstd, fmaf(-h[i][j], mean, f[i][j]), add[j]);
                R::store(a.dx, row * a.dxs, c, H, f[i]);
            }
        }
    }
    ring.finish(it);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (c0 + i * step + j >= 0 && c0 + i * step + j < H) a.part[blockIdx.x * a.H + c0 + i * step + j] = acc[i][j];
}

// dw: 32 columns a CTA, the parts over 32 rows of threads, then a tree.
template <int DT>
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float *part, int64_t parts, int64_t H, void *dw) {
    __shared__ float sh[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < H)
        for (int64_t p = threadIdx.y; p < parts; p += 32) s += part[p * H + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = warp_sum_f32(sh[threadIdx.x][threadIdx.y]);  // column threadIdx.y
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < H) Part<DT, 1>::store(dw, col, &s);
}

// Threads and rows of a CTA: H / E threads a row, whole warps, at least 128
// threads a CTA.
dim3 norm_block(int64_t H, int E) {
    const int t = (int)(((H + E - 1) / E + 31) / 32 * 32);
    return dim3(t, t >= 128 ? 1 : 128 / t);
}
// Elements a thread: few for short rows, so that enough loads are under way, and
// for rows of single elements, of which the registers hold no more than 8 three times.
int norm_elems(int64_t H, bool vec) { return H <= (vec ? 2048 : 4096) ? 8 : kNormElems; }

// Whether many long rows go through shared memory, and how.  Fewer than four
// rows an SM leave next to nothing to fetch ahead (bf16 with a residual, ring and
// registers: 608 x 5,120 7.4 and 6.8 us, 1,216 x 5,120 11.8 and 12.1, 1,216 x 8,192
// 15.8 and 20.5), and rows of up to 2,048 elements take small CTAs of which many fit.
struct RingPlan {
    int stages, ctas, cls, threads;  // stages 0: no ring
    size_t smem;
};
constexpr int kRingCtas = 8, kRingBackRows = 2;
// Threads of a row of H elements, of which `odd` ones may start up to 15 bytes into their first 16.
int ring_block(int64_t H, int es, bool odd) { return (int)norm_block(H + (odd ? 16 / es - 1 : 0), kNormElems).x; }
// CTAs an SM that 80 registers a thread leave, and that have `each` rows
int64_t ring_most(int64_t N, int threads, int each) {
    const int64_t regs = threads > ring_threads(0) ? 1 : 65536 / (80 * threads), rows = N / 152 / each;
    const int64_t most = regs < rows ? regs : rows;
    return most < kRingCtas ? most : kRingCtas;
}
RingPlan ring_plan(int64_t N, int64_t H, int es, int rows, int64_t least, bool odd, int each) {
    RingPlan p = {0, 0, 0, 0, 0};
    if (H <= least || N < 4 * 152) return p;
    const size_t stage = (size_t)ring_pitch((uint32_t)(H * es), odd) * rows, all = 200 * 1024;
    p.threads = ring_block(H, es, odd);
    if (p.threads > ring_threads(2)) return p;
    while (ring_threads(p.cls) < p.threads) ++p.cls;
    // two stages each at least
    const int64_t fit = (int64_t)(all / (2 * stage)), most = ring_most(N, p.threads, each);
    p.ctas = (int)(fit < 1 ? 1 : fit < most ? fit : most);
    p.stages = (int)(all / p.ctas / stage);
    if (p.stages > kRingStages) p.stages = kRingStages;
    if (p.stages < 2) p.stages = 0;
    p.smem = stage * p.stages;
    return p;
}
// Rows that start anywhere go through the ring from 512 elements on (two warps: the stages' uses are a barrier apart);
// in registers they go by single elements.  bf16 with a residual, registers and ring: 608 x 515 4.9 and 3.8 us, 16,384 x
// 1,001 76 and 36, 608 x 4,881 26.7 and 8.2, 16,384 x 4,881 436 and 126, 4,096 x 12,345 338 and 83.  The backward pass
// has as many parts of dw as CTAs, two rows each at least (with one 1,216 x 1,001 takes 14.1 us, with two 12.6, with
// four 15.1), so that few short rows stay in registers: 1,216 x 1,001 10.7 and 12.6 us, 2,432 x 1,001 15.8 and 16.7, but
// 4,096 x 515 20.7 and 20.2, 16,384 x 1,001 73 and 55, 1,216 x 2,051 18.0 and 14.8, 16,384 x 4,881 1,167 and 183.
constexpr int64_t kRingOdd = 512;

template <int DT, int W, bool NORM, bool Q>
const void *norm_fn(int E) {
    return E == 8 ? reinterpret_cast<const void *>(&norm_kernel<DT, W, 8, NORM, Q>)
                  : reinterpret_cast<const void *>(&norm_kernel<DT, W, kNormElems, NORM, Q>);
}
template <int DT, int W>
const void *norm_form(int E, bool norm, bool q) {
    return !norm ? norm_fn<DT, W, false, true>(E) : q ? norm_fn<DT, W, true, true>(E) : norm_fn<DT, W, true, false>(E);
}
template <int DT, bool ODD, int C>
const void *norm_ring_fn(bool q) {
    return q ? reinterpret_cast<const void *>(&norm_ring_kernel<DT, ODD, true, C>)
             : reinterpret_cast<const void *>(&norm_ring_kernel<DT, ODD, false, C>);
}
template <int DT, bool ODD>
const void *norm_ring_fn(bool q, int cls) {
    return cls == 0 ? norm_ring_fn<DT, ODD, 0>(q) : cls == 1 ? norm_ring_fn<DT, ODD, 1>(q) : norm_ring_fn<DT, ODD, 2>(q);
}
template <int DT>
const void *norm_ring_fn(bool odd, bool q, int cls) {
    return odd ? norm_ring_fn<DT, true>(q, cls) : norm_ring_fn<DT, false>(q, cls);
}
template <int DT, int W>
const void *back_fn(int E, bool big) {  // big only with 16 elements
    return E == 8 ? reinterpret_cast<const void *>(&norm_back_kernel<DT, W, 8, false>)
           : big  ? reinterpret_cast<const void *>(&norm_back_kernel<DT, W, kNormElems, true>)
                  : reinterpret_cast<const void *>(&norm_back_kernel<DT, W, kNormElems, false>);
}
template <int DT, bool ODD>
const void *back_ring_fn(int cls) {
    return cls == 0   ? reinterpret_cast<const void *>(&norm_back_ring_kernel<DT, ODD, 0>)
           : cls == 1 ? reinterpret_cast<const void *>(&norm_back_ring_kernel<DT, ODD, 1>)
                      : reinterpret_cast<const void *>(&norm_back_ring_kernel<DT, ODD, 2>);
}
template <int DT>
const void *back_ring_fn(bool odd, int cls) {
    return odd ? back_ring_fn<DT, true>(cls) : back_ring_fn<DT, false>(cls);
}

// Whether every row of a tensor starts on `bytes` (a row alone needs no stride).
bool rows_on(const void *p, int64_t stride, int64_t N, int es, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (N <= 1 || stride * es % bytes == 0));
}

// Whether a tensor's rows each start as far into 16 bytes of x's type as x's do (`es` bytes an element, x's `xes`), and
// far enough from one another that what shares a row's first and last 16 bytes is in the tensor but at its two ends.
bool rows_alike(const void *p, int64_t stride, int es, const void *x, int64_t xs, int xes) {
    const int64_t ae = 16 / xes;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) / es, x_at = reinterpret_cast<uintptr_t>(x) / xes;
    return !p || (stride >= ae && (stride - xs) % ae == 0 && at % ae == x_at % ae);
}

}  // namespace

int norm_launch(const NormArgs &args, int dtype, bool norm, bool q, cudaStream_t st) {
    NormArgs a = args;
    const int es = dtype == 0 ? 4 : 2, ae = 16 / es;
    const bool vec = a.H % ae == 0 && rows_on(a.x, a.xs, a.N, es, 16) && rows_on(a.r, a.rs, a.N, es, 16) &&
                     rows_on(a.res, a.ress, a.N, es, 16) && rows_on(a.w, 0, 1, 1, 16) &&
                     rows_on(a.out, a.os, a.N, q ? 1 : es, q ? ae : 16);
    const bool odd = !vec && rows_alike(a.x, a.xs, es, a.x, a.xs, es) && rows_alike(a.r, a.rs, es, a.x, a.xs, es) &&
                     rows_alike(a.res, a.ress, es, a.x, a.xs, es) && rows_alike(a.out, a.os, q ? 1 : es, a.x, a.xs, es);
    const RingPlan ring =
        norm && (vec || odd) ? ring_plan(a.N, a.H, es, a.r ? 2 : 1, vec ? 2048 : kRingOdd, odd, 1) : RingPlan{0, 0, 0, 0, 0};
    if (ring.stages > 0) {
        const void *fn = dtype == 0   ? norm_ring_fn<0>(odd, q, ring.cls)
                         : dtype == 1 ? norm_ring_fn<1>(odd, q, ring.cls)
                                      : norm_ring_fn<2>(odd, q, ring.cls);
        if (prepare_kernel(fn, ring.smem, 1) != 0) return -1;
        int stages = ring.stages;
        void *params[] = {&a, &stages};
        return cudaLaunchKernel(fn, dim3((unsigned)(152 * ring.ctas)), dim3((unsigned)ring.threads), params, ring.smem, st) ==
                       cudaSuccess
                   ? 0
                   : -1;
    }
    const int E = norm_elems(a.H, vec);
    const void *fn = dtype == 0   ? (vec ? norm_form<0, 4>(E, norm, q) : norm_form<0, 1>(E, norm, q))
                     : dtype == 1 ? (vec ? norm_form<1, 8>(E, norm, q) : norm_form<1, 1>(E, norm, q))
                                  : (vec ? norm_form<2, 8>(E, norm, q) : norm_form<2, 1>(E, norm, q));
    const dim3 block = norm_block(a.H, E);
    void *params[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)((a.N + block.y - 1) / block.y)), block, params, 0, st) == cudaSuccess
               ? 0
               : -1;
}

unsigned int *norm_status_ptr() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_norm_status) != cudaSuccess) return nullptr;
    return reinterpret_cast<unsigned int *>(p);
}

// Parts of dw: two CTAs an SM (a ring's up to eight), and no more than there are rows.
int64_t norm_back_parts(int64_t N, int64_t H, bool vec) {
    const int64_t y = norm_block(H, norm_elems(H, vec)).y, ctas = (N + y - 1) / y;
    return (ctas < 304 ? ctas : 304) * y;
}
int64_t norm_back_parts(int64_t N, int64_t H) {
    const int64_t a = norm_back_parts(N, H, true), b = norm_back_parts(N, H, false),
                  c = H > kRingOdd && N >= 4 * 152 ? 152 * ring_most(N, ring_block(H, 4, false), kRingBackRows) : 0;
    return a > b ? (a > c ? a : c) : b > c ? b : c;
}

int norm_back_launch(const NormBackArgs &args, int dtype, cudaStream_t st) {
    NormBackArgs a = args;
    const int es = dtype == 0 ? 4 : 2, ae = 16 / es;
    const bool vec = a.H % ae == 0 && rows_on(a.x, a.xs, a.N, es, 16) && rows_on(a.g, a.gs, a.N, es, 16) &&
                     rows_on(a.gr, a.grs, a.N, es, 16) && rows_on(a.dx, a.dxs, a.N, es, 16) && rows_on(a.w, 0, 1, 1, 16);
    const int E = norm_elems(a.H, vec);
    const dim3 block = norm_block(a.H, E);
    int64_t parts = norm_back_parts(a.N, a.H, vec);
    // Up to 4,096 elements two CTAs an SM hold their next row in registers, and as much is under way (16,384 x 4,096
    // bf16 with a residual's gradient, registers and ring: 85 and 96 us, x 5,120 149 and 118, 8,192 x 8,192 94 and 95,
    // 4,096 x 16,384 159 and 140).
    const bool odd = !vec && rows_alike(a.x, a.xs, es, a.x, a.xs, es) && rows_alike(a.g, a.gs, es, a.x, a.xs, es) &&
                     rows_alike(a.gr, a.grs, es, a.x, a.xs, es) && rows_alike(a.dx, a.dxs, es, a.x, a.xs, es);
    const int64_t least = vec ? 4096 : a.N > 16 * 152 ? kRingOdd : 2048;
    const RingPlan ring =
        vec || odd ? ring_plan(a.N, a.H, es, a.gr ? 3 : 2, least, odd, kRingBackRows) : RingPlan{0, 0, 0, 0, 0};
    if (ring.stages > 0) {
        const void *fn = dtype == 0   ? back_ring_fn<0>(odd, ring.cls)
                         : dtype == 1 ? back_ring_fn<1>(odd, ring.cls)
                                      : back_ring_fn<2>(odd, ring.cls);
        if (prepare_kernel(fn, ring.smem, 1) != 0) return -1;
        int stages = ring.stages;
        void *params[] = {&a, &stages};
        parts = 152 * ring.ctas;
        if (cudaLaunchKernel(fn, dim3((unsigned)parts), dim3((unsigned)ring.threads), params, ring.smem, st) != cudaSuccess)
            return -1;
    } else if (a.N > 0) {
        const bool big = a.H > kNormElems * norm_threads(false);
        const void *fn = dtype == 0   ? (vec ? back_fn<0, 4>(E, big) : back_fn<0, 1>(E, big))
                         : dtype == 1 ? (vec ? back_fn<1, 8>(E, big) : back_fn<1, 1>(E, big))
                                      : (vec ? back_fn<2, 8>(E, big) : back_fn<2, 1>(E, big));
        void *params[] = {&a};
        if (cudaLaunchKernel(fn, dim3((unsigned)(parts / block.y)), block, params, 0, st) != cudaSuccess) return -1;
    }
    const float *part = a.part;
    int64_t H = a.H;
    void *dw = a.dw;
    const int wt = a.w_f32 ? 0 : dtype;
    const void *fn = wt == 0   ? reinterpret_cast<const void *>(&norm_weight_grad_kernel<0>)
                     : wt == 1 ? reinterpret_cast<const void *>(&norm_weight_grad_kernel<1>)
                               : reinterpret_cast<const void *>(&norm_weight_grad_kernel<2>);
    void *params[] = {&part, &parts, &H, &dw};
    return cudaLaunchKernel(fn, dim3((unsigned)((H + 31) / 32)), dim3(32, 32), params, 0, st) == cudaSuccess ? 0 : -1;
}

}  // namespace tsa
