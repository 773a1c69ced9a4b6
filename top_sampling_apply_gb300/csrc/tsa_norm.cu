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

#include "tsa_device.cuh"
#include "tsa_host.h"

namespace tsa {

namespace {

constexpr int kNormThreads = 512;  // most threads a row: 32 elements each are kNormMaxH

// W elements of a row at `i`: a 16-byte vector, or single elements where a
// row does not start on 16 bytes.  Plain loads: an output may be an input's
// own memory, and every element is read by the thread that writes it.
template <int DT, int W>
struct Part {
    static __device__ __forceinline__ void load(const void *p, int64_t i, float *x) {
        if constexpr (W > 1) {
            const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * Elem<DT>::SIZE);
            Elem<DT>::unpack(v, x);
        } else if constexpr (DT == 0) {
            x[0] = static_cast<const float *>(p)[i];
        } else if constexpr (DT == 1) {
            x[0] = __half2float(static_cast<const __half *>(p)[i]);
        } else {
            x[0] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
        }
    }
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

// NORM = false: the rows themselves in 8 bits.
template <int DT, int W, int E, bool NORM, bool Q>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
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
        const float most = __uint_as_float(row_max(top, sh_max, 0));
        // A largest value under 2^-100 would overflow the reciprocal: such rows
        // are brought up by 2^64 first.  A row that is not finite has codes 0
        // under a scale of NaN.
        const bool finite = most < INFINITY;
        const float up = most < 0x1p-100f ? 0x1p64f : 1.f;
        const float f = finite && most > 0.f ? 127.f / (most * up) : 0.f;
        if (in && threadIdx.x == 0) a.scale[row] = finite ? most / 127.f : __int_as_float(0x7FC00000);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = finite ? v[i][j] * up * f : 0.f;
                P::store_codes(static_cast<int8_t *>(a.out), row * a.os + c, v[i]);
            }
        }
    }
}

// Rows go round the CTAs, so that a thread keeps its columns' part of dw in
// registers; a part a CTA (and row of threads) goes to the workspace.
template <int DT, int W, int E>
__global__ void __launch_bounds__(kNormThreads) norm_back_kernel(NormBackArgs a) {
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
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.N; r0 += (int64_t)gridDim.x * blockDim.y, turn ^= 1) {
        const int64_t row = r0 + threadIdx.y;
        const bool in = row < a.N;
        const float rstd = in ? a.rstd[row] : 0.f;
        float h[NV][W], f[NV][W], dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
#pragma unroll
            for (int j = 0; j < W; ++j) h[i][j] = f[i][j] = 0.f;
            if (in && c < H) {
                P::load(a.x, row * a.xs + c, h[i]);
                P::load(a.g, row * a.gs + c, f[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
                float w[W];
                P::weight(a.w, a.w_f32, c, w);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    h[i][j] *= rstd;
                    acc[i][j] = fmaf(f[i][j], h[i][j], acc[i][j]);
                    f[i][j] *= w[j];
                    dot = fmaf(f[i][j], h[i][j], dot);
                }
            }
        }
        const float mean = row_sum(dot, sh, turn) / (float)H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (in && c < H) {
                float add[W];
#pragma unroll
                for (int j = 0; j < W; ++j) add[j] = 0.f;
                if (a.gr) P::load(a.gr, row * a.grs + c, add);
#pragma unroll
                for (int j = 0; j < W; ++j) f[i][j] = fmaf(rstd, fmaf(-h[i][j], mean, f[i][j]), add[j]);
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
// Elements a thread: few for short rows, so that enough loads are under way.
int norm_elems(int64_t H) { return H <= 2048 ? 8 : H <= 8192 ? 16 : 32; }

template <int DT, int W, bool NORM, bool Q>
const void *norm_fn(int E) {
    return E == 8    ? reinterpret_cast<const void *>(&norm_kernel<DT, W, 8, NORM, Q>)
           : E == 16 ? reinterpret_cast<const void *>(&norm_kernel<DT, W, 16, NORM, Q>)
                     : reinterpret_cast<const void *>(&norm_kernel<DT, W, 32, NORM, Q>);
}
template <int DT, int W>
const void *norm_form(int E, bool norm, bool q) {
    return !norm ? norm_fn<DT, W, false, true>(E) : q ? norm_fn<DT, W, true, true>(E) : norm_fn<DT, W, true, false>(E);
}
template <int DT, int W>
const void *back_fn(int E) {
    return E == 8    ? reinterpret_cast<const void *>(&norm_back_kernel<DT, W, 8>)
           : E == 16 ? reinterpret_cast<const void *>(&norm_back_kernel<DT, W, 16>)
                     : reinterpret_cast<const void *>(&norm_back_kernel<DT, W, 32>);
}

// Whether every row of a tensor starts on `bytes` (a row alone needs no stride).
bool rows_on(const void *p, int64_t stride, int64_t N, int es, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (N <= 1 || stride * es % bytes == 0));
}

}  // namespace

int norm_launch(const NormArgs &args, int dtype, bool norm, bool q, cudaStream_t st) {
    NormArgs a = args;
    const int es = dtype == 0 ? 4 : 2, ae = 16 / es;
    const bool vec = a.H % ae == 0 && rows_on(a.x, a.xs, a.N, es, 16) && rows_on(a.r, a.rs, a.N, es, 16) &&
                     rows_on(a.res, a.ress, a.N, es, 16) && rows_on(a.w, 0, 1, 1, 16) &&
                     rows_on(a.out, a.os, a.N, q ? 1 : es, q ? ae : 16);
    const int E = norm_elems(a.H);
    const void *fn = dtype == 0   ? (vec ? norm_form<0, 4>(E, norm, q) : norm_form<0, 1>(E, norm, q))
                     : dtype == 1 ? (vec ? norm_form<1, 8>(E, norm, q) : norm_form<1, 1>(E, norm, q))
                                  : (vec ? norm_form<2, 8>(E, norm, q) : norm_form<2, 1>(E, norm, q));
    const dim3 block = norm_block(a.H, E);
    void *params[] = {&a};
    return cudaLaunchKernel(fn, dim3((unsigned)((a.N + block.y - 1) / block.y)), block, params, 0, st) == cudaSuccess
               ? 0
               : -1;
}

// Parts of dw: two CTAs an SM, and no more than there are rows.
int64_t norm_back_parts(int64_t N, int64_t H) {
    const int64_t y = norm_block(H, norm_elems(H)).y, ctas = (N + y - 1) / y;
    return (ctas < 304 ? ctas : 304) * y;
}

int norm_back_launch(const NormBackArgs &args, int dtype, cudaStream_t st) {
    NormBackArgs a = args;
    const int es = dtype == 0 ? 4 : 2, ae = 16 / es;
    const bool vec = a.H % ae == 0 && rows_on(a.x, a.xs, a.N, es, 16) && rows_on(a.g, a.gs, a.N, es, 16) &&
                     rows_on(a.gr, a.grs, a.N, es, 16) && rows_on(a.dx, a.dxs, a.N, es, 16) && rows_on(a.w, 0, 1, 1, 16);
    const int E = norm_elems(a.H);
    const dim3 block = norm_block(a.H, E);
    int64_t parts = norm_back_parts(a.N, a.H);
    if (a.N > 0) {
        const void *fn = dtype == 0   ? (vec ? back_fn<0, 4>(E) : back_fn<0, 1>(E))
                         : dtype == 1 ? (vec ? back_fn<1, 8>(E) : back_fn<1, 1>(E))
                                      : (vec ? back_fn<2, 8>(E) : back_fn<2, 1>(E));
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
