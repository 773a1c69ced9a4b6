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

namespace tsa {

namespace {

constexpr float kLog2eH = 1.4426950408889634f;
constexpr int kPlainThreads = 256, kPlainChunk = 256, kPlainRows = 4;

__device__ __forceinline__ float row_temp(const LmLogprobArgs &a, int64_t row) {
    const float T = a.temperature ? __ldg(a.temperature + row) : a.temperature_s;
    return T > 0.f ? T : 1.f;
}
// (m, Z) of two parts against the larger maximum; c2 = log2(e) / T.  An empty
// part is (-inf, 0).
__device__ __forceinline__ float2 join(float2 a, float2 b, float c2) {
    const bool up = b.x > a.x;
    const float2 hi = up ? b : a, lo = up ? a : b;
    const float f = hi.x == lo.x ? 1.f : ex2_approx(fmaxf((lo.x - hi.x) * c2, -1.0e4f));
    return make_float2(hi.x, fmaf(lo.y, f, hi.y));
}
// cap tanh(z / cap) = cap (1 - 2 / (1 + e^(2 z / cap))): within 2^-22 cap.
__device__ __forceinline__ float soft_cap(float z, float cap, float k) {
    return cap > 0.f ? cap - __fdividef(2.f * cap, 1.f + ex2_approx(z * k)) : z;
}

__global__ void __launch_bounds__(kPlainThreads) lm_logprob_plain_kernel(LmLogprobArgs a) {
    __shared__ float2 sh[kPlainThreads / 32][kPlainRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t v0 = (int64_t)blockIdx.x * kPlainChunk, m0 = (int64_t)blockIdx.y * kPlainRows;
    const float k = a.cap > 0.f ? 2.f * kLog2eH / a.cap : 0.f;
    float2 s[kPlainRows];
    float c2[kPlainRows];
    for (int r = 0; r < kPlainRows; ++r) {
        s[r] = make_float2(-INFINITY, 0.f);
        c2[r] = m0 + r < a.M ? kLog2eH / row_temp(a, m0 + r) : 1.f;
    }
    for (int64_t v = v0 + warp; v < v0 + kPlainChunk && v < a.V; v += kPlainThreads / 32) {
        float d[kPlainRows] = {};
        for (int64_t h = lane; h < a.H; h += 32) {
            const float w = Elem<2>::load1(a.weight + v * a.wstride, h);
            for (int r = 0; r < kPlainRows; ++r)
                if (m0 + r < a.M) d[r] = fmaf(w, Elem<2>::load1(a.hidden + (m0 + r) * a.hstride, h), d[r]);
        }
        for (int r = 0; r < kPlainRows; ++r) {
            if (m0 + r >= a.M) break;
            float z = warp_sum_f32(d[r]);
            if (a.bias) z += a.bias[v];
            z = fmaxf(soft_cap(z, a.cap, k), -INFINITY);
            if (a.mask && !(((uint32_t)a.mask[(m0 + r) * a.mstride + (v >> 5)] >> (v & 31)) & 1u)) z = -INFINITY;
            if (lane == 0 && a.tokens[m0 + r] == v) a.tok[m0 + r] = z;
            if (z > -INFINITY) s[r] = join(s[r], make_float2(z, 1.f), c2[r]);
        }
    }
    if (lane == 0)
        for (int r = 0; r < kPlainRows; ++r) sh[warp][r] = s[r];
    __syncthreads();
    if (threadIdx.x < kPlainRows && m0 + threadIdx.x < a.M) {
        float2 t = sh[0][threadIdx.x];
        for (int w = 1; w < kPlainThreads / 32; ++w) t = join(t, sh[w][threadIdx.x], c2[threadIdx.x]);
        a.part[(int64_t)blockIdx.x * a.M + m0 + threadIdx.x] = t;
    }
}

// A row's parts: 32 rows a CTA, 16 threads a row, then a tree over them.
constexpr int kJoinY = 16;
__global__ void __launch_bounds__(32 * kJoinY) lm_logprob_join_kernel(LmLogprobArgs a, int64_t parts) {
    __shared__ float2 sh[kJoinY][32];
    pdl_wait_primary();
    const int64_t row = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const float T = row < a.M ? row_temp(a, row) : 1.f, c2 = kLog2eH / T;
    float2 s = make_float2(-INFINITY, 0.f);
    if (row < a.M)
        for (int64_t p = threadIdx.y; p < parts; p += kJoinY) s = join(s, a.part[p * a.M + row], c2);
    sh[threadIdx.y][threadIdx.x] = s;
#pragma unroll
    for (int o = kJoinY / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.y < o)
            sh[threadIdx.y][threadIdx.x] = join(sh[threadIdx.y][threadIdx.x], sh[threadIdx.y + o][threadIdx.x], c2);
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

int64_t lm_logprob_parts(int64_t, int64_t V) { return (V + kPlainChunk - 1) / kPlainChunk; }

int lm_logprob_launch(const LmLogprobArgs &args, cudaStream_t st) {
    int64_t parts = lm_logprob_parts(args.M, args.V);
    LmLogprobArgs a = args;
    void *params[] = {&a, &parts};
    const dim3 grid((unsigned)parts, (unsigned)((a.M + kPlainRows - 1) / kPlainRows));
    if (cudaLaunchKernel(reinterpret_cast<const void *>(&lm_logprob_plain_kernel), grid, dim3(kPlainThreads), params, 0,
                         st) != cudaSuccess)
        return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + 31) / 32));
    cfg.blockDim = dim3(32, kJoinY);
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

}  // namespace tsa
