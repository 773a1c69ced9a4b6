// The cross entropy of the head's scores with its gradients, without the
// scores.  With z = h W^T + b, z <- cap tanh(z / cap), l = ln sum_j exp(z_j):
//     row = l - z_t + c l^2,   loss = sum over rows of w row,
//     g_j = w ((1 + 2 c l) exp(z_j - l) - [j = t]) (1 - (z_j / cap)^2),
//     dH = G W,  dW = G^T H,  db = sum over rows of G.
// The rows that count are brought together first, so that skipped ones cost
// nothing and whatever they hold stays out of the products.  Their
// log-sum-exps come from the products of lm_head_logprob; then the vocabulary
// goes by in pieces: a piece's scores again, turned into its part of G in
// bf16, and that part's products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_tcgen05.cuh"

namespace tsa {

namespace {

// One CTA: where each row that counts goes, in order; its target and weight.
// Without weights each has 1 / (number of them).  Places up to the next
// multiple of 128 get a weight of 0 and no target.
__global__ void __launch_bounds__(1024) xent_rows_kernel(const XentArgs a) {
    __shared__ int s_warp[32], s_base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_base = 0;
    __syncthreads();
    for (int64_t m0 = 0; m0 < a.M; m0 += 1024) {
        const int64_t m = m0 + threadIdx.x;
        int64_t t = -1;
        float w = 1.f;
        if (m < a.M) {
            t = a.targets[m];
            if (a.row_weight) w = a.row_weight[m];
        }
        const bool live = t >= 0 && t < a.V && w != 0.f;
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, live);
        if (lane == 0) s_warp[warp] = __popc(vote);
        __syncthreads();
        if (warp == 0) {
            const int own = s_warp[lane];
            int sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += x;
            }
            s_warp[lane] = sum - own + s_base;
            __syncwarp();
            if (lane == 31) s_base += sum;
        }
        __syncthreads();
        if (m < a.M) {
            const int at = s_warp[warp] + __popc(vote & ((1u << lane) - 1u));
            a.place[m] = live ? at : -1;
            if (live) {
                a.rows[at] = (int32_t)m;
                a.tokens[at] = t;
                a.weight_c[at] = w;
            }
        }
        __syncthreads();
    }
    const int n = s_base;
    if (threadIdx.x == 0) a.count[0] = n;
    const int64_t pad = xent_padded(a.M);
    for (int64_t i = threadIdx.x; i < pad; i += 1024) {
        if (i >= n) {
            a.tokens[i] = -1;
            a.weight_c[i] = 0.f;
            a.row_loss_c[i] = 0.f;
        } else if (!a.row_weight) {
            a.weight_c[i] = 1.f / (float)n;
        }
    }
}

// The rows that count, one after another; zeros up to a multiple of 128 of
// them (128 at least), and in the outputs of skipped rows.
__global__ void __launch_bounds__(128) xent_gather_kernel(const XentArgs a) {
    const int64_t b = blockIdx.x, vecs = a.H / 8;
    const int n = a.count[0];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (b >= a.M) {
        const int64_t i = n + (b - a.M), end = n < 1 ? 128 : ((int64_t)n + 127) / 128 * 128;
        if (i < end)
            for (int64_t v = threadIdx.x; v < vecs; v += 128) reinterpret_cast<uint4 *>(a.hidden_c)[i * vecs + v] = zero;
        return;
    }
    const int at = a.place[b];
    if (at >= 0) {
        const uint4 *from = reinterpret_cast<const uint4 *>(a.hidden + b * a.hstride);
        for (int64_t v = threadIdx.x; v < vecs; v += 128) reinterpret_cast<uint4 *>(a.hidden_c)[at * vecs + v] = from[v];
        return;
    }
    if (a.dh)
        for (int64_t v = threadIdx.x; v < vecs; v += 128) reinterpret_cast<uint4 *>(a.dh + b * a.dhstride)[v] = zero;
    if (threadIdx.x == 0) a.row_loss[b] = a.lse[b] = 0.f;
}

// The losses of the rows that count, and what their gradients need.
__global__ void __launch_bounds__(256) xent_finish_kernel(const XentArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= xent_padded(a.M)) return;
    if (i >= a.count[0]) {
        a.coef[i] = make_float4(0.f, 0.f, INFINITY, 0.f);
        return;
    }
    const float l = a.lse_c[i], w = a.weight_c[i], c = a.z_loss;
    const float loss = -a.logprob_c[i] + (c != 0.f ? c * l * l : 0.f);
    a.row_loss_c[i] = loss;
    a.row_loss[a.rows[i]] = loss;
    a.lse[a.rows[i]] = l;
    a.coef[i] = make_float4(c != 0.f ? w * fmaf(2.f * c, l, 1.f) : w, w, l, 0.f);
}

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// 64 x 64 outputs of sum_k A(m, k) B(n, k) a CTA of 256 threads, both from any
// strides; 4 x 4 outputs a thread.
struct Operand {
    const uint16_t *p;
    int64_t row, col, rows;  // strides of m (or n) and k; rows beyond `rows` are 0
};
__device__ __forceinline__ void tile_64(const Operand &A, const Operand &B, int64_t m0, int64_t n0, int64_t K,
                                        float (&acc)[4][4]) {
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            // along whichever of the two is contiguous
            const int ra = A.col == 1 ? i >> 4 : i & 63, ka = A.col == 1 ? i & 15 : i >> 6;
            const int rb = B.col == 1 ? i >> 4 : i & 63, kb = B.col == 1 ? i & 15 : i >> 6;
            sa[ka][ra] = m0 + ra < A.rows && k0 + ka < K ? bf(A.p[(m0 + ra) * A.row + (k0 + ka) * A.col]) : 0.f;
            sb[kb][rb] = n0 + rb < B.rows && k0 + kb < K ? bf(B.p[(n0 + rb) * B.row + (k0 + kb) * B.col]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) xent_scores_kernel(const XentArgs a, int64_t v0, int64_t width) {
    __shared__ float s_col[16][64];
    const int n = a.count[0], tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int64_t end = n < 1 ? 128 : ((int64_t)n + 127) / 128 * 128;
    if (m0 >= end) return;
    float z[4][4] = {};
    tile_64({a.hidden_c, a.H, 1, end}, {a.weight, a.wstride, 1, a.V}, m0, v0 + c0, a.H, z);
    float col[4] = {};
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        const float4 k = a.coef[m];
        const int64_t t = a.tokens[m] - v0;
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + tx + 16 * j, v = v0 + c;
            float g = 0.f;
            if (c < width && v < a.V && m < n) {
                float x = z[i][j] + (a.bias ? a.bias[v] : 0.f), slope = 1.f;
                if (a.cap > 0.f) {
                    const float y = tanhf(x / a.cap);
                    x = a.cap * y;
                    slope = 1.f - y * y;
                }
                x = fmaxf(x, -INFINITY);
                g = (k.x * expf(x - k.z) - (c == t ? k.y : 0.f)) * slope;
            }
            col[j] += g;
            if (c < width) a.grad[m * width + c] = __bfloat16_as_ushort(__float2bfloat16_rn(g));
        }
    }
    if (!a.db) return;
    for (int j = 0; j < 4; ++j) s_col[ty][tx + 16 * j] = col[j];
    __syncthreads();
    if (threadIdx.x < 64 && c0 + threadIdx.x < width) {
        float s = 0.f;
        for (int i = 0; i < 16; ++i) s += s_col[i][threadIdx.x];
        a.db_part[(m0 / 64) * width + c0 + threadIdx.x] = s;
    }
}

__global__ void __launch_bounds__(256) xent_bias_kernel(const XentArgs a, int64_t v0, int64_t width) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= width || v0 + c >= a.V) return;
    const int n = a.count[0];
    float s = 0.f;
    for (int64_t p = 0; p * 64 < n; ++p) s += a.db_part[p * width + c];
    a.db[v0 + c] = s;
}

// z = 0: a piece's dW; 1: its part of dH.
__global__ void __launch_bounds__(256) xent_products_kernel(const XentArgs a, int64_t v0, int64_t width, int dh) {
    const int n = a.count[0], tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, h0 = (int64_t)blockIdx.x * 64;
    const int64_t end = n < 1 ? 128 : ((int64_t)n + 127) / 128 * 128;
    const int64_t last = v0 + width < a.V ? v0 + width : a.V;
    float z[4][4] = {};
    if (dh) {
        if (m0 >= n) return;
        tile_64({a.grad, width, 1, end}, {a.weight + v0 * a.wstride, 1, a.wstride, a.H}, m0, h0, last - v0, z);
    } else {
        tile_64({a.grad, 1, width, width}, {a.hidden_c, 1, a.H, a.H}, m0, h0, end, z);
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i, h = h0 + tx + 16 * j;
            if (h >= a.H) continue;
            if (!dh) {
                if (v0 + m < last && m < width)
                    a.dw[(v0 + m) * a.dwstride + h] = __bfloat16_as_ushort(__float2bfloat16_rn(z[i][j]));
            } else if (m < n) {
                float s = z[i][j];
                if (v0 > 0) s += a.acc[m * a.H + h];
                if (last < a.V)
                    a.acc[m * a.H + h] = s;
                else
                    a.dh[a.rows[m] * a.dhstride + h] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
            }
        }
}

}  // namespace

// A piece of the vocabulary: its part of G takes at most 128 MB.
int64_t xent_piece(int64_t M, int64_t V) {
    const int64_t most = (V + 255) / 256 * 256;
    const int64_t fit = ((int64_t)128 << 20) / (2 * xent_padded(M)) / 256 * 256;
    return fit < 256 ? 256 : fit < most ? fit : most;
}

int xent_launch(const XentArgs &args, const LmLogprobArgs &scores, cudaStream_t st) {
    const XentArgs &a = args;
    xent_rows_kernel<<<1, 1024, 0, st>>>(a);
    xent_gather_kernel<<<(unsigned)(a.M + 128), 128, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return -1;
    for (int64_t m = 0; m < a.M; m += kLmRows) {
        LmLogprobArgs s = scores;
        s.M = a.M - m < kLmRows ? a.M - m : kLmRows;
        s.hidden = scores.hidden + m * a.H;
        s.tokens = scores.tokens + m;
        s.out = scores.out + m;
        s.lse = scores.lse + m;
        s.first = m;
        if (lm_logprob_launch(s, st) != 0) return -1;
    }
    const int64_t pad = xent_padded(a.M);
    xent_finish_kernel<<<(unsigned)((pad + 255) / 256), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return -1;
    if (weighted_sum_launch(a.row_loss_c, a.weight_c, 0.f, a.M, a.loss, st) != 0) return -1;
    if (!a.dh && !a.dw && !a.db) return 0;
    const int64_t piece = xent_piece(a.M, a.V);
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const unsigned rows = (unsigned)(pad / 64), cols = (unsigned)(piece / 64), width = (unsigned)((a.H + 63) / 64);
        xent_scores_kernel<<<dim3(cols, rows), 256, 0, st>>>(a, v0, piece);
        if (a.db) xent_bias_kernel<<<(unsigned)((piece + 255) / 256), 256, 0, st>>>(a, v0, piece);
        if (a.dh) xent_products_kernel<<<dim3(width, rows), 256, 0, st>>>(a, v0, piece, 1);
        if (a.dw) xent_products_kernel<<<dim3(width, cols), 256, 0, st>>>(a, v0, piece, 0);
        if (cudaGetLastError() != cudaSuccess) return -1;
    }
    return 0;
}

}  // namespace tsa
