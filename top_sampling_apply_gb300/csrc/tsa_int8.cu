// The head's scores from 8-bit integers with a scale for each hidden row and
// each vocabulary entry:
//     z[m, v] = hs[m] ws[v] sum_k h[m, k] w[v, k]  (+ b[v]),
// the sum over integers exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_host.h"

namespace tsa {

namespace {

__device__ __forceinline__ void store_score(void *p, int64_t i, float x, int dtype) {
    if (dtype == 0)
        static_cast<float *>(p)[i] = x;
    else if (dtype == 1)
        static_cast<__half *>(p)[i] = __float2half_rn(x);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// A warp a vocabulary entry, eight hidden rows at a time, 16 columns a lane.
__global__ void __launch_bounds__(256) int8_scores_kernel(const Int8Args a) {
    const int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (v >= a.V) return;
    for (int64_t m0 = (int64_t)blockIdx.y * 8; m0 < a.M; m0 += (int64_t)gridDim.y * 8) {
        int acc[8] = {};
        for (int64_t k = lane * 16; k < a.H; k += 512) {
            const int4 w = *reinterpret_cast<const int4 *>(a.weight + v * a.wstride + k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (m0 + i >= a.M) break;
                const int4 h = *reinterpret_cast<const int4 *>(a.hidden + (m0 + i) * a.hstride + k);
                acc[i] = __dp4a(w.x, h.x, __dp4a(w.y, h.y, __dp4a(w.z, h.z, __dp4a(w.w, h.w, acc[i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = __reduce_add_sync(0xFFFFFFFFu, acc[i]);
            if (lane == i && m0 + i < a.M) {
                const float z = (float)s * a.hscale[m0 + i] * a.wscale[v] + (a.bias ? a.bias[v] : 0.f);
                store_score(a.out, (m0 + i) * a.ostride + v, z, a.dtype);
            }
        }
    }
}

}  // namespace

int int8_launch(const Int8Args &a, cudaStream_t st) {
    const int64_t y = (a.M + 7) / 8;
    int8_scores_kernel<<<dim3((unsigned)((a.V + 7) / 8), (unsigned)(y < 65535 ? y : 65535)), 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace tsa
