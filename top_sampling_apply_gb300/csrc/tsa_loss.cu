// Host side of the row losses, the preference loss's pairs and the final sums.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "tsa_device.cuh"
#include "tsa_host.h"
#include "tsa_loss.cuh"

namespace tsa {

namespace {

using loss_detail::block_sum;
using loss_detail::Sum2;

constexpr int kSumThreads = 1024;
constexpr int kPairThreads = 256;

// One CTA, a fixed order: the same loss for the same rows on every call.
__global__ void __launch_bounds__(kSumThreads) weighted_sum_kernel(const float *x, const float *w, float w_s,
                                                                   int64_t n, float *out) {
    __shared__ Sum2 sh[kSumThreads / 32];
    pdl_wait_primary();
    Sum2 s = {0.f, 0.f};
    for (int64_t i = threadIdx.x; i < n; i += kSumThreads) {
        const float wi = w ? w[i] : w_s;
        if (wi != 0.f) s.add_product(wi, x[i]);
    }
    s = block_sum<kSumThreads>(s, sh);
    if (threadIdx.x == 0) out[0] = s.value();
}

// One CTA a pair: the two sequences' log-ratios, the pair's loss, and the
// coefficient of each of their rows.  With h = beta (R_c - R_r) - margin,
//     loss = (1 - eps) ln(1 + e^-h) + eps ln(1 + e^h),
//     d loss / dh = -(1 - eps) / (1 + e^h) + eps / (1 + e^-h).
// A row counts if its weight is not 0, its token is in the vocabulary
// (skipped rows have Z = 1, m = 0 and log-probability 0, and the sums' pass
// left their coefficients 0) and its log-probability is not -inf.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(PairArgs a, RowLossArgs r) {
    __shared__ Sum2 sh[kPairThreads / 32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int64_t p = blockIdx.x;
    Sum2 R[2];
    float W[2];
    int64_t lo[2], hi[2];
    auto weight = [&](int64_t i) {  // 0 for a row that does not count
        const float w = a.weight ? a.weight[i] : 1.f;
        const int64_t tok = r.tokens[i];
        return tok >= 0 && tok < r.V && a.logprob[i] != -INFINITY && r.fin[i].w != -INFINITY ? w : 0.f;
    };
    for (int s = 0; s < 2; ++s) {
        const int64_t q = p + s * a.P;
        lo[s] = min(max(a.seq_start[q], (int64_t)0), a.N);
        hi[s] = min(max(a.seq_start[q + 1], lo[s]), a.N);
        Sum2 sum = {0.f, 0.f}, n = {0.f, 0.f};
        for (int64_t i = lo[s] + threadIdx.x; i < hi[s]; i += kPairThreads) {
            const float w = weight(i);
            if (w == 0.f) continue;
            // the difference with its rounding error
            Sum2 d = {a.logprob[i], 0.f};
            if (a.ref_logprob) d.add(-a.ref_logprob[i]);
            sum.add_product(w, d.s);
            if (fabsf(d.s) < INFINITY) sum.add_product(w, d.c);  // a reference of -inf leaves no error, but NaN
            n.add(w);
        }
        R[s] = block_sum<kPairThreads>(sum, sh);
        W[s] = 1.f;
        if (a.average) {
            const float total = block_sum<kPairThreads>(n, sh).value();
            W[s] = total != 0.f ? 1.f / total : 0.f;
            Sum2 mean = {0.f, 0.f};
            mean.add_product(R[s].s, W[s]);
            mean.c += R[s].c * W[s];
            R[s] = mean;
        }
    }
    Sum2 diff = R[0];
    diff.add(Sum2{-R[1].s, -R[1].c});
    const float h = a.beta * diff.value() - a.margin;
    // ln(1 + e^-|h|) and the two logistic values from one exponential
    const float q = expf(-fabsf(h)), l1 = log1pf(q), big = 1.f / (1.f + q), small = q / (1.f + q);
    const float plus = h > 0.f ? big : small, minus = h > 0.f ? small : big;  // s(h), s(-h)
    if (threadIdx.x == 0) {
        const float soft_m = l1 + fmaxf(-h, 0.f), soft_p = l1 + fmaxf(h, 0.f);
        // a coefficient of 0 leaves its term out, even where that is infinite
        a.pair_loss[p] = h != h ? h
                                : (a.smooth != 1.f ? (1.f - a.smooth) * soft_m : 0.f) +
                                      (a.smooth != 0.f ? a.smooth * soft_p : 0.f);
        a.reward[p] = a.beta * R[0].value();
        a.reward[p + a.P] = a.beta * R[1].value();
    }
    const float dh = h != h ? h : -(1.f - a.smooth) * minus + a.smooth * plus;
    for (int s = 0; s < 2; ++s) {
        const float d = (s == 0 ? dh : -dh) * a.beta / (float)a.P * W[s];
        for (int64_t i = lo[s] + threadIdx.x; i < hi[s]; i += kPairThreads) {
            const float w = weight(i);
            if (w == 0.f) continue;
            // from (0, Z, 0, m) to k1, k2, a and m
            const float4 k = r.fin[i];
            const float T = r.temperature_s > 0.f ? r.temperature_s : 1.f, g = d * w / T;
            float f;
            loss_detail::near_shift(k.w, loss_detail::kLog2eL / T, &f);
            r.fin[i] = make_float4(-g / k.y * f, 0.f, g, k.w);
        }
    }
}

__device__ unsigned int g_loss_status;

const void *loss_kernel(int dtype, int mode, bool ent) {
    return dtype == 0 ? row_loss_kernel_f32(mode, ent)
                      : (dtype == 1 ? row_loss_kernel_f16(mode, ent) : row_loss_kernel_bf16(mode, ent));
}
const void *held_kernel(int dtype, bool ent, int threads) {
    return dtype == 0 ? row_held_kernel_f32(ent, threads)
                      : (dtype == 1 ? row_held_kernel_f16(ent, threads) : row_held_kernel_bf16(ent, threads));
}
const void *grad_kernel(int dtype, bool ent) {
    return dtype == 0 ? row_grad_kernel_f32(ent) : (dtype == 1 ? row_grad_kernel_f16(ent) : row_grad_kernel_bf16(ent));
}

// A launch that may start its prologue while the kernel before it drains;
// such a kernel waits for it before it touches memory.
int launch_pdl(const void *fn, dim3 grid, int threads, void **params, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, params) == cudaSuccess ? 0 : -1;
}

}  // namespace

unsigned int *row_loss_status_ptr() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_loss_status) != cudaSuccess) return nullptr;
    return reinterpret_cast<unsigned int *>(p);
}

// Clusters of C CTAs that the GPU runs at once; asked once a kernel, size and
// device.
static int64_t resident_clusters(const void *fn, const cudaLaunchConfig_t &cfg, int C) {
    struct Known {
        const void *fn;
        int device, C, n;
    };
    static std::mutex mu;
    static Known known[256];
    static int count = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < count; ++i)
        if (known[i].fn == fn && known[i].device == dev && known[i].C == C) return known[i].n;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) return 0;
    if (count < 256) known[count++] = Known{fn, dev, C, n};
    return n;
}

// The CTAs that share a streamed row: one, and more where there are fewer rows
// than SMs, down to 256 vectors a CTA.
static int row_cluster(int64_t B, int64_t V, int es) {
    const int64_t bytes = V * es;
    int C = 1;
    while (C < loss_detail::kRowMaxCluster && B * C * 2 <= 152 && bytes / 16 >= 512 * C) C *= 2;
    return C;
}

// The threads of a CTA that holds a row, or its share of one.
static int held_threads(int64_t V, int es) {
    const int64_t nvec = V * es / 16;
    for (int t = 128; t < loss_detail::kHeldThreads; t *= 2)
        if (nvec <= (int64_t)t * loss_detail::kHeldVecs) return t;
    return loss_detail::kHeldThreads;
}
// The CTAs that hold a row together, 0 if its vectors do not fit eight.  Fewer
// rows than SMs are spread further, down to one vector a thread: 8 rows of
// 8,192 fp32 logits use 64 CTAs instead of 8.
static int held_cluster(int64_t B, int64_t V, int es) {
    const int64_t nvec = V * es / 16;
    const int64_t one = held_threads(V, es), per = one * loss_detail::kHeldVecs;
    int C = 1;
    while (C <= loss_detail::kHeldCluster && (nvec + C - 1) / C > per) C *= 2;
    if (C > loss_detail::kHeldCluster) return 0;
    while (C < loss_detail::kHeldCluster && B * C * 2 <= 152 && nvec / (2 * C) >= one) C *= 2;
    return C;
}

// A launch of clusters of C CTAs, a row each; more rows than clusters that run
// at once go round them.
static int launch_rows(const void *fn, int64_t B, int C, int threads, size_t smem, void **params, cudaStream_t st) {
    if (prepare_kernel(fn, smem, C) != 0) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((B < 65536 ? B : 65536) * C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int64_t n = resident_clusters(fn, cfg, C);
    if (n < 1) return -1;
    if (B > n) cfg.gridDim.x = (unsigned)(n * C);
    return cudaLaunchKernelExC(&cfg, fn, params) == cudaSuccess ? 0 : -1;
}

bool row_is_held(int64_t V, int dtype) { return held_cluster(1 << 20, V, dtype == 0 ? 4 : 2) > 0; }

int row_loss_launch(const RowLossArgs &args, int dtype, int mode, bool ent, cudaStream_t st) {
    using namespace loss_detail;
    const int es = dtype == 0 ? 4 : 2;
    RowLossArgs a = args;
    unsigned int *status = row_loss_status_ptr();
    if (!status) return -1;
    int lg = 0;
    if (args.grad) {
        const int C = held_cluster(args.B, args.V, es);
        if (C == 0) return -1;
        while ((1 << lg) < C) ++lg;
        void *params[] = {&a, &lg, &status};
        const int threads = held_threads(args.V, es);
        return launch_rows(held_kernel(dtype, ent, threads), args.B, C, threads, held_smem(threads), params, st);
    }
    const int C = row_cluster(args.B, args.V, es);
    while ((1 << lg) < C) ++lg;
    const int64_t vecs = (args.V * es / 16 + C - 1) / C;  // a CTA's vectors at most
    int stages = (int)((vecs + kRowStage - 1) / kRowStage);
    if (stages < 1) stages = 1;
    // a stage as long as fits, in whole steps of the working warps
    int nu = (int)((vecs < kRowStage ? vecs : kRowStage) + kRowUsers - 1) / kRowUsers;
    if (nu < 1) nu = 1;
    void *params[] = {&a, &lg, &stages, &nu, &status};
    return launch_rows(loss_kernel(dtype, mode, ent), args.B, C, kRowThreads, kRowSmem, params, st);
}

int row_grad_launch(const RowLossArgs &args, int dtype, bool ent, const float *pair_loss, int64_t pairs, float *loss,
                    cudaStream_t st) {
    const void *fn = grad_kernel(dtype, ent);
    const int64_t per = (int64_t)loss_detail::kKnownThreads * loss_detail::kKnownU * (dtype == 0 ? 4 : 8);
    const unsigned slices = (unsigned)((args.V + per - 1) / per);
    const unsigned y = (unsigned)(args.B < 32768 ? args.B : 32768);
    const unsigned z = (unsigned)((args.B + y - 1) / y);
    RowLossArgs a = args;
    void *params[] = {&a, &pair_loss, &pairs, &loss};
    return launch_pdl(fn, dim3(slices, y, z), loss_detail::kKnownThreads, params, st);
}

int pair_launch(const PairArgs &args, const RowLossArgs &rows, cudaStream_t st) {
    PairArgs a = args;
    RowLossArgs r = rows;
    void *params[] = {&a, &r};
    return launch_pdl(reinterpret_cast<const void *>(&pair_kernel), dim3((unsigned)args.P), kPairThreads, params, st);
}

int weighted_sum_launch(const float *x, const float *w, float w_s, int64_t n, float *out, cudaStream_t st) {
    void *params[] = {&x, &w, &w_s, &n, &out};
    return launch_pdl(reinterpret_cast<const void *>(&weighted_sum_kernel), dim3(1), kSumThreads, params, st);
}

}  // namespace tsa
