// C-ABI entry points of the training-side calls: argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/tsa.h"
#include "tsa_host.h"

using namespace tsa;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The gradient's rows: the logits themselves with their own stride, or rows
// apart from them.
int check_grad(const void *logits, const void *grad, int dtype, int64_t B, int64_t V, int64_t stride,
               int64_t gstride) {
    if (!grad) return TSA_OK;
    const size_t es = dtype == TSA_F32 ? 4 : 2;
    if (gstride < V) return TSA_ERR_SHAPE;
    if (!aligned(grad, es)) return TSA_ERR_ALIGN;
    if (grad == logits && gstride != stride) return TSA_ERR_SHAPE;
    (void)B;
    return TSA_OK;
}

}  // namespace

extern "C" {

int tsa_policy_loss(const void *logits, tsa_dtype dtype, int64_t B, int64_t V, int64_t logits_row_stride,
                    const int32_t *bitmask, int64_t mask_row_stride, const float *temperature, float temperature_s,
                    const int64_t *tokens, const float *old_logprob, const float *advantage,
                    const float *ref_logprob, const float *weight, float clip_low, float clip_high, float kl_coef,
                    float entropy_coef, float *loss_out, float *row_loss_out, float *logprob_out,
                    float *entropy_out, void *grad_out, int64_t grad_row_stride, void *stream) {
    int st = rows_check_args(logits, dtype, B, V, logits_row_stride);
    if (st != TSA_OK) return st;
    if (!(clip_low >= 0.f) || !(clip_high >= 0.f) || !isfinite(clip_low) || !isfinite(clip_high) ||
        !isfinite(kl_coef) || !isfinite(entropy_coef))
        return TSA_ERR_VALUE;
    if (B > 0 && (!tokens || !old_logprob || !advantage || !loss_out || !row_loss_out || !logprob_out))
        return TSA_ERR_NULL;
    if (bitmask && mask_row_stride < (V + 31) / 32) return TSA_ERR_STRIDE;
    if (!aligned(bitmask, 4) || !aligned(temperature, 4) || !aligned(tokens, 8) || !aligned(old_logprob, 4) ||
        !aligned(advantage, 4) || !aligned(ref_logprob, 4) || !aligned(weight, 4) || !aligned(loss_out, 4) ||
        !aligned(row_loss_out, 4) || !aligned(logprob_out, 4) || !aligned(entropy_out, 4))
        return TSA_ERR_ALIGN;
    st = check_grad(logits, grad_out, dtype, B, V, logits_row_stride, grad_row_stride);
    if (st != TSA_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (B == 0) {
        if (!loss_out) return TSA_OK;
        return weighted_sum_launch(nullptr, nullptr, 0.f, 0, loss_out, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
    }
    RowLossArgs a = {};
    a.logits = logits;
    a.B = B;
    a.V = V;
    a.stride = logits_row_stride;
    a.mask = bitmask;
    a.mstride = mask_row_stride;
    a.temperature = temperature;
    a.temperature_s = temperature_s;
    a.tokens = tokens;
    a.weight = weight;
    a.weight_s = (float)(1.0 / (double)B);
    a.old_logprob = old_logprob;
    a.advantage = advantage;
    a.ref_logprob = ref_logprob;
    a.clip_lo = 1.f - clip_low;
    a.clip_hi = 1.f + clip_high;
    a.kl = kl_coef;
    a.ent = entropy_coef;
    a.row_loss = row_loss_out;
    a.logprob = logprob_out;
    a.entropy = entropy_out;
    a.grad = grad_out;
    a.gstride = grad_row_stride;
    const bool ent = entropy_out != nullptr || entropy_coef != 0.f;
    if (row_loss_launch(a, dtype, 0, ent, s) != 0) return TSA_ERR_CUDA;
    return weighted_sum_launch(row_loss_out, weight, a.weight_s, B, loss_out, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_preference_loss_workspace_bytes(int64_t N) {
    return N < 1 ? 0 : 3 * align256((size_t)N * sizeof(float));
}

int tsa_preference_loss(const void *logits, tsa_dtype dtype, int64_t N, int64_t V, int64_t logits_row_stride,
                        float temperature, const int64_t *tokens, const int64_t *seq_start, int64_t P,
                        const float *weight, const float *ref_logprob, float beta, float label_smoothing,
                        float margin, int average, float *loss_out, float *pair_loss_out, float *reward_out,
                        float *logprob_out, void *grad_out, int64_t grad_row_stride, void *workspace,
                        size_t workspace_bytes, void *stream) {
    int st = rows_check_args(logits, dtype, N, V, logits_row_stride);
    if (st != TSA_OK) return st;
    if (P < 0 || P > 0x3FFFFFFFll) return TSA_ERR_SHAPE;
    if (!isfinite(beta) || !isfinite(margin) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
        return TSA_ERR_VALUE;
    if (P > 0 && (!seq_start || !loss_out || !pair_loss_out || !reward_out)) return TSA_ERR_NULL;
    if (N > 0 && (!tokens || !logprob_out)) return TSA_ERR_NULL;
    if (!aligned(tokens, 8) || !aligned(seq_start, 8) || !aligned(weight, 4) || !aligned(ref_logprob, 4) ||
        !aligned(loss_out, 4) || !aligned(pair_loss_out, 4) || !aligned(reward_out, 4) || !aligned(logprob_out, 4))
        return TSA_ERR_ALIGN;
    st = check_grad(logits, grad_out, dtype, N, V, logits_row_stride, grad_row_stride);
    if (st != TSA_OK) return st;
    const size_t need = tsa_preference_loss_workspace_bytes(N);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TSA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    }
    const cudaStream_t s = (cudaStream_t)stream;
    const size_t each = need / 3;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    RowLossArgs a = {};
    a.logits = logits;
    a.B = N;
    a.V = V;
    a.stride = logits_row_stride;
    a.temperature_s = temperature;
    a.tokens = tokens;
    a.weight = weight;
    a.weight_s = 1.f;
    a.logprob = logprob_out;
    a.row_m = reinterpret_cast<float *>(ws);
    a.row_z = reinterpret_cast<float *>(ws + each);
    a.coef = reinterpret_cast<float *>(ws + 2 * each);
    if (N > 0 && row_loss_launch(a, dtype, 1, false, s) != 0) return TSA_ERR_CUDA;
    if (P > 0) {
        PairArgs p = {};
        p.P = P;
        p.N = N;
        p.seq_start = seq_start;
        p.logprob = logprob_out;
        p.ref_logprob = ref_logprob;
        p.weight = weight;
        p.beta = beta;
        p.smooth = label_smoothing;
        p.margin = margin;
        p.average = average;
        p.pair_loss = pair_loss_out;
        p.reward = reward_out;
        p.coef = a.coef;
        if (pair_launch(p, a, s) != 0) return TSA_ERR_CUDA;
    }
    if (loss_out && weighted_sum_launch(pair_loss_out, nullptr, P > 0 ? (float)(1.0 / (double)P) : 0.f, P, loss_out,
                                        s) != 0)
        return TSA_ERR_CUDA;
    if (N == 0 || !grad_out) return TSA_OK;
    a.grad = grad_out;
    a.gstride = grad_row_stride;
    return row_grad_launch(a, dtype, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

}  // extern "C"
