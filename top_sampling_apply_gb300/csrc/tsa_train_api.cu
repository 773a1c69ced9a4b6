// C-ABI entry points of the training-side calls: argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tsa.h"
#include "tsa_host.h"

#include <new>

using namespace tsa;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The gradient's rows: the logits themselves with their own stride, or rows
// apart from them.
int check_grad(const void *logits, const void *grad, int dtype, int64_t V, int64_t stride, int64_t gstride) {
    if (!grad) return TSA_OK;
    const size_t es = dtype == TSA_F32 ? 4 : 2;
    if (gstride < V) return TSA_ERR_SHAPE;
    if (!aligned(grad, es)) return TSA_ERR_ALIGN;
    if (grad == logits && gstride != stride) return TSA_ERR_SHAPE;
    return TSA_OK;
}

static_assert(sizeof(AdamTensor) == sizeof(tsa_adamw_tensor) && offsetof(AdamTensor, n) == offsetof(tsa_adamw_tensor, n),
              "the C description of a tensor is passed to the kernels as it is");

// The pointers of a list of tensors: present and aligned where n > 0.
int check_tensors(const tsa_adamw_tensor *t, int64_t count, size_t ps, size_t gs, int bits, bool step) {
    if (count < 0 || count > 0x7FFFFFFFll) return TSA_ERR_SHAPE;
    if (count > 0 && !t) return TSA_ERR_NULL;
    for (int64_t i = 0; i < count; ++i) {
        // one random word an element from a 32-bit counter of groups of four
        if (t[i].n < 0 || t[i].n > (1ll << 34)) return TSA_ERR_SHAPE;
        if (t[i].n == 0) continue;
        if ((step && (!t[i].param || !t[i].grad)) || !t[i].exp_avg || !t[i].exp_avg_sq ||
            (bits == 8 && (!t[i].exp_avg_exp || !t[i].exp_avg_sq_exp)))
            return TSA_ERR_NULL;
        if ((step && (!aligned(t[i].param, ps) || !aligned(t[i].grad, gs))) ||
            (bits == 32 && (!aligned(t[i].exp_avg, 4) || !aligned(t[i].exp_avg_sq, 4))))
            return TSA_ERR_ALIGN;
    }
    return TSA_OK;
}

}  // namespace

extern "C" {

size_t tsa_policy_loss_workspace_bytes(int64_t B, int64_t V, tsa_dtype dtype) {
    if (B < 1 || V < 1 || (dtype != TSA_F32 && dtype != TSA_F16 && dtype != TSA_BF16) || row_is_held(V, dtype)) return 0;
    return align256((size_t)B * sizeof(float4));
}

int tsa_policy_loss(const void *logits, tsa_dtype dtype, int64_t B, int64_t V, int64_t logits_row_stride,
                    const int32_t *bitmask, int64_t mask_row_stride, const float *temperature, float temperature_s,
                    const int64_t *tokens, const float *old_logprob, const float *advantage,
                    const float *ref_logprob, const float *weight, float clip_low, float clip_high, float kl_coef,
                    float entropy_coef, float *loss_out, float *row_loss_out, float *logprob_out,
                    float *entropy_out, void *grad_out, int64_t grad_row_stride, void *workspace,
                    size_t workspace_bytes, void *stream) {
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
    st = check_grad(logits, grad_out, dtype, V, logits_row_stride, grad_row_stride);
    if (st != TSA_OK) return st;
    const size_t need = grad_out ? tsa_policy_loss_workspace_bytes(B, V, dtype) : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TSA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    }
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
    const bool ent = entropy_out != nullptr || entropy_coef != 0.f;
    a.gstride = grad_row_stride;
    if (need > 0)
        a.fin = static_cast<float4 *>(workspace);
    else
        a.grad = grad_out;
    if (row_loss_launch(a, dtype, 0, ent, s) != 0) return TSA_ERR_CUDA;
    if (need > 0) {
        a.grad = grad_out;
        if (row_grad_launch(a, dtype, ent, nullptr, 0, nullptr, s) != 0) return TSA_ERR_CUDA;
    }
    return weighted_sum_launch(row_loss_out, weight, a.weight_s, B, loss_out, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_preference_loss_workspace_bytes(int64_t N) {
    return N < 1 ? 0 : align256((size_t)N * sizeof(float4));
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
    if (P > 0 && (!seq_start || !pair_loss_out || !reward_out)) return TSA_ERR_NULL;
    if (N > 0 && (!tokens || !logprob_out)) return TSA_ERR_NULL;
    if ((P > 0 || N > 0) && !loss_out) return TSA_ERR_NULL;
    if (!aligned(tokens, 8) || !aligned(seq_start, 8) || !aligned(weight, 4) || !aligned(ref_logprob, 4) ||
        !aligned(loss_out, 4) || !aligned(pair_loss_out, 4) || !aligned(reward_out, 4) || !aligned(logprob_out, 4))
        return TSA_ERR_ALIGN;
    st = check_grad(logits, grad_out, dtype, V, logits_row_stride, grad_row_stride);
    if (st != TSA_OK) return st;
    const size_t need = tsa_preference_loss_workspace_bytes(N);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TSA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    }
    const cudaStream_t s = (cudaStream_t)stream;
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
    a.fin = static_cast<float4 *>(workspace);
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
        if (pair_launch(p, a, s) != 0) return TSA_ERR_CUDA;
    }
    if (N == 0 || !grad_out) {
        if (!loss_out) return TSA_OK;
        const float each_pair = P > 0 ? (float)(1.0 / (double)P) : 0.f;
        return weighted_sum_launch(pair_loss_out, nullptr, each_pair, P, loss_out, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
    }
    a.grad = grad_out;
    a.gstride = grad_row_stride;
    return row_grad_launch(a, dtype, false, pair_loss_out, P, loss_out, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

int tsa_adamw_step(const tsa_adamw_tensor *tensors, int64_t count, tsa_dtype param_dtype, tsa_dtype grad_dtype,
                   int32_t state_bits, double lr, double beta1, double beta2, double eps, double weight_decay,
                   int64_t step, const float *grad_scale, uint64_t seed, uint64_t offset, void *stream) {
    if ((param_dtype != TSA_F32 && param_dtype != TSA_BF16) ||
        (grad_dtype != TSA_F32 && grad_dtype != TSA_F16 && grad_dtype != TSA_BF16))
        return TSA_ERR_DTYPE;
    if ((state_bits != 8 && state_bits != 32) || step < 1 || !(lr >= 0.0) || !isfinite(lr) || !(eps >= 0.0) ||
        !isfinite(eps) || !(weight_decay >= 0.0) || !isfinite(weight_decay) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0))
        return TSA_ERR_VALUE;
    const int st = check_tensors(tensors, count, param_dtype == TSA_F32 ? 4 : 2, grad_dtype == TSA_F32 ? 4 : 2,
                                 state_bits, true);
    if (st != TSA_OK) return st;
    if (!aligned(grad_scale, 4)) return TSA_ERR_ALIGN;
    if (count == 0) return TSA_OK;
    AdamArgs a = {};
    a.b1 = (float)beta1;
    a.b1c = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.b2c = (float)(1.0 - beta2);
    a.keep = (float)(1.0 - lr * weight_decay);
    a.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    a.rsc2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.scale = grad_scale;
    a.seed = seed;
    a.offset = offset;
    return adamw_launch(reinterpret_cast<const AdamTensor *>(tensors), count, param_dtype, grad_dtype, state_bits, a,
                        (cudaStream_t)stream) == 0
               ? TSA_OK
               : TSA_ERR_CUDA;
}

int tsa_adamw_state_values(const tsa_adamw_tensor *tensors, int64_t count, void *const *exp_avg_out,
                           void *const *exp_avg_sq_out, void *stream) {
    const int st = check_tensors(tensors, count, 1, 1, 8, false);
    if (st != TSA_OK) return st;
    if (count == 0) return TSA_OK;
    if (!exp_avg_out || !exp_avg_sq_out) return TSA_ERR_NULL;
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].n == 0) continue;
        if (!exp_avg_out[i] || !exp_avg_sq_out[i]) return TSA_ERR_NULL;
        if (!aligned(exp_avg_out[i], 2) || !aligned(exp_avg_sq_out[i], 2)) return TSA_ERR_ALIGN;
    }
    AdamTensor *list = new (std::nothrow) AdamTensor[(size_t)count];
    if (!list) return TSA_ERR_CUDA;
    for (int64_t i = 0; i < count; ++i) {
        list[i] = reinterpret_cast<const AdamTensor *>(tensors)[i];
        list[i].param = exp_avg_out[i];
        list[i].grad = exp_avg_sq_out[i];
    }
    const int r = adamw_values_launch(list, count, (cudaStream_t)stream);
    delete[] list;
    return r == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_lm_head_logprob_workspace_bytes(int64_t M, int64_t V) {
    if (M < 1 || V < 1) return 0;
    const int64_t rows = M < kLmRows ? M : kLmRows;
    return align256((size_t)rows * 4) + align256((size_t)lm_logprob_parts(rows, V) * (size_t)rows * sizeof(float2));
}

int tsa_lm_head_logprob(const void *hidden, int64_t M, int64_t H, int64_t hidden_row_stride, const void *weight,
                        int64_t V, int64_t weight_row_stride, const float *bias, float softcap,
                        const int32_t *bitmask, int64_t mask_row_stride, const float *temperature,
                        float temperature_s, const int64_t *tokens, float *out, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (M < 0 || M > 0x7FFFFFFFll || H < 8 || H > 16384 || H % 8 != 0 || V < 1 || V > tsa_max_vocab(TSA_BF16) ||
        hidden_row_stride < H || weight_row_stride < H)
        return TSA_ERR_SHAPE;
    if (!(softcap >= 0.f) || !isfinite(softcap)) return TSA_ERR_VALUE;
    if (M == 0) return TSA_OK;
    if (!hidden || !weight || !tokens || !out) return TSA_ERR_NULL;
    if (bitmask && mask_row_stride < (V + 31) / 32) return TSA_ERR_STRIDE;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || hidden_row_stride % 8 != 0 || weight_row_stride % 8 != 0 ||
        !aligned(bias, 4) || !aligned(bitmask, 4) || !aligned(temperature, 4) || !aligned(tokens, 8) ||
        !aligned(out, 4))
        return TSA_ERR_ALIGN;
    const size_t need = tsa_lm_head_logprob_workspace_bytes(M, V);
    if (!workspace || workspace_bytes < need) return TSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    for (int64_t m = 0; m < M; m += kLmRows) {  // the passes share the workspace, one after another
        LmLogprobArgs a = {};
        a.M = M - m < kLmRows ? M - m : kLmRows;
        a.hidden = static_cast<const uint16_t *>(hidden) + m * hidden_row_stride;
        a.H = H;
        a.hstride = hidden_row_stride;
        a.weight = static_cast<const uint16_t *>(weight);
        a.V = V;
        a.wstride = weight_row_stride;
        a.bias = bias;
        a.cap = softcap;
        a.mask = bitmask ? bitmask + m * mask_row_stride : nullptr;
        a.mstride = mask_row_stride;
        a.temperature = temperature ? temperature + m : nullptr;
        a.temperature_s = temperature_s;
        a.tokens = tokens + m;
        a.out = out + m;
        a.tok = reinterpret_cast<float *>(ws);
        a.part = reinterpret_cast<float2 *>(ws + align256((size_t)(M < kLmRows ? M : kLmRows) * 4));
        if (lm_logprob_launch(a, (cudaStream_t)stream) != 0) return TSA_ERR_CUDA;
    }
    return TSA_OK;
}

}  // extern "C"
