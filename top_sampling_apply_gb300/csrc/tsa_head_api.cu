// C-ABI entry points of the calls around the vocabulary head: argument checks,
// workspace layouts and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tsa.h"
#include "tsa_host.h"

using namespace tsa;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int64_t kHeadMaxH = 16384, kInt8MaxRows = 1 << 20;

int check_norm_rows(tsa_dtype dtype, int64_t N, int64_t H, int64_t stride) {
    if (dtype != TSA_F32 && dtype != TSA_F16 && dtype != TSA_BF16) return TSA_ERR_DTYPE;
    if (N < 0 || N > 0x7FFFFFFFll || H < 1 || H > kNormMaxH || stride < H) return TSA_ERR_SHAPE;
    return TSA_OK;
}
int check_norm_weight(const void *weight, tsa_dtype dtype, tsa_dtype weight_dtype) {
    if (weight_dtype != dtype && weight_dtype != TSA_F32) return TSA_ERR_DTYPE;
    if (!weight) return TSA_ERR_NULL;
    return aligned(weight, weight_dtype == TSA_F32 ? 4 : 2) ? TSA_OK : TSA_ERR_ALIGN;
}

// An output may be an input's own rows, or apart from them.
bool same_rows(const void *out, int64_t stride, const void *in, int64_t in_stride) {
    return out != in || !out || stride == in_stride;
}

// The cross entropy's workspace: where each part starts, and its end.
struct XentLayout {
    size_t count, rows, tokens, weight, loss, coef, hidden, part, tok, grad, acc, db, end;
};
XentLayout xent_layout(int64_t M, int64_t H, int64_t V, bool grads, bool bias) {
    const size_t n = (size_t)xent_padded(M);
    const int64_t few = M < kXentPass ? M : kXentPass;
    const size_t piece = (size_t)xent_piece(M, V);
    XentLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t start = at;
        at += align256(bytes);
        return start;
    };
    l.count = take(8);
    l.rows = take(n * 4);
    l.tokens = take(n * 8);
    l.weight = take(n * 4);
    l.loss = take(n * 4);
    l.coef = take(n * 16);
    l.hidden = take(n * (size_t)xent_width(H) * 2);
    l.part = take((size_t)xent_parts(M, V) * (size_t)few * sizeof(float2));
    l.tok = take((size_t)few * 4);
    l.grad = take(grads ? n * piece * 2 : 0);
    const int splits = xent_splits(M, H, V);
    l.acc = take(grads && (piece < (size_t)V || splits > 1) ? (size_t)splits * n * (size_t)H * 4 : 0);
    l.db = take(grads && bias ? n / 32 * piece * 4 : 0);
    l.end = at;
    return l;
}

}  // namespace

extern "C" {

int tsa_rms_norm(const void *x, tsa_dtype dtype, int64_t N, int64_t H, int64_t x_row_stride, const void *weight,
                 tsa_dtype weight_dtype, const void *residual, int64_t residual_row_stride, float eps, int quantize,
                 void *out, int64_t out_row_stride, float *scale_out, void *residual_out,
                 int64_t residual_out_row_stride, float *rstd_out, void *stream) {
    int st = check_norm_rows(dtype, N, H, x_row_stride);
    if (st != TSA_OK) return st;
    if (weight_dtype != dtype && weight_dtype != TSA_F32) return TSA_ERR_DTYPE;
    if (!(eps >= 0.f) || !isfinite(eps)) return TSA_ERR_VALUE;
    if (out_row_stride < H || (residual && residual_row_stride < H) || (residual_out && residual_out_row_stride < H))
        return TSA_ERR_SHAPE;
    if (residual_out && residual_out == out) return TSA_ERR_SHAPE;
    if (quantize ? out && (out == x || out == residual)
                 : !same_rows(out, out_row_stride, x, x_row_stride) ||
                       !same_rows(out, out_row_stride, residual, residual_row_stride))
        return TSA_ERR_SHAPE;
    if (!same_rows(residual_out, residual_out_row_stride, x, x_row_stride) ||
        !same_rows(residual_out, residual_out_row_stride, residual, residual_row_stride))
        return TSA_ERR_SHAPE;
    if (N == 0) return TSA_OK;
    if (!x || !out || (quantize && !scale_out) || (residual_out && !residual)) return TSA_ERR_NULL;
    st = check_norm_weight(weight, dtype, weight_dtype);
    if (st != TSA_OK) return st;
    const size_t es = dtype == TSA_F32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(residual_out, es) || (!quantize && !aligned(out, es)) ||
        !aligned(scale_out, 4) || !aligned(rstd_out, 4))
        return TSA_ERR_ALIGN;
    NormArgs a = {};
    a.x = x;
    a.N = N;
    a.H = H;
    a.xs = x_row_stride;
    a.w = weight;
    a.w_f32 = weight_dtype == TSA_F32;
    a.r = residual;
    a.rs = residual_row_stride;
    a.eps = eps;
    a.out = out;
    a.os = out_row_stride;
    a.scale = scale_out;
    a.res = residual_out;
    a.ress = residual_out_row_stride;
    a.rstd = rstd_out;
    return norm_launch(a, dtype, true, quantize != 0, (cudaStream_t)stream) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

int tsa_quantize_rows(const void *x, tsa_dtype dtype, int64_t N, int64_t H, int64_t x_row_stride, int8_t *out,
                      int64_t out_row_stride, float *scale_out, void *stream) {
    const int st = check_norm_rows(dtype, N, H, x_row_stride);
    if (st != TSA_OK) return st;
    if (out_row_stride < H || (x && x == out)) return TSA_ERR_SHAPE;
    if (N == 0) return TSA_OK;
    if (!x || !out || !scale_out) return TSA_ERR_NULL;
    if (!aligned(x, dtype == TSA_F32 ? 4 : 2) || !aligned(scale_out, 4)) return TSA_ERR_ALIGN;
    NormArgs a = {};
    a.x = x;
    a.N = N;
    a.H = H;
    a.xs = x_row_stride;
    a.out = out;
    a.os = out_row_stride;
    a.scale = scale_out;
    return norm_launch(a, dtype, false, true, (cudaStream_t)stream) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_rms_norm_backward_workspace_bytes(int64_t N, int64_t H) {
    if (N < 1 || H < 1 || H > kNormMaxH) return 0;
    return align256((size_t)norm_back_parts(N, H) * (size_t)H * 4);
}

int tsa_rms_norm_backward(const void *grad, int64_t grad_row_stride, const void *x, tsa_dtype dtype, int64_t N,
                          int64_t H, int64_t x_row_stride, const void *weight, tsa_dtype weight_dtype,
                          const float *rstd, const void *grad_residual, int64_t grad_residual_row_stride,
                          void *grad_x_out, int64_t grad_x_row_stride, void *grad_weight_out, void *workspace,
                          size_t workspace_bytes, void *stream) {
    int st = check_norm_rows(dtype, N, H, x_row_stride);
    if (st != TSA_OK) return st;
    if (grad_row_stride < H || grad_x_row_stride < H || (grad_residual && grad_residual_row_stride < H))
        return TSA_ERR_SHAPE;
    if (!same_rows(grad_x_out, grad_x_row_stride, grad, grad_row_stride) ||
        !same_rows(grad_x_out, grad_x_row_stride, x, x_row_stride) ||
        !same_rows(grad_x_out, grad_x_row_stride, grad_residual, grad_residual_row_stride))
        return TSA_ERR_SHAPE;
    st = check_norm_weight(weight, dtype, weight_dtype);
    if (st != TSA_OK) return st;
    if (!grad_weight_out || (N > 0 && (!grad || !x || !rstd || !grad_x_out))) return TSA_ERR_NULL;
    const size_t es = dtype == TSA_F32 ? 4 : 2;
    if (!aligned(grad, es) || !aligned(x, es) || !aligned(grad_residual, es) || !aligned(grad_x_out, es) ||
        !aligned(rstd, 4) || !aligned(grad_weight_out, weight_dtype == TSA_F32 ? 4 : 2))
        return TSA_ERR_ALIGN;
    const size_t need = tsa_rms_norm_backward_workspace_bytes(N, H);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TSA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    }
    NormBackArgs a = {};
    a.g = grad;
    a.x = x;
    a.N = N;
    a.H = H;
    a.gs = grad_row_stride;
    a.xs = x_row_stride;
    a.w = weight;
    a.w_f32 = weight_dtype == TSA_F32;
    a.rstd = rstd;
    a.gr = grad_residual;
    a.grs = grad_residual_row_stride;
    a.dx = grad_x_out;
    a.dxs = grad_x_row_stride;
    a.dw = grad_weight_out;
    a.part = static_cast<float *>(workspace);
    return norm_back_launch(a, dtype, (cudaStream_t)stream) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_lm_head_int8_workspace_bytes(int64_t M, int64_t H) {
    return M < 1 || M > kInt8MaxRows || H < 1 || H > kHeadMaxH ? 0 : align256((size_t)M * (size_t)int8_padded(H) * 2);
}

int tsa_lm_head_int8(const int8_t *hidden, int64_t M, int64_t H, int64_t hidden_row_stride, const float *hidden_scale,
                     const int8_t *weight, int64_t V, int64_t weight_row_stride, const float *weight_scale,
                     const float *bias, void *out, tsa_dtype out_dtype, int64_t out_row_stride, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (out_dtype != TSA_F32 && out_dtype != TSA_F16 && out_dtype != TSA_BF16) return TSA_ERR_DTYPE;
    if (M < 0 || M > kInt8MaxRows || H < 16 || H > kHeadMaxH || H % 16 != 0 || V < 1 || V > tsa_max_vocab(out_dtype) ||
        hidden_row_stride < H || weight_row_stride < H || out_row_stride < V)
        return TSA_ERR_SHAPE;
    if (M == 0) return TSA_OK;
    if (!hidden || !hidden_scale || !weight || !weight_scale || !out) return TSA_ERR_NULL;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || hidden_row_stride % 16 != 0 || weight_row_stride % 16 != 0 ||
        !aligned(hidden_scale, 4) || !aligned(weight_scale, 4) || !aligned(bias, 4) ||
        !aligned(out, out_dtype == TSA_F32 ? 4 : 2))
        return TSA_ERR_ALIGN;
    if (!workspace || workspace_bytes < tsa_lm_head_int8_workspace_bytes(M, H)) return TSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    Int8Args a = {};
    a.half = static_cast<uint16_t *>(workspace);
    a.hidden = hidden;
    a.M = M;
    a.H = H;
    a.hstride = hidden_row_stride;
    a.weight = weight;
    a.V = V;
    a.wstride = weight_row_stride;
    a.hscale = hidden_scale;
    a.wscale = weight_scale;
    a.bias = bias;
    a.out = out;
    a.ostride = out_row_stride;
    a.dtype = out_dtype;
    return int8_launch(a, (cudaStream_t)stream) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

size_t tsa_lm_head_cross_entropy_workspace_bytes(int64_t M, int64_t H, int64_t V, int grads, int bias) {
    if (M < 1 || M > kXentMaxRows || H < 8 || H > kHeadMaxH || V < 1 || V > tsa_max_vocab(TSA_BF16)) return 0;
    return xent_layout(M, H, V, grads != 0, bias != 0).end;
}

int tsa_lm_head_cross_entropy(const void *hidden, int64_t M, int64_t H, int64_t hidden_row_stride, const void *weight,
                              int64_t V, int64_t weight_row_stride, const float *bias, float softcap,
                              const int64_t *targets, const float *row_weight, float z_loss, float *loss_out,
                              float *row_loss_out, float *lse_out, void *grad_hidden_out,
                              int64_t grad_hidden_row_stride, void *grad_weight_out, int64_t grad_weight_row_stride,
                              float *grad_bias_out, void *workspace, size_t workspace_bytes, void *stream) {
    if (M < 0 || M > kXentMaxRows || H < 8 || H > kHeadMaxH || H % 8 != 0 || V < 1 || V > tsa_max_vocab(TSA_BF16) ||
        hidden_row_stride < H || weight_row_stride < H || (grad_hidden_out && grad_hidden_row_stride < H) ||
        (grad_weight_out && grad_weight_row_stride < H))
        return TSA_ERR_SHAPE;
    // later pieces read what earlier ones would have written
    if ((grad_hidden_out && grad_hidden_out == hidden) || (grad_weight_out && grad_weight_out == weight) ||
        (grad_bias_out && grad_bias_out == bias))
        return TSA_ERR_SHAPE;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !isfinite(z_loss)) return TSA_ERR_VALUE;
    if (!weight || !loss_out || (M > 0 && (!hidden || !targets || !row_loss_out || !lse_out)) ||
        (grad_bias_out && !bias))
        return TSA_ERR_NULL;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || hidden_row_stride % 8 != 0 || weight_row_stride % 8 != 0 ||
        !aligned(bias, 4) || !aligned(targets, 8) || !aligned(row_weight, 4) || !aligned(loss_out, 4) ||
        !aligned(row_loss_out, 4) || !aligned(lse_out, 4) || !aligned(grad_bias_out, 4) ||
        (grad_hidden_out && (!aligned(grad_hidden_out, 16) || grad_hidden_row_stride % 8 != 0)) ||
        (grad_weight_out && (!aligned(grad_weight_out, 16) || grad_weight_row_stride % 8 != 0)))
        return TSA_ERR_ALIGN;
    const bool grads = grad_hidden_out || grad_weight_out || grad_bias_out;
    const XentLayout l = xent_layout(M, H, V, grads, grad_bias_out != nullptr);
    const cudaStream_t s = (cudaStream_t)stream;
    if (M == 0) {
        if (weighted_sum_launch(nullptr, nullptr, 0.f, 0, loss_out, s) != 0) return TSA_ERR_CUDA;
        if (grad_weight_out && cudaMemset2DAsync(grad_weight_out, (size_t)grad_weight_row_stride * 2, 0, (size_t)H * 2,
                                                 (size_t)V, s) != cudaSuccess)
            return TSA_ERR_CUDA;
        if (grad_bias_out && cudaMemsetAsync(grad_bias_out, 0, (size_t)V * 4, s) != cudaSuccess) return TSA_ERR_CUDA;
        return TSA_OK;
    }
    if (!workspace || workspace_bytes < l.end) return TSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TSA_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    XentArgs a = {};
    a.hidden = static_cast<const uint16_t *>(hidden);
    a.M = M;
    a.H = H;
    a.hstride = hidden_row_stride;
    a.weight = static_cast<const uint16_t *>(weight);
    a.V = V;
    a.wstride = weight_row_stride;
    a.bias = bias;
    a.cap = softcap;
    a.z_loss = z_loss;
    a.targets = targets;
    a.row_weight = row_weight;
    a.loss = loss_out;
    a.row_loss = row_loss_out;
    a.lse = lse_out;
    a.dh = static_cast<uint16_t *>(grad_hidden_out);
    a.dhstride = grad_hidden_row_stride;
    a.dw = static_cast<uint16_t *>(grad_weight_out);
    a.dwstride = grad_weight_row_stride;
    a.db = grad_bias_out;
    a.count = reinterpret_cast<int32_t *>(ws + l.count);
    a.scale = reinterpret_cast<float *>(ws + l.count) + 1;
    a.rows = reinterpret_cast<int32_t *>(ws + l.rows);
    a.tokens = reinterpret_cast<int64_t *>(ws + l.tokens);
    a.weight_c = reinterpret_cast<float *>(ws + l.weight);
    a.row_loss_c = reinterpret_cast<float *>(ws + l.loss);
    a.coef = reinterpret_cast<float4 *>(ws + l.coef);
    a.hidden_c = reinterpret_cast<uint16_t *>(ws + l.hidden);
    a.grad = reinterpret_cast<uint16_t *>(ws + l.grad);
    a.acc = reinterpret_cast<float *>(ws + l.acc);
    a.padded = xent_padded(M);
    a.splits = xent_splits(M, H, V);
    a.db_part = reinterpret_cast<float *>(ws + l.db);
    a.part = reinterpret_cast<float2 *>(ws + l.part);
    a.tok = reinterpret_cast<float *>(ws + l.tok);
    return xent_launch(a, s) == 0 ? TSA_OK : TSA_ERR_CUDA;
}

}  // extern "C"
