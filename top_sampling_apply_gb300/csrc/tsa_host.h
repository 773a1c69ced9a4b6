// Internal host-side interface between the C-ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tsa {

// Batches of at least this many rows run one CTA per row and need no
// workspace; smaller ones split rows into slices across the whole GPU.
constexpr int64_t kRowKernelMinB = 128;

struct SampleArgs {
    const void *logits;
    int64_t B, V, stride;
    const int32_t *mask;
    int64_t mstride;
    const float *temperature;
    float temperature_s;
    const int32_t *top_k;
    int32_t top_k_s;
    const float *top_p;
    float top_p_s;
    const float *min_p;
    float min_p_s;
    uint64_t seed, offset;
    int64_t *tokens;
    float *vstar_out;
    void *workspace;    // row counters (zero between calls), slice summaries, candidates
    int64_t max_vec;    // vector slots per slice buffer (set by the launcher)
    int64_t max_words;  // mask words per slice buffer (set by the launcher)
    int slices;         // slices per row
    size_t summ_off, cand_off;  // workspace offsets (set by the launcher)
};

struct TopkArgs {
    const void *logits;
    int64_t B, V, stride;
    int32_t k;
    float *values;
    int64_t *indices;
    int64_t max_vec;
};

// Row split: cluster size and vector slots per CTA for a row of V elements of
// `esize` bytes, keeping each CTA's slice within `slice_target` bytes where
// possible and never above `slice_max`.  Returns false if V does not fit.
bool choose_split(int64_t V, int esize, size_t slice_target, size_t slice_max, int *cluster,
                  int64_t *max_vec);

// Sets the kernel's dynamic shared-memory limit (and non-portable cluster
// sizes) once per device; returns 0 or -1.
int prepare_kernel(const void *fn, size_t smem, int cluster);

// The checks every call makes of its rows of logits; TSA_OK or a status.
int rows_check_args(const void *logits, int dtype, int64_t B, int64_t V, int64_t stride);
// The argument checks of tsa_sample (everything but the workspace); returns
// TSA_OK or the status tsa_sample would return.
int sample_check_args(const void *logits, int dtype, int64_t B, int64_t V, int64_t stride, const int32_t *mask,
                      int64_t mstride, const float *temperature, const int32_t *top_k, const float *top_p,
                      const float *min_p, const int64_t *tokens, const float *vstar);

// Sample split: slices per row, vector slots per slice and slice buffers (1 or 2).
bool choose_sample_split(int64_t V, int esize, int *slices, int64_t *max_vec, int *nbuf);
size_t sample_workspace_layout(int64_t B, int S, size_t *summ_off, size_t *cand_off);
size_t sample_smem_bytes(int64_t max_vec, int64_t max_words, int nbuf);
int sample_launch(const SampleArgs &args, int dtype, int slices, int64_t max_vec, int nbuf, cudaStream_t st);
unsigned int *sample_status_ptr();
// One CTA per row (large batches); its own device status word.
int sample_row_launch(const SampleArgs &args, int dtype, cudaStream_t st);
unsigned int *sample_row_status_ptr();
// Specialised row kernels (nullptr for a specialisation not built) and their
// status words, one translation unit per element type.
const void *sample_row_spec_kernel_f32(int spec);
const void *sample_row_spec_kernel_f16(int spec);
const void *sample_row_spec_kernel_bf16(int spec);
unsigned int *sample_row_spec_status_ptr_f32();
unsigned int *sample_row_spec_status_ptr_f16();
unsigned int *sample_row_spec_status_ptr_bf16();
inline const void *sample_row_spec_kernel(int dtype, int spec) {
    return dtype == 0 ? sample_row_spec_kernel_f32(spec)
                      : (dtype == 1 ? sample_row_spec_kernel_f16(spec) : sample_row_spec_kernel_bf16(spec));
}

size_t topk_smem_bytes(int64_t max_vec);
int topk_launch(const TopkArgs &args, int dtype, int cluster, int64_t max_vec, cudaStream_t st);
unsigned int *topk_status_ptr();

// The dense lm-head projection fused with top-k: pass 1 (per 512-entry chunk
// of the vocabulary, its best min(k, 512) as candidates).
struct LmHeadArgs {
    const uint16_t *hidden;  // bf16 [M, hstride]
    int64_t M, H, hstride;
    const uint16_t *weight;  // bf16 [V, wstride]
    int64_t V, wstride;
    const float *bias;       // [V] or NULL
    int32_t k, kk;           // kk = min(k, chunk)
    int64_t nchunks, cand_stride;  // candidates per row = nchunks * kk
    float *cand_vals;
    int32_t *cand_idx;
};
size_t lm_head_smem_bytes(int64_t M, int64_t H);
int64_t lm_head_chunks(int64_t V);
int32_t lm_head_kk(int32_t k);
int lm_head_pass1_launch(const LmHeadArgs &args, cudaStream_t st);
int lm_head_gather_launch(const int64_t *pos, const int32_t *cand_idx, int64_t cand_stride, int64_t M, int32_t k,
                          int64_t *indices_out, cudaStream_t st);

// The inverse-CDF draw over the keep set of a sample call that ran before it
// (its v* per row), and the allow-set packer.
struct IcdfArgs {
    const void *logits;
    int64_t B, V, stride;
    const int32_t *mask;
    int64_t mstride;
    const float *temperature;
    float temperature_s;
    const int32_t *top_k;
    int32_t top_k_s;
    const float *uniform;
    const float *vstar;
    int64_t *tokens;
};
int icdf_launch(const IcdfArgs &args, int dtype, cudaStream_t st);
int pack_launch(const uint8_t *allowed, int64_t B, int64_t V, int64_t astride, int32_t *bits, int64_t wstride,
                cudaStream_t st);

int mask_launch(void *logits, int dtype, int64_t B, int64_t V, int64_t stride, const int32_t *mask,
                int64_t mstride, cudaStream_t st);
// Bitmask (row stride ceil(V / 32)) of the tokens allowed by `mask` whose
// logit is >= floor[b].
int floor_mask_launch(const void *logits, int dtype, int64_t B, int64_t V, int64_t stride, const int32_t *mask,
                      int64_t mstride, const float *floor, int32_t *out, cudaStream_t st);
int logprob_launch(const void *logits, int dtype, int64_t B, int64_t V, int64_t stride, const int32_t *mask,
                   int64_t mstride, const float *temperature, float temperature_s, const int64_t *index,
                   float *out, cudaStream_t st);
// The row losses: policy (mode 0, with or without a gradient) and the sums a
// preference loss needs (mode 1); then the preference loss's pairs and the
// gradient of rows whose sums are known.
struct RowLossArgs {
    const void *logits;
    int64_t B, V, stride;
    const int32_t *mask;
    int64_t mstride;
    const float *temperature;
    float temperature_s;
    const int64_t *tokens;
    const float *weight;
    float weight_s;  // every row's weight when `weight` is NULL
    const float *old_logprob, *advantage, *ref_logprob;
    float clip_lo, clip_hi, kl, ent;  // the ratio's bounds, the KL and entropy coefficients
    float *row_loss, *logprob, *entropy;
    void *grad;
    int64_t gstride;
    // a row between two passes, or NULL: k1, k2, a and m of its gradient; from
    // mode 1's sums 0, Z, 0 and m
    float4 *fin;
};
struct PairArgs {
    int64_t P, N;
    const int64_t *seq_start;
    const float *logprob, *ref_logprob, *weight;
    float beta, smooth, margin;
    int average;
    float *pair_loss, *reward;
};
// Whether rows of V logits are held on chip for their gradient; longer ones
// take two passes (sums, then row_grad_launch) with `fin` between them.
bool row_is_held(int64_t V, int dtype);
int row_loss_launch(const RowLossArgs &args, int dtype, int mode, bool ent, cudaStream_t st);
unsigned int *row_loss_status_ptr();
// The gradient of rows whose coefficients are known, and the pairs' mean loss
// (loss NULL: none).
int row_grad_launch(const RowLossArgs &args, int dtype, bool ent, const float *pair_loss, int64_t pairs, float *loss,
                    cudaStream_t st);
int pair_launch(const PairArgs &args, const RowLossArgs &rows, cudaStream_t st);
// out[0] = sum_i w_i x_i over the entries with w_i != 0 (w NULL: w_s each).
int weighted_sum_launch(const float *x, const float *w, float w_s, int64_t n, float *out, cudaStream_t st);
// The kernels of one element type.
const void *row_loss_kernel_f32(int mode, bool ent);
const void *row_loss_kernel_f16(int mode, bool ent);
const void *row_loss_kernel_bf16(int mode, bool ent);
const void *row_held_kernel_f32(bool ent, int threads);
const void *row_held_kernel_f16(bool ent, int threads);
const void *row_held_kernel_bf16(bool ent, int threads);
const void *row_grad_kernel_f32(bool ent);
const void *row_grad_kernel_f16(bool ent);
const void *row_grad_kernel_bf16(bool ent);

// AdamW over many tensors: one tensor's pointers, and the step's numbers.
struct AdamTensor {
    void *param;
    const void *grad;
    void *m, *v;
    uint8_t *me, *ve;
    int64_t n;
};
struct AdamArgs {
    float b1, b1c, b2, b2c;        // the two decay rates and one less each
    float keep, rate, rsc2, eps;   // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t), eps
    const float *scale;
    uint64_t seed, offset;
    uint32_t first;                // list index of the launch's first tensor (its random row)
};
int adamw_launch(const AdamTensor *tensors, int64_t count, int param_dtype, int grad_dtype, int bits,
                 const AdamArgs &args, cudaStream_t st);
// param, grad: the bf16 outputs of m and v
int adamw_values_launch(const AdamTensor *tensors, int64_t count, cudaStream_t st);

// The log-probability of a token from the hidden rows.
struct LmLogprobArgs {
    const uint16_t *hidden;  // bf16 [M, hstride]
    int64_t M, H, hstride;
    const uint16_t *weight;  // bf16 [V, wstride]
    int64_t V, wstride;
    const float *bias;       // [V] or NULL
    float cap;               // 0: none
    const int32_t *mask;
    int64_t mstride;
    const float *temperature;
    float temperature_s;
    const int64_t *tokens;
    float *out;
    float2 *part;            // [parts][rows]: a part's largest score and its sum against it
    float *tok;              // [rows]: the token's score
};
constexpr int64_t kLmRows = 8192;  // rows a pass over the weight takes
int64_t lm_logprob_parts(int64_t M, int64_t V);
int lm_logprob_launch(const LmLogprobArgs &args, cudaStream_t st);
unsigned int *lm_logprob_status_ptr();

// The root-mean-square norm of rows with the residual's addition, and rows in
// 8 bits; its backward pass.
constexpr int64_t kNormMaxH = 16384;
struct NormArgs {
    const void *x;  // [N, xs]
    int64_t N, H, xs;
    const void *w;  // [H], of the rows' type or fp32
    bool w_f32;
    const void *r;  // [N, rs] or NULL
    int64_t rs;
    float eps;
    void *out;      // [N, os] of the rows' type, or int8
    int64_t os;
    float *scale;   // [N], 8-bit rows only
    void *res;      // [N, ress] or NULL: the sum
    int64_t ress;
    float *rstd;    // [N] or NULL
};
// norm false: the rows themselves in 8 bits (w, r, eps, res and rstd not used).
int norm_launch(const NormArgs &args, int dtype, bool norm, bool q, cudaStream_t st);
struct NormBackArgs {
    const void *g, *x;
    int64_t N, H, gs, xs;
    const void *w;
    bool w_f32;
    const float *rstd;
    const void *gr;  // [N, grs] or NULL
    int64_t grs;
    void *dx;
    int64_t dxs;
    void *dw;        // [H] of the weight's type
    float *part;     // [norm_back_parts][H]
};
unsigned int *norm_status_ptr();
int64_t norm_back_parts(int64_t N, int64_t H);
int norm_back_launch(const NormBackArgs &args, int dtype, cudaStream_t st);

// Scores from 8-bit integers.
struct Int8Args {
    const int8_t *hidden;  // [M, hstride]
    int64_t M, H, hstride;
    const int8_t *weight;  // [V, wstride]
    int64_t V, wstride;
    const float *hscale, *wscale, *bias;
    void *out;             // [M, ostride] of dtype
    int64_t ostride;
    int dtype;
    uint16_t *half;        // workspace: [M, int8_padded(H)], the hidden rows in f16
};
constexpr int kInt8Stage = 128;
__host__ __device__ inline int64_t int8_padded(int64_t H) { return (H + kInt8Stage - 1) / kInt8Stage * kInt8Stage; }
unsigned int *int8_status_ptr();
int int8_launch(const Int8Args &args, cudaStream_t st);

// The cross entropy from the hidden rows, with its gradients.
struct XentArgs {
    const uint16_t *hidden;  // bf16 [M, hstride]
    int64_t M, H, hstride;
    const uint16_t *weight;  // bf16 [V, wstride]
    int64_t V, wstride;
    const float *bias;
    float cap, z_loss;
    const int64_t *targets;
    const float *row_weight;
    float *loss, *row_loss, *lse;
    uint16_t *dh, *dw;       // bf16 [M, dhstride], [V, dwstride], or NULL
    int64_t dhstride, dwstride;
    float *db;               // [V] or NULL
    // workspace; "c": of the rows that count, one after another
    float *scale;            // [1]: the largest row weight, which G is without
    int32_t *count, *rows;   // [1]; [M]: a place's row
    int64_t *tokens;
    float *weight_c, *row_loss_c;
    float2 *part;            // of a pass's rows: a part's largest score and its sum against it
    float *tok;              // of a pass's rows: the target's score
    float4 *coef;            // what a place's gradient needs, and 1 if it has a row
    uint16_t *hidden_c;      // [padded, xent_width(H)]
    uint16_t *grad;          // [padded, piece]: a piece of the vocabulary's part of G
    float *acc;              // [splits][padded, H]: dH so far
    int64_t padded;
    int splits;
    float *db_part;
};
__host__ __device__ inline int64_t xent_padded(int64_t M) { return M < 1 ? 128 : (M + 127) / 128 * 128; }
__host__ __device__ inline int64_t xent_width(int64_t H) { return (H + 63) / 64 * 64; }
constexpr int64_t kXentMaxRows = 1 << 16, kXentMaxPiece = 1 << 16;
int64_t xent_piece(int64_t M, int64_t V);
int xent_splits(int64_t M, int64_t H, int64_t V);
unsigned int *xent_status_ptr();
constexpr int64_t kXentPass = 8192;  // rows of a first pass over the scores
inline int64_t xent_parts(int64_t M, int64_t V) { return M <= 128 ? (V + 63) / 64 : (V + 127) / 128; }
int xent_launch(const XentArgs &args, cudaStream_t st);

int selftest_launch(uint32_t limit_us, cudaStream_t st);

}  // namespace tsa
