/*
 * tsa.h -- per-row vocabulary selection on NVIDIA GB300 (sm_103a).
 *
 * The step between a model's logits and its next token: a packed grammar
 * mask, a fused temperature + top-k / top-p / min-p filter with a Gumbel-max
 * draw, and an exact sorted top-k.  Plain C ABI: device pointers, sizes and a
 * CUDA stream passed as void*; no framework types.
 *
 * Conventions shared by every call
 *   - Pointers named logits / bitmask / workspace / *_out and per-row
 *     parameter arrays are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory and keeps no state between calls.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the call returns without synchronising.
 *   - Rows are row-major: element (b, i) of logits is at
 *     logits + (b * logits_row_stride + i) * element_size.  Row starts need
 *     only element alignment; 16-byte aligned rows take the fastest path.
 *   - Arguments are validated before anything is enqueued.  A negative
 *     return value means nothing was launched (TSA_ERR_CUDA: the launch itself
 *     failed).  B == 0 is a valid no-op.
 *   - The bitmask layout is [B, mask_row_stride] int32 with
 *     mask_row_stride >= ceil(V / 32); token i is allowed iff bit (i & 31) of
 *     word (i >> 5) is 1 (least significant bit first).  Bits at or beyond V
 *     are ignored.
 *   - Device-side faults of the library's own making (a bounded wait that ran
 *     out) never hang the GPU: the kernel records a flag, finishes, and
 *     tsa_device_status() reports it.
 */
#ifndef TSA_H
#define TSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { TSA_F32 = 0, TSA_F16 = 1, TSA_BF16 = 2 } tsa_dtype;

enum {
    TSA_OK = 0,
    TSA_ERR_NULL = -1,           /* a required pointer is NULL */
    TSA_ERR_SHAPE = -2,          /* a size or a row stride is out of its range: B < 0, V < 1, V too large,
                                    row stride < V, H not a multiple of 8 */
    TSA_ERR_DTYPE = -3,          /* dtype not one of tsa_dtype */
    TSA_ERR_K_RANGE = -4,        /* topk: k < 1, k > 2048 or k > V */
    TSA_ERR_STRIDE = -5,         /* mask_row_stride < ceil(V / 32) */
    TSA_ERR_WORKSPACE = -6,      /* sample: workspace NULL or smaller than required */
    TSA_ERR_CUDA = -7,           /* a CUDA runtime call failed (launch / attribute) */
    TSA_ERR_DEVICE_TIMEOUT = -8, /* a kernel's bounded wait ran out (see tsa_device_status) */
    TSA_ERR_ALIGN = -9,          /* a pointer is not aligned to its element size */
    TSA_ERR_VALUE = -10          /* a scalar parameter is out of its range or not finite */
};

/* Largest vocabulary a row may have, per element type (elements). */
int64_t tsa_max_vocab(tsa_dtype dtype);

/*
 * apply_token_bitmask -- logits-processor, "API" (apply_token_bitmask) and
 * "Correctness": set to -inf, in place, exactly the logits whose mask bit is
 * 0; allowed logits are left bit-identical; V need not be a multiple of 32.
 *   logits   [B, logits_row_stride] of dtype, read and written in place
 *   bitmask  [B, mask_row_stride] int32, read only
 * Returns TSA_OK or a negative status.
 */
int tsa_apply_token_bitmask(void *logits, tsa_dtype dtype, int64_t B, int64_t V,
                            int64_t logits_row_stride, const int32_t *bitmask,
                            int64_t mask_row_stride, void *stream);

/*
 * sample -- logits-processor, "API" (sample) and "Method": one token per row.
 * Temperature scaling, then the intersection of the top-k, top-p and min-p
 * keep sets, which is one keep-threshold v* on the logit (the kept set is
 * every allowed token with logit >= v*), then a Gumbel-max draw over the kept
 * set: token = argmax_i (l_i / T + G_i), ties to the lower index, where G_i is
 * the standard Gumbel variate of the i-th token's Philox4x32-10 word under key
 * (seed lo, seed hi) and counter (i >> 2, row, offset lo, offset hi).
 * logits-mask-xpu, "Method": top_k == 1 returns the argmax.
 *   logits       [B, logits_row_stride] of dtype, read only
 *   bitmask      [B, mask_row_stride] int32 or NULL; a disallowed token is
 *                treated as -inf (the logits are not modified)
 *   temperature  [B] float or NULL to use temperature_s for every row;
 *                T <= 0 is greedy (argmax, lowest index on ties)
 *   top_k        [B] int32 or NULL (top_k_s); k <= 0 disables, k == 1 argmax,
 *                k >= number of allowed tokens keeps all; ties at the k-th
 *                value are all kept
 *   top_p        [B] float or NULL (top_p_s); p >= 1 disables; keeps every
 *                token whose probability mass strictly above it is < p; the
 *                argmax class is always kept
 *   min_p        [B] float or NULL (min_p_s); <= 0 disables; keeps tokens with
 *                probability >= min_p times the largest probability
 *   seed, offset the draw key; advance offset every decoding step
 *   tokens_out   [B] int64: the token, or -1 for a row with no allowed finite
 *                logit
 *   min_kept_logit_out  [B] float or NULL: v* (the argmax value for greedy
 *                rows, -inf when no filter is active, NaN for an empty row)
 *   workspace    device scratch of at least tsa_sample_workspace_bytes(B, V,
 *                dtype) bytes, 256-byte aligned, no initialisation needed, or
 *                NULL when that size is 0 (batches of 128 rows or more: one
 *                CTA holds each row's state on chip).  Smaller batches split
 *                rows across the GPU; the workspace then holds per-slice
 *                summaries and candidate lists, all written by the call before
 *                it reads them.  Calls that may run concurrently must use
 *                different workspaces.  TSA_ERR_WORKSPACE if a size > 0 is
 *                needed and the workspace is NULL or too small.
 * NaN logits are treated as -inf.  Rows with identical arguments give
 * bit-identical tokens on every call.
 */
int tsa_sample(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
               int64_t logits_row_stride, const int32_t *bitmask, int64_t mask_row_stride,
               const float *temperature, float temperature_s, const int32_t *top_k,
               int32_t top_k_s, const float *top_p, float top_p_s, const float *min_p,
               float min_p_s, uint64_t seed, uint64_t offset, int64_t *tokens_out,
               float *min_kept_logit_out, void *workspace, size_t workspace_bytes,
               void *stream);
/* Workspace bytes `sample` needs for B rows of V elements: 0 when B >= 128
 * (every row is resolved on chip by one CTA), and 0 for invalid sizes. */
size_t tsa_sample_workspace_bytes(int64_t B, int64_t V, tsa_dtype dtype);

/*
 * lm_head_topk -- lm-head-topk, "API", "Method" and "Correctness" (the dense
 * head): the exact top-k of scores = hidden . weight^T (+ bias) per hidden
 * row, without writing the [M, V] score matrix.  One CTA per 512-entry chunk
 * of the vocabulary computes its scores (fp32 accumulation of bf16 products)
 * and keeps its best min(k, 512); the exact top-k of those candidates follows
 * (tsa_topk), and their positions are mapped back to vocabulary indices.
 * Values are sorted descending, ties to the lower vocabulary index.  The
 * weight is read once per call; every hidden row is scored in that one read.
 *   hidden       bf16 [M, hidden_row_stride], 1 <= M <= 4 (M == 0: no-op)
 *   weight       bf16 [V, weight_row_stride]; H a multiple of 8, 8 <= H <=
 *                8192; both row strides multiples of 8 elements and both
 *                bases 16-byte aligned (TSA_ERR_ALIGN)
 *   bias         float [V] or NULL
 *   k            1 <= k <= min(2048, V) (TSA_ERR_K_RANGE)
 *   values_out   float [M, k]; indices_out int64 [M, k]
 *   workspace    at least tsa_lm_head_topk_workspace_bytes(M, V, k) bytes,
 *                256-byte aligned (the chunks' candidates)
 */
int tsa_lm_head_topk(const void *hidden, int64_t M, int64_t H, int64_t hidden_row_stride,
                     const void *weight, int64_t V, int64_t weight_row_stride, const float *bias,
                     int32_t k, float *values_out, int64_t *indices_out, void *workspace,
                     size_t workspace_bytes, void *stream);
size_t tsa_lm_head_topk_workspace_bytes(int64_t M, int64_t V, int32_t k);

/*
 * sample_sequential -- tsa_sample with top-p taken over the softmax
 * renormalised over the top-k survivors, the reading of the transformers
 * processor chain that logits-processor names as its reference (top-k, then
 * top-p, then min-p, each on what the one before kept), instead of the
 * intersection on the full softmax.  Without top-k (or top-p) the two
 * readings agree.  Three steps on `stream`: tsa_sample with top-p and min-p
 * off gives the top-k cut v_k per row; a bitmask of the tokens the caller's
 * mask allows with logit >= v_k; tsa_sample over that mask with every filter.
 * The draw is keyed as in tsa_sample (same seed and offset, same Philox word
 * per token), so a row whose keep set is the same gets the same token.
 *   arguments as tsa_sample, except
 *   workspace   at least tsa_sample_sequential_workspace_bytes(B, V, dtype)
 *               bytes, 256-byte aligned (never NULL for B >= 1: it holds the
 *               survivors' bitmask and v_k)
 */
int tsa_sample_sequential(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
                          int64_t logits_row_stride, const int32_t *bitmask,
                          int64_t mask_row_stride, const float *temperature, float temperature_s,
                          const int32_t *top_k, int32_t top_k_s, const float *top_p,
                          float top_p_s, const float *min_p, float min_p_s, uint64_t seed,
                          uint64_t offset, int64_t *tokens_out, float *min_kept_logit_out,
                          void *workspace, size_t workspace_bytes, void *stream);
/* Workspace bytes sample_sequential needs: B ceil(V / 32) words of bitmask and
 * B floats (each rounded up to 256 bytes) plus tsa_sample's workspace; 0 for
 * invalid sizes. */
size_t tsa_sample_sequential_workspace_bytes(int64_t B, int64_t V, tsa_dtype dtype);

/*
 * sample_icdf -- logits-mask-xpu, "Usage" (pass uniform [B] for deterministic
 * draws) and "Method" (the cooperative inverse-CDF draw).  The keep set is
 * tsa_sample's: every allowed finite logit >= v*.  With weights
 * w_i = exp((l_i - m) / T) over it, walked in token-index order with running
 * sums S_i, the token is the first kept one with S_i > u W, W the kept total
 * (the last kept token if rounding leaves u W unpassed).  Each row takes one
 * CTA: one read forms the masses of eight contiguous chunks, a scan over them
 * finds the chunk holding u W, and only that chunk is walked again.  Greedy
 * rows (T <= 0 or top_k == 1) give the argmax and empty rows -1, as
 * tsa_sample does.  The sums run in compensated fp32, so a token whose
 * boundary S_i lies within about 1e-6 W of u W may differ from an exact
 * (double precision) walk.
 *   uniform             [B] float in [0, 1), read only; u outside it gives
 *                       the first (u < 0) or last (u >= 1) kept token
 *   min_kept_logit_out  [B] float, REQUIRED here: v* per row, written by the
 *                       selection and read by the draw
 *   every other argument as tsa_sample (the same workspace size; no seed)
 * The call enqueues tsa_sample's kernels and then the draw's kernel.
 */
int tsa_sample_icdf(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
                    int64_t logits_row_stride, const int32_t *bitmask, int64_t mask_row_stride,
                    const float *temperature, float temperature_s, const int32_t *top_k,
                    int32_t top_k_s, const float *top_p, float top_p_s, const float *min_p,
                    float min_p_s, const float *uniform, int64_t *tokens_out,
                    float *min_kept_logit_out, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * bitmask_from_allowed -- logits-mask-xpu, "Usage": pack a [B, V] bool
 * allow-set, one byte per token (nonzero = allowed), into the bitmask layout
 * every call here reads: token i is bit (i & 31) of word (i >> 5); the bits
 * of the last word past V are written 0.
 *   allowed      [B, allowed_row_stride] uint8, read only
 *   bitmask_out  [B, mask_row_stride] int32, words 0 .. ceil(V / 32) - 1 of
 *                each row written
 * Returns TSA_OK or a negative status (TSA_ERR_SHAPE, TSA_ERR_NULL,
 * TSA_ERR_STRIDE, TSA_ERR_ALIGN, TSA_ERR_CUDA).
 */
int tsa_bitmask_from_allowed(const uint8_t *allowed, int64_t B, int64_t V,
                             int64_t allowed_row_stride, int32_t *bitmask_out,
                             int64_t mask_row_stride, void *stream);

/*
 * sample_noalloc -- tsa_sample without a caller workspace.  The papers this
 * library follows have no counterpart: it exists for callers that cannot
 * allocate device memory when they sample (fixed, fully handed-out memory
 * pools; hosts that expose only the tensors they pass in; paths where an
 * allocation could synchronise the device or fail).  Arguments, results and
 * errors are those of tsa_sample, minus workspace / workspace_bytes.
 *   - Scratch is a fixed device array of TSA_SAMPLE_NOALLOC_SCRATCH_BYTES
 *     inside the library, held on every GPU where the library's module is
 *     loaded until the process exits.  The call itself allocates nothing.
 *   - The arguments are checked first, exactly as tsa_sample checks them.
 *     Then, when tsa_sample_workspace_bytes(B, V, dtype) exceeds
 *     TSA_SAMPLE_NOALLOC_SCRATCH_BYTES, the call returns TSA_ERR_WORKSPACE
 *     and launches nothing.  Only batches under 128 rows use the scratch;
 *     127 rows fit vocabularies up to about 265,000 fp32 or 530,000 bf16 /
 *     f16 entries, and 64 rows of an 800,000-entry fp32 vocabulary are
 *     refused.
 *   - A call on a stream that is not capturing looks up the array's device
 *     address on the current device (the first lookup may load the library's
 *     module there); a call on a capturing stream reuses the address that the
 *     last call outside capture found, so make the first call on each device
 *     outside any stream capture.
 *   - All calls on a device share the one array.  Calls that overlap on the
 *     GPU (different streams or threads without ordering between them) race
 *     and give wrong tokens; calls ordered on one stream are safe.  The array
 *     keeps the last call's contents, and nothing in it needs to start at
 *     zero.
 */
#define TSA_SAMPLE_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)
int tsa_sample_noalloc(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
                       int64_t logits_row_stride, const int32_t *bitmask, int64_t mask_row_stride,
                       const float *temperature, float temperature_s, const int32_t *top_k,
                       int32_t top_k_s, const float *top_p, float top_p_s, const float *min_p,
                       float min_p_s, uint64_t seed, uint64_t offset, int64_t *tokens_out,
                       float *min_kept_logit_out, void *stream);

/*
 * topk -- lm-head-topk, "API" and "Method": the exact k largest logits of
 * every row, sorted by value descending with ties resolved to the lower
 * vocabulary index (the order of torch.topk on the materialised row).
 *   logits       [B, logits_row_stride] of dtype, read only
 *   k            1 <= k <= min(2048, V)
 *   values_out   [B, k] float: exact copies of the selected logits
 *   indices_out  [B, k] int64
 *   workspace    reserved; pass NULL / 0 (tsa_topk_workspace_bytes is 0)
 * -0.0 and +0.0 compare equal (the index decides); NaN ranks above +inf.
 */
int tsa_topk(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
             int64_t logits_row_stride, int32_t k, float *values_out, int64_t *indices_out,
             void *workspace, size_t workspace_bytes, void *stream);
size_t tsa_topk_workspace_bytes(int64_t B, int64_t V, int32_t k, tsa_dtype dtype);

/*
 * selective_log_softmax ("Selective Log Softmax": one log-probability per
 * row, the row's logit at a given index less the row's log-sum-exp), over the
 * allowed tokens of the temperature-scaled row:
 *   out[b] = (l[b, i_b] - m_b) / T_b - ln sum_{j allowed} exp((l[b, j] - m_b) / T_b),
 *   m_b the row's largest allowed logit.  Called with sample's tokens, it gives
 *   the log-probability of each sampled token before top-k / top-p / min-p.
 *   logits, dtype, B, V, logits_row_stride, bitmask, mask_row_stride,
 *   temperature, temperature_s: as for tsa_sample (device pointers; bitmask and
 *                temperature may be NULL); T <= 0 uses T = 1, the page's
 *                unscaled definition.
 *   index        [B] int64 device pointer, read only.
 *   out          [B] float device pointer: -inf for a disallowed index; NaN
 *                for an index outside [0, V) or a row with no allowed finite
 *                logit.  NaN logits count as -inf; +inf logits give NaN.
 * Reads each row once from HBM.  Errors as for tsa_apply_token_bitmask;
 * TSA_ERR_NULL when index or out is NULL (B > 0); TSA_ERR_ALIGN for a
 * misaligned index (8 bytes) or out / temperature (4 bytes).
 */
int tsa_selective_log_softmax(const void *logits, tsa_dtype dtype, int64_t B, int64_t V,
                              int64_t logits_row_stride, const int32_t *bitmask, int64_t mask_row_stride,
                              const float *temperature, float temperature_s, const int64_t *index,
                              float *out, void *stream);

/*
 * policy_loss -- the clipped policy loss of sampled tokens with a KL term and
 * an entropy bonus, and its gradient on the logits, in one call.  The rows and
 * tokens are those of sample and selective_log_softmax.  With x = l / T over a
 * row's allowed tokens, p = softmax(x), lp = ln p[token], H = -sum p ln p and
 * r = exp(lp - old):
 *   row_loss = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *              + kl_coef (exp(ref - lp) - (ref - lp) - 1) - entropy_coef H
 *   loss     = sum over rows of weight * row_loss
 *   grad     = d loss / d logits: weight / T (c (1{j = token} - p_j)
 *              + entropy_coef p_j (ln p_j + H)), c the derivative of the first
 *              two terms by lp (-A r where the unclipped branch is taken).
 *   logits, dtype, B, V, logits_row_stride, bitmask, mask_row_stride,
 *   temperature, temperature_s: as for selective_log_softmax
 *   tokens       [B] int64; a token outside [0, V) (sample's -1 for a row
 *                with nothing allowed) skips its row
 *   old_logprob, advantage  [B] float; an advantage of 0 contributes 0 even
 *                where the ratio overflows
 *   ref_logprob  [B] float or NULL: no KL term (nor with kl_coef 0, whatever it holds)
 *   weight       [B] float or NULL: 1 / B for every row; 0 skips a row
 *   clip_low, clip_high >= 0, kl_coef, entropy_coef: finite (TSA_ERR_VALUE)
 *   loss_out     [1] float (0 for B == 0); row_loss_out, logprob_out [B] float
 *   entropy_out  [B] float or NULL
 *   grad_out     [B, grad_row_stride] of dtype, or NULL for the loss alone; it
 *                may be `logits` itself (same row stride), and otherwise must
 *                not overlap it.  Fastest where its rows start at the same
 *                address modulo 16 bytes as the logits' rows.
 *   workspace    at least tsa_policy_loss_workspace_bytes(B, V, dtype) bytes,
 *                256-byte aligned, or NULL where that is 0 (rows of up to 512
 *                KB) or grad_out is NULL
 * f16 gradients of less than 2^-25 become 0, as 1/4096 of a probability of 1e-4
 * does: larger weights carry a loss scale, which adamw_step's grad_scale takes out.
 * A skipped row's logits are not read; its loss, log-probability, entropy and
 * gradient are 0.  A row whose token the mask excludes, or whose mask leaves
 * nothing, also has loss and gradient 0; its logprob_out is -inf, or NaN for
 * the empty row.  NaN logits count as -inf; a +inf logit makes its row NaN.
 * Rows of up to 512 KB are read from HBM once; longer ones twice if there is a
 * gradient.  The sums run in fp32 and the loss over rows in a fixed order:
 * equal calls give equal bits.
 */
int tsa_policy_loss(const void *logits, tsa_dtype dtype, int64_t B, int64_t V, int64_t logits_row_stride,
                    const int32_t *bitmask, int64_t mask_row_stride, const float *temperature,
                    float temperature_s, const int64_t *tokens, const float *old_logprob,
                    const float *advantage, const float *ref_logprob, const float *weight, float clip_low,
                    float clip_high, float kl_coef, float entropy_coef, float *loss_out,
                    float *row_loss_out, float *logprob_out, float *entropy_out, void *grad_out,
                    int64_t grad_row_stride, void *workspace, size_t workspace_bytes, void *stream);
size_t tsa_policy_loss_workspace_bytes(int64_t B, int64_t V, tsa_dtype dtype);

/*
 * preference_loss -- the loss of preferred over rejected answers from their
 * paired log-ratios, and its gradient on the logits.  The N rows of logits are
 * the tokens of 2 P sequences one after another: sequence s is rows
 * seq_start[s] .. seq_start[s + 1] - 1, pair p is sequence p (preferred) and
 * sequence P + p (rejected).  With lp_i row i's log-probability of its token,
 *   R_s  = sum_{i in s} weight_i (lp_i - ref_i)   (average: divided by
 *          sum_{i in s} weight_i; 0 for a sequence without counted rows)
 *   h_p  = beta (R_p - R_{P+p}) - margin
 *   pair_loss_p = (1 - label_smoothing) ln(1 + e^-h) + label_smoothing ln(1 + e^h)
 *   loss = mean of the pair losses,  reward_s = beta R_s
 *   grad = d loss / d logits
 *   logits, dtype, N, V, logits_row_stride, tokens: rows as above; temperature
 *                one value for every row (<= 0: 1)
 *   seq_start    [2 P + 1] int64 device pointer, not decreasing, within
 *                [0, N]; rows outside every sequence get gradient 0, and
 *                values out of range are brought into it
 *   weight       [N] float or NULL (1): 0 skips a row (prompt or padding)
 *   ref_logprob  [N] float or NULL (reference-free); -inf, for a token that the
 *                reference excludes, gives the infinite R and loss of the formula
 *                and the gradient of the logistic's end
 *   0 <= label_smoothing <= 1, beta and margin finite (TSA_ERR_VALUE)
 *   loss_out     [1] float; pair_loss_out [P], reward_out [2 P], logprob_out
 *                [N] float
 *   grad_out     as for policy_loss
 *   workspace    at least tsa_preference_loss_workspace_bytes(N) bytes,
 *                256-byte aligned
 * Skipped and excluded rows as in policy_loss.  A row's coefficient needs
 * every row of its pair, so the logits are read twice, the second time from
 * the row last read back to the first.
 */
int tsa_preference_loss(const void *logits, tsa_dtype dtype, int64_t N, int64_t V, int64_t logits_row_stride,
                        float temperature, const int64_t *tokens, const int64_t *seq_start, int64_t P,
                        const float *weight, const float *ref_logprob, float beta, float label_smoothing,
                        float margin, int average, float *loss_out, float *pair_loss_out, float *reward_out,
                        float *logprob_out, void *grad_out, int64_t grad_row_stride, void *workspace,
                        size_t workspace_bytes, void *stream);
size_t tsa_preference_loss_workspace_bytes(int64_t N);

/*
 * adamw_step -- one AdamW step over many tensors in one call, with 32-bit or
 * 8-bit states.  For every element, with g the gradient times *grad_scale:
 *   m' = beta1 m + (1 - beta1) g
 *   v' = beta2 v + (1 - beta2) g^2
 *   p' = p (1 - lr weight_decay)
 *        - lr / (1 - beta1^step) m' / (sqrt(v' / (1 - beta2^step)) + eps)
 * computed in fp32 from the unrounded m' and v', denormal ones included; m' = v'
 * = 0 with eps = 0 is an update of 0.
 *   tensors      HOST array of `count` descriptions, read during the call; its
 *                pointers are device pointers to contiguous elements, aligned
 *                to their element size (16-byte aligned ones take the fastest
 *                path); n may be 0 and may pass 2^32.  No two may overlap.
 *   param_dtype  TSA_F32 or TSA_BF16; grad_dtype any tsa_dtype
 *   state_bits   32: exp_avg, exp_avg_sq are float [n]; the *_exp pointers are
 *                not used.  8: they are uint8 [n], and exp_avg_exp,
 *                exp_avg_sq_exp uint8 [ceil(n / 256)] (all 0 for a new state).
 *   lr, eps, weight_decay >= 0; 0 <= beta1, beta2 < 1; step >= 1 counts from 1
 *                (TSA_ERR_VALUE)
 *   grad_scale   device pointer to one float, or NULL for 1: the clipping or
 *                inverse loss scale.  If it is not finite, the step changes
 *                nothing.
 *   seed, offset the key of the random words used in rounding; advance offset
 *                every step.  sample's words come from the same function: give one of
 *                the two another seed
 * bf16 parameters are rounded stochastically: an update far below half a step
 * of the parameter still moves it in the mean.
 * An 8-bit state holds blocks of 256 elements, each with one exponent b (the
 * *_exp byte: the largest biased exponent in the block less 30 for exp_avg_sq
 * and less 14 for exp_avg, at least 0).  A code c != 0 stands for the float
 * with bits (c + 8 b) << 20, eight steps an octave: c is 1 to 255 for
 * exp_avg_sq, 1 to 127 for exp_avg, whose bit 7 is the sign; 0 stands for 0.
 * exp_avg is rounded to nearest (ties to even); exp_avg_sq stochastically
 * (nearest rounding would lose every change of less than half a step, and a
 * step of beta2 = 0.999 changes it by a thousandth), and a value above 0 never
 * becomes 0.
 * A non-finite gradient element makes its parameter NaN; its 8-bit states take
 * their largest code and leave their block's exponent alone.
 */
typedef struct {
    void *param;             /* [n] of param_dtype, updated */
    const void *grad;        /* [n] of grad_dtype */
    void *exp_avg;           /* [n], updated */
    void *exp_avg_sq;        /* [n], updated */
    uint8_t *exp_avg_exp;    /* [ceil(n / 256)], 8-bit states only */
    uint8_t *exp_avg_sq_exp; /* [ceil(n / 256)], 8-bit states only */
    int64_t n;
} tsa_adamw_tensor;
int tsa_adamw_step(const tsa_adamw_tensor *tensors, int64_t count, tsa_dtype param_dtype,
                   tsa_dtype grad_dtype, int32_t state_bits, double lr, double beta1, double beta2,
                   double eps, double weight_decay, int64_t step, const float *grad_scale, uint64_t seed,
                   uint64_t offset, void *stream);

/*
 * adamw_state_values -- the values that 8-bit states stand for, as bf16 (which
 * holds them exactly): for checkpoints and inspection.
 *   tensors      as for adamw_step with state_bits 8 (param and grad unused)
 *   exp_avg_out, exp_avg_sq_out  HOST arrays of `count` device pointers to
 *                bf16 [n]
 */
int tsa_adamw_state_values(const tsa_adamw_tensor *tensors, int64_t count, void *const *exp_avg_out,
                           void *const *exp_avg_sq_out, void *stream);

/*
 * lm_head_logprob -- selective_log_softmax of scores that are never written:
 * with z = hidden . weight^T (+ bias), capped to softcap tanh(z / softcap)
 * where softcap > 0, out[m] = ln softmax(z[m] / T over the allowed
 * tokens)[tokens[m]].  The log-probabilities of sampled tokens under a rollout
 * or reference policy, which policy_loss and preference_loss take as inputs.
 *   hidden       bf16 [M, hidden_row_stride], M >= 0
 *   weight       bf16 [V, weight_row_stride]; H a multiple of 8, 8 <= H <=
 *                16384; both row strides multiples of 8 elements and both
 *                bases 16-byte aligned (TSA_ERR_ALIGN)
 *   bias         float [V] or NULL; softcap >= 0, finite (0: none)
 *                (a capped score is within 2^-21 of itself, whatever the cap)
 *   bitmask, mask_row_stride, temperature, temperature_s: as for
 *                selective_log_softmax, one row for each hidden row
 *   tokens       [M] int64; out [M] float, with selective_log_softmax's special
 *                values (-inf for a disallowed token; NaN for a token outside
 *                [0, V) or a row with no allowed finite score)
 *   workspace    at least tsa_lm_head_logprob_workspace_bytes(M, V) bytes,
 *                256-byte aligned
 * bf16 products, fp32 sums (of at most 1024 columns in the tensor cores, which
 * truncate, and to nearest beyond).  The weight is read once for up to 8192
 * rows.
 */
int tsa_lm_head_logprob(const void *hidden, int64_t M, int64_t H, int64_t hidden_row_stride,
                        const void *weight, int64_t V, int64_t weight_row_stride, const float *bias,
                        float softcap, const int32_t *bitmask, int64_t mask_row_stride,
                        const float *temperature, float temperature_s, const int64_t *tokens, float *out,
                        void *workspace, size_t workspace_bytes, void *stream);
size_t tsa_lm_head_logprob_workspace_bytes(int64_t M, int64_t V);

/* Human-readable name of a status code. */
const char *tsa_status_string(int status);

/*
 * Device status: a bit set by any kernel of this library whose bounded wait
 * ran out on the current device.  Synchronises the device, returns TSA_OK or
 * TSA_ERR_DEVICE_TIMEOUT, and clears the flag when `clear` is non-zero.
 */
int tsa_device_status(int clear);

/*
 * Self-test of the bounded-wait path: launches one block that waits on a
 * barrier nothing will complete, with a wait limit of `limit_us`
 * microseconds; the kernel gives up, records the timeout flag and returns.
 * Used by the test-suite to check the failure path without hanging a GPU.
 */
int tsa_selftest_wait_timeout(uint32_t limit_us, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* TSA_H */
