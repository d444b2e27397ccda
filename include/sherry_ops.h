/*
 * sherry_ops.h -- operators around the packed ternary layer of libsherry:
 * adapters of many requests beside a packed projection, the norms before and
 * after a block with its gate and residual scale, the orthogonalised
 * (Newton-Schulz) update of latent weights, the distillation of a student
 * from a teacher's top logits, the packed product with bias, activation and
 * residual, and a mixture-of-experts layer of packed experts for a few tokens.
 *
 * Conventions are those of sherry.h (streams as void*, caller-provided
 * workspaces, host-side argument checks before any launch, no allocation, no
 * synchronisation), and its status codes are used here too; arguments that
 * only these operators have return SHERRY_ERR_ARG.
 */
#ifndef SHERRY_OPS_H
#define SHERRY_OPS_H

#include "sherry.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the gate of a block is shared: none; one value a token; one value a
 * channel; one row of channels for every `gate_rows` consecutive tokens (1: a
 * value an element). */
typedef enum {
  SHERRY_GATE_NONE = 0,
  SHERRY_GATE_TOKEN = 1,
  SHERRY_GATE_CHANNEL = 2,
  SHERRY_GATE_ROWS = 3
} sherry_gate;

/*
 * sherry_block_norm -- what stands between two blocks: the norm after a
 * block, its gate, the scaled residual, and the norm before the next block,
 * for `rows` tokens of `dim` channels (x^ = x / sqrt(mean(x^2) + eps)):
 *
 *   p = w_post * y^;   h_out = res_scale * h + gate * p;   n_out = w_pre * h_out^
 *
 *   h, y, h_out, n_out   [rows, dim], dtype SHERRY_F32 or SHERRY_BF16; n_out
 *            is the norm of h_out before its rounding.  Outputs do not overlap inputs.
 *   w_post, w_pre   [dim], w_dtype SHERRY_F32 or SHERRY_BF16.
 *   gate     dtype of h: [rows] (token), [dim] (channel), [rows / gate_rows, dim] (rows).
 *   y NULL: h_out is not written and n_out = w_pre * h^ (no w_post, no gate,
 *   res_scale 1).  w_post NULL: p = y.  w_pre NULL: n_out is not written.
 *   rows 1 .. 2^31 - 1, dim 1 .. 2^24; pointers need their element's alignment
 *   only (16-byte aligned rows are read 16 bytes a lane).
 */
int32_t sherry_block_norm(int64_t rows, int64_t dim, const void* h, const void* y, int32_t dtype,
                          const void* w_post, const void* w_pre, int32_t w_dtype, const void* gate,
                          int32_t gate_kind, int64_t gate_rows, float res_scale, float eps, void* h_out,
                          void* n_out, void* stream);

/* Workspace bytes of sherry_block_norm_backward; (size_t)-1 on invalid arguments. */
size_t sherry_block_norm_backward_bytes(int64_t rows, int64_t dim, int32_t gate_kind, int64_t gate_rows);

/*
 * sherry_block_norm_backward -- gradients of the above from those of its
 * outputs: dh_out (NULL: zero) and dn_out (NULL: none; dw_pre is zero), dtype of h.
 *   dh, dy   [rows, dim]; dgate the gate's shape; dtype of h.
 *   dw_post, dw_pre   [dim], w_dtype.  Sums over rows are taken in fp32 in an
 *   order fixed by the sizes and rounded once.
 *   Required: dh; dy with y; dw_post with w_post; dw_pre with w_pre; dgate with gate.
 */
int32_t sherry_block_norm_backward(int64_t rows, int64_t dim, const void* h, const void* y, const void* dh_out,
                                   const void* dn_out, int32_t dtype, const void* w_post, const void* w_pre,
                                   int32_t w_dtype, const void* gate, int32_t gate_kind, int64_t gate_rows,
                                   float res_scale, float eps, void* dh, void* dy, void* dw_post, void* dw_pre,
                                   void* dgate, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of sherry_adapter_gemv (decode 1) or sherry_adapter_gemm
 * (decode 0) for `tokens` rows; (size_t)-1 on invalid arguments. */
size_t sherry_adapter_workspace_bytes(int64_t n, int64_t k, int32_t granularity, int32_t group_size,
                                      int64_t tokens, int32_t rank, int32_t decode);

/*
 * sherry_adapter_gemv / sherry_adapter_gemm -- a packed projection with a
 * low-rank adapter of its own for each token, beside the shared weight:
 *
 *   y[m, n] = sum_k x[m, k] T[n, k] alpha(n, k)
 *           + scale[c] sum_{r < ranks[c]} b[c, n, r] sum_k a[c, r, k] x[m, k],   c = ids[m]
 *
 *   a [adapters, rank, K], b [adapters, N, rank]  bf16; rank a multiple of 8, 8 .. 256.
 *   scale [adapters] fp32; ranks [adapters] int32 or NULL (all of `rank`): rows
 *   of a and columns of b from ranks[c] on are never used, whatever they hold.
 *   ids [tokens] int32, in any order; a token whose id lies outside
 *   [0, adapters) gets the projection alone.
 *   Both products are added in fp32 before y's one rounding.
 *   gemv: batch 1..16, y bf16 or fp32.  gemm: m >= 1, y bf16.  The packed
 *   operand and x as for sherry_gemv and sherry_gemm.
 *   scale, ranks and ids need 4-byte alignment, the rest 16-byte.
 */
int32_t sherry_adapter_gemv(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                            const float* alpha, const void* x, int32_t batch, void* y, int32_t y_dtype,
                            const void* a, const void* b, const float* scale, const int32_t* ranks,
                            const int32_t* ids, int32_t adapters, int32_t rank, void* workspace,
                            size_t workspace_bytes, void* stream);
int32_t sherry_adapter_gemm(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                            const float* alpha, const void* x, int64_t m, void* y, const void* a, const void* b,
                            const float* scale, const int32_t* ranks, const int32_t* ids, int32_t adapters,
                            int32_t rank, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of the two calls below; (size_t)-1 on invalid arguments. */
size_t sherry_muon_workspace_bytes(int32_t count, int64_t n, int64_t k);

/*
 * sherry_orthogonalize -- `steps` Newton-Schulz steps on each of `count`
 * matrices g [N, K]: X = g / (|g| + eps) (Frobenius norm; transposed where
 * N > K), then X <- a X + (b A + c A A) X with A = X X^T.  With the default
 * quintic coefficients five steps bring every singular value that is not far below the
 * norm near 1.  The products keep 22 bits of each factor and fp32 sums;
 * results in fp32 are nearer to 64 bits than the same steps in fp32 products.
 *   g, out   [count, N, K] contiguous, dtype SHERRY_F32 or SHERRY_BF16; out may be g.
 *   steps 1..16.  Coefficients: with m_0 = 1 and m_i+1 the largest |a s + b s^3 + c s^5| of s in [0, m_i]
 *   (the largest singular value that a step can give), every step has to begin below m_i = 2.82 with
 *   |b t + c t^2| below 7.98 for t in [0, m_i^2], the range in which the products are kept; others return
 *   SHERRY_ERR_ARG.
 *   N, K 1 .. 16384, count 1 .. 65535.
 */
int32_t sherry_orthogonalize(int32_t count, int64_t n, int64_t k, const void* g, int32_t dtype, void* out,
                             int32_t steps, float a, float b, float c, float eps, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * sherry_muon_step -- momentum, orthogonalisation and the update of latent
 * weights in one call:
 *   buf_out = momentum * buf + grad;  u = nesterov ? grad + momentum * buf_out : buf_out
 *   w_out = w * (1 - lr * weight_decay) - lr * scale * orthogonalize(u)
 * Wide and tall matrices take their steps in groups (as sherry_orthogonalize does in bf16): the update is
 * off by up to 2.5 times as much as with steps one by one, about what fp32 products are off by.
 *   w, grad, buf, w_out, buf_out   [count, N, K], one dtype; w_out may be w, grad or buf, buf_out grad or buf.
 *   Outputs that overlap an input otherwise, and buf_out on w or w_out, return SHERRY_ERR_ARG.
 */
int32_t sherry_muon_step(int32_t count, int64_t n, int64_t k, const void* w, const void* grad, const void* buf,
                         int32_t dtype, void* w_out, void* buf_out, float lr, float momentum, int32_t nesterov,
                         float weight_decay, float scale, int32_t steps, float a, float b, float c, float eps,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of sherry_distill_loss (dtype of the logits); (size_t)-1 on invalid arguments. */
size_t sherry_distill_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype);

/*
 * sherry_distill_loss -- the loss of `rows` student rows s [vocab] against a teacher's `slots` top logits u_j of
 * ids i_j (t the temperature, q = softmax(s / t)):
 *
 *   p_j = exp(u_j / t - teacher_lse), rest = max(0, 1 - sum_j p_j);   teacher_lse NULL: p = softmax(u / t), rest = 0
 *   kd = t^2 (sum_j p_j log(p_j / q_ij) + rest log(rest / q_rest)),   q_rest = the sum of q outside the ids
 *   loss = kd_weight kd + (1 - kd_weight) (-log softmax(s)_label)
 *
 *   logits   [rows, vocab], dtype SHERRY_F32 or SHERRY_BF16, rows `row_stride` >= vocab elements apart.
 *   teacher  [rows, slots], teacher_dtype; ids [rows, slots] int32 (ids_64: int64).  A slot whose id lies outside
 *            [0, vocab) is empty, whatever its logit.  An id in several slots counts once for each, and once as a
 *            place outside the tail.  A row without a slot (without teacher_lse also one whose logits are all
 *            -infinity) has kd = 0; where the ids are the whole vocabulary, rest is 0.
 *   teacher_lse [rows] fp32: log of the sum of exp(u / t) over the teacher's whole vocabulary.
 *   labels   [rows] int32 (labels_64: int64) or NULL; outside [0, vocab): no label, the second term is 0.
 *   loss     [rows] fp32.  stats [rows, 6 + slots] fp32 for the backward pass, or NULL.
 *   A kd_weight of 0 (1) leaves the first (second) term out, whatever it is.
 *   rows 1 .. 2^31 - 1, vocab 1 .. 2^30, slots 1 .. 1024, temperature 1e-3 .. 1e3; pointers need
 *   their element's alignment (16-byte aligned rows are not needed for 16-byte loads).  Single exponentials
 *   and sums of 16 bytes of logits are fp32, a row's sums past those and its logarithms are taken in 64 bits.
 */
int32_t sherry_distill_loss(int64_t rows, int64_t vocab, const void* logits, int64_t row_stride, int32_t dtype,
                            const void* teacher, int32_t teacher_dtype, const void* ids, int32_t ids_64,
                            int32_t slots, float temperature, const float* teacher_lse, const void* labels,
                            int32_t labels_64, float kd_weight, float* loss, float* stats, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * sherry_distill_loss_backward -- dlogits [rows, vocab], dtype of the logits, from the gradients g [rows] of the
 * losses and the stats of a sherry_distill_loss with the same arguments.  A row with g = 0 gets zeros and is not
 * read.  dlogits may be logits (same rows); outputs that overlap them otherwise return SHERRY_ERR_ARG.
 */
int32_t sherry_distill_loss_backward(int64_t rows, int64_t vocab, const float* g, const void* logits,
                                     int64_t row_stride, int32_t dtype, const void* ids, int32_t ids_64,
                                     int32_t slots, float temperature, const void* labels, int32_t labels_64,
                                     float kd_weight, const float* stats, void* dlogits, int64_t dlogits_stride,
                                     void* stream);

typedef enum {
  SHERRY_ACT_NONE = 0,
  SHERRY_ACT_RELU = 1,
  SHERRY_ACT_RELU2 = 2,     /* max(z, 0)^2 */
  SHERRY_ACT_SILU = 3,
  SHERRY_ACT_GELU = 4,      /* z Phi(z) */
  SHERRY_ACT_GELU_TANH = 5  /* its tanh form */
} sherry_activation;

/*
 * sherry_linear_gemv / sherry_linear_gemm -- the packed product of 1..16 tokens (one launch, no workspace) or of m
 * tokens (MFMA), with what follows it before its one rounding:
 *
 *   z[m, n] = sum_k x[m, k] T[n, k] alpha(n, k) + bias[n]
 *   y = f(z) + res_scale * residual;   gated: y[m, j] = f(z[m, j]) z[m, N/2 + j] + res_scale * residual[m, j]
 *
 *   The packed operand and x as for sherry_gemv.  gated: N is even, rows [gate; values] packed as one weight.
 *   y        [tokens, N or N/2], bf16; gemv also SHERRY_F32.
 *   bias     [N], bias_dtype SHERRY_F32 or SHERRY_BF16, or NULL.
 *   residual [tokens, N or N/2] bf16 or NULL (res_scale 1).  y (bf16) may be residual; outputs that overlap it
 *            otherwise, or x, return SHERRY_ERR_ARG.
 *   bias, and gemv's residual and y, need their element's alignment, gemm's residual 8-byte, the rest 16-byte.
 *   Without bias, activation, gate and residual gemm is sherry_gemm.  gemm takes sherry_gemm's workspace:
 *   sherry_workspace_bytes(SHERRY_OP_GEMM, n, k, .., m, 1).
 */
int32_t sherry_linear_gemv(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                           const float* alpha, const void* x, int32_t batch, void* y, int32_t y_dtype,
                           const void* bias, int32_t bias_dtype, int32_t activation, int32_t gated,
                           const void* residual, float res_scale, void* stream);
int32_t sherry_linear_gemm(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                           const float* alpha, const void* x, int64_t m, void* y, const void* bias,
                           int32_t bias_dtype, int32_t activation, int32_t gated, const void* residual,
                           float res_scale, void* workspace, size_t workspace_bytes, void* stream);

typedef enum { SHERRY_SCORE_SOFTMAX = 0, SHERRY_SCORE_SIGMOID = 1 } sherry_scoring;

/* Workspace bytes of sherry_moe_decode; (size_t)-1 on invalid arguments. */
size_t sherry_moe_workspace_bytes(int32_t tokens, int64_t dim, int64_t hidden, int32_t experts, int32_t shared,
                                  int32_t top_k);

/*
 * sherry_moe_decode -- a whole mixture-of-experts layer of packed experts for 1..16 tokens x [tokens, dim]:
 *
 *   l = x router^T;  s = softmax(l) over the experts, or sigmoid(l)
 *   the top_k largest of s, or of s + bias (the lowest index of equal ones);  w = s (normalize: / their sum) * scale
 *   y = sum_j w_j down_j h_j + sum of the shared experts' down h + residual
 *   h = f(up x), or with gated f(gate x) * (up x), rows [gate; up] packed as one weight
 *
 *   x        bf16; router [experts, dim], router_dtype SHERRY_F32 or SHERRY_BF16; bias [experts] fp32 or NULL.
 *   An expert whose key is -infinity (a bias of -infinity) is off: a token with fewer than top_k others meets only
 *   those, with none only the shared experts.  Equal logits count as equal scores.
 *   up       [experts + shared] packed weights [hidden (gated: 2 hidden), dim], one after another, and their scales
 *            [experts + shared][sherry_num_scales]; the shared experts, which every token meets with the weight 1,
 *            are the last.  down the same for [dim, hidden].
 *   residual [tokens, dim] bf16 or NULL; y [tokens, dim] SHERRY_BF16 or SHERRY_F32; y may be residual (bf16) or x.
 *   h is kept in fp32's 24 bits; sums are fp32 in an order fixed by the sizes and the choices.
 *   dim, hidden multiples of 128, at most 65536; experts 1 .. 512, top_k 1 .. min(16, experts), shared 0 .. 4.
 *   No token's values reach another's result, nor does an expert's scale that is not finite reach a token that it
 *   does not serve; but the order of its sums follows the experts that the batch uses.
 *   No host synchronisation; capturable.
 */
int32_t sherry_moe_decode(int32_t tokens, int64_t dim, int64_t hidden, const void* x, const void* router,
                          int32_t router_dtype, int32_t experts, int32_t shared, int32_t top_k, int32_t scoring,
                          int32_t normalize, const float* bias, float scale, int32_t activation, int32_t gated,
                          const void* up, const float* up_alpha, int32_t up_granularity, int32_t up_group,
                          const void* down, const float* down_alpha, int32_t down_granularity, int32_t down_group,
                          const void* residual, void* y, int32_t y_dtype, void* workspace, size_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SHERRY_OPS_H */
