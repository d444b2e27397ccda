/*
 * sherry_ops.h -- operators around the packed ternary layer of libsherry:
 * adapters of many requests beside a packed projection, the norms before and
 * after a block with its gate and residual scale, and the orthogonalised
 * (Newton-Schulz) update of latent weights.
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

#ifdef __cplusplus
}
#endif

#endif /* SHERRY_OPS_H */
