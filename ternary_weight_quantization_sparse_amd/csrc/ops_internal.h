// Internal declarations of the operators around the packed layer
// (include/sherry_ops.h): block norms, adapters, orthogonalised updates.
#pragma once

#include "../../include/sherry_ops.h"
#include "sherry_internal.h"

namespace sherry {

// ---------------------------------------------------------------- block norms
struct NormArgs {
  int64_t rows;
  int dim;
  const void *h, *y, *w_post, *w_pre, *gate;
  int gate_kind;
  int64_t gate_rows;
  float res_scale, eps;
  void *h_out, *n_out;
};
struct NormGrads {
  const void *dh_out, *dn_out;
  void *dh, *dy, *dw_post, *dw_pre, *dgate;
  float *part_pre, *part_post, *part_gate;   // column sums of each workgroup's rows
  float* stats;                              // rows longer than registers: 3 floats a row
};
// Rows of the backward pass's workgroups; a "sequence" is the rows that share
// a gate row (all rows where there is none).
struct NormSplit {
  int64_t seqs, seq_rows;        // sequences and the rows of each
  int64_t block_rows;            // rows of a workgroup inside one sequence
  int64_t blocks_per_seq;        // workgroups of a sequence
  int64_t seqs_per_block;        // > 1: whole sequences of a workgroup
  int64_t blocks;
};
struct NormBackwardWs {
  size_t pre, post, gate, stats, bytes;
};
NormSplit plan_norm_backward(int64_t rows, int64_t dim, int gate_kind, int64_t gate_rows);
NormBackwardWs norm_backward_ws(const NormSplit& s, int64_t rows, int64_t dim, int gate_kind, int64_t gate_rows);
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool w_bf16, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, const NormGrads& d, const NormSplit& sp, bool bf16, bool w_bf16,
                                hipStream_t s);

// ---------------------------------------------------------------- adapters
struct AdapterArgs {
  const uint16_t* a;        // [count, rank, K] bf16
  const uint16_t* b;        // [count, N, rank] bf16
  const float* scale;       // [count]
  const int32_t* ranks;     // [count]: rows of a / columns of b in use; null: all
  const int32_t* ids;       // [tokens]: the token's adapter; outside [0, count): none
  int count, rank;
};
// Rows of a (columns of b) that adapter c uses.
__device__ inline int adapter_rank(const AdapterArgs& a, int c) {
  return a.ranks ? min(max(a.ranks[c], 0), a.rank) : a.rank;
}
// The adapters' term of a product: scale * a x of each token, [tokens, rank],
// as two bf16 terms.
struct AdapterTerm {
  AdapterArgs a;
  const uint16_t *vh, *vl;
};
hipError_t launch_gemm_adapted(const GemmPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m,
                               uint16_t* y, float* ws, const AdapterTerm& ad, hipStream_t s);
struct AdapterPlan {
  size_t base_offset;       // the packed product's own workspace
  size_t y_offset;          // fp32 base product (decode)
  size_t v_offset;          // low-rank products [tokens, rank]: fp32 (decode), or bf16 hi and lo
  size_t workspace_bytes;
};
AdapterPlan plan_adapter(int64_t n, int64_t k, int gran, int group_size, int64_t tokens, int rank, bool decode);
hipError_t launch_adapter_gemv(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int batch, void* y,
                               bool y_bf16, const AdapterArgs& ad, char* ws, hipStream_t s);
hipError_t launch_adapter_gemm(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m, uint16_t* y,
                               const AdapterArgs& ad, char* ws, hipStream_t s);

// ---------------------------------------------------------------- orthogonalised updates
struct MuonArgs {
  int count;
  int64_t n, k;
  const void *w, *grad, *buf;     // orthogonalize: the matrix in grad, w and buf null
  void *w_out, *buf_out;          // orthogonalize: the result in w_out
  float lr, momentum, decay, scale, eps;
  bool nesterov;
  int steps;
  float ca, cb, cc;
};
struct MuonCut {
  int rows, cols, splits;         // an output tile, and the K ranges of it
};
struct MuonPlan {
  int group;                      // steps between two looks at X
  MuonCut gram, sym, pair, apply, last;
  int64_t r, l, rp, lp;           // smaller and larger side, and padded to whole tiles
  int64_t parts;                  // workgroups of the sum of squares
  size_t u, sums, x, xt0, xt1, a, b, pa, d0, d1, partial, workspace_bytes;
};
// loose: steps may be taken in groups (see muon.hip).
MuonPlan plan_muon(int count, int64_t n, int64_t k, bool loose);
hipError_t launch_muon(const MuonPlan& p, const MuonArgs& a, bool bf16, char* ws, hipStream_t s);

}  // namespace sherry
