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
  int64_t row0;              // a launch's first row, where rows take several launches
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
// The adapters' term of a product: scale * a x of each token, [tokens, rank], as
// a sum of bf16 terms, each in a plane of its own, the largest first.
constexpr int kAdapterTerms = 3;
struct AdapterTerm {
  AdapterArgs a;
  const uint16_t* v;
  int64_t plane;
};
hipError_t launch_gemm_adapted(const GemmPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m,
                               uint16_t* y, float* ws, const AdapterTerm& ad, hipStream_t s);
struct AdapterPlan {
  size_t partial_offset;    // the packed product's workspace: decode, fp32 partials [splits, tokens, N]
  size_t v_offset;          // low-rank products [tokens, rank]: fp32 (decode), or bf16 terms
  size_t workspace_bytes;
};
AdapterPlan plan_adapter(int64_t n, int64_t k, int gran, int group_size, int64_t tokens, int rank, bool decode);
hipError_t launch_adapter_gemv(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int batch, void* y,
                               bool y_bf16, const AdapterArgs& ad, char* ws, hipStream_t s);
hipError_t launch_adapter_gemm(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m, uint16_t* y,
                               const AdapterArgs& ad, char* ws, hipStream_t s);

// Decode's low-rank products v = scale * a x, computed by workgroups of the
// packed product's launch past its own `panels`: a wave per (token, row of a).
// They run beside the packed product instead of before it.
struct AdapterShrink {
  AdapterArgs a;
  float* v;        // [tokens, rank]
  int tokens, panels;
};
hipError_t launch_gemv_partials(const GemvPlan& p, int64_t n, int64_t k, int gran, int group_size,
                                const uint8_t* packed, const float* alpha, const uint16_t* x, int batch,
                                float* partial, AdapterShrink ad, hipStream_t s);
template <int WAVES>
unsigned adapter_shrink_blocks(unsigned depth, const AdapterShrink& ad) {
  const unsigned items = (unsigned)(ad.tokens * ad.a.rank), per = WAVES * depth;
  return (items + per - 1) / per;
}
__device__ inline int adapter_of(const AdapterArgs& a, int64_t token) {
  const int c = a.ids[token];
  return c >= 0 && c < a.count ? c : -1;
}
// 8 products of bf16 pairs, added in fp32
typedef uint32_t adapter_u32x4 __attribute__((ext_vector_type(4)));
__device__ inline float dot8(const adapter_u32x4 a, const adapter_u32x4 b, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += __uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16);
    s += __uint_as_float(a[i] & 0xFFFF0000u) * __uint_as_float(b[i] & 0xFFFF0000u);
  }
  return s;
}
template <int WAVES>
__device__ inline bool adapter_shrink_block(const uint16_t* x, int64_t k, const AdapterShrink& ad) {
  if ((int)blockIdx.x < ad.panels) return false;
  const int lane = threadIdx.x & 63;
  const int item = (int)((blockIdx.x - ad.panels) * gridDim.z + blockIdx.z) * WAVES +
                   __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = item / ad.a.rank, row = item % ad.a.rank;
  if (token >= ad.tokens) return true;
  const int c = adapter_of(ad.a, token);
  if (c < 0 || row >= adapter_rank(ad.a, c)) return true;   // never read
  const adapter_u32x4* ar = reinterpret_cast<const adapter_u32x4*>(ad.a.a + ((int64_t)c * ad.a.rank + row) * k);
  const adapter_u32x4* xr = reinterpret_cast<const adapter_u32x4*>(x + token * k);
  float s = 0.f;
  const int all = (int)(k / 8);
  int i = lane;
  for (; i + 3 * 64 < all; i += 4 * 64) {   // four steps' loads in flight
    const adapter_u32x4 a0 = ar[i], a1 = ar[i + 64], a2 = ar[i + 128], a3 = ar[i + 192];
    const adapter_u32x4 x0 = xr[i], x1 = xr[i + 64], x2 = xr[i + 128], x3 = xr[i + 192];
    s = dot8(a3, x3, dot8(a2, x2, dot8(a1, x1, dot8(a0, x0, s))));
  }
  for (; i < all; i += 64) s = dot8(ar[i], xr[i], s);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) ad.v[token * ad.a.rank + row] = s * ad.a.scale[c];
  return true;
}

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
  int count;                      // matrices at a time
  int group;                      // steps between two looks at X
  MuonCut gram, sym, pair, apply, last;
  int64_t r, l, rp, lp;           // smaller and larger side, and padded to whole tiles
  int64_t parts;                  // workgroups of the sum of squares
  size_t u, sums, x, xt0, xt1, a, b, pa, d0, d1, partial, workspace_bytes;
};
// Whether everything that the steps keep stays in the range of its float16
// planes for every matrix of norm 1: taken one by one, and in groups.
struct MuonRange {
  bool steps, groups;
};
MuonRange muon_range(double a, double b, double c, int steps);
// loose: steps may be taken in groups (see muon.hip).
MuonPlan plan_muon(int matrices, int64_t n, int64_t k, bool loose);
hipError_t launch_muon(const MuonPlan& p, const MuonArgs& a, bool bf16, char* ws, hipStream_t s);

}  // namespace sherry
