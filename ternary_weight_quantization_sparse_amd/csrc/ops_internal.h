// Internal declarations of the operators around the packed layer
// (include/sherry_ops.h): block norms, adapters, orthogonalised updates,
// distillation, the product with an epilogue, mixture of experts.
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

// ---------------------------------------------------------------- distillation
constexpr int kDistillSlots = 1024;   // teacher slots a row
constexpr int kDistillHead = 6;       // floats of a row's statistics before its slots
struct DistillRange {
  double s, s1;      // sums of exp((s - m) / t) and exp(s - m)
  float m;
  int twice;         // an id stands in two slots
};
struct DistillSplit {
  int ranges;                // workgroups of a row
  int64_t range_groups;      // 16-byte groups of each
  size_t workspace_bytes;
};
struct DistillArgs {
  const void* logits;
  int64_t stride, vocab;
  const void *teacher, *ids, *labels;
  bool ids_wide, labels_wide;     // int64 indexes
  int slots;
  const float* teacher_lse;
  double inv_t;                   // 1 / temperature
  float exp_hi, exp_lo;           // log2(e) / temperature
  float kd_weight;
  int ranges;
  int64_t range_groups;
  DistillRange* part;
  float *loss, *stats;
};
struct DistillGrad {
  const float* g;
  const void* logits;
  int64_t stride, vocab;
  const void *ids, *labels;
  bool ids_wide, labels_wide;
  int slots;
  const float* stats;
  double inv_t;
  float exp_hi, exp_lo, kd_weight;
  int ranges;
  int64_t range_groups;
  void* out;
  int64_t out_stride;
};
DistillSplit plan_distill(int64_t rows, int64_t vocab, bool bf16, bool backward);
hipError_t launch_distill(const DistillArgs& a, int64_t rows, bool bf16, bool teacher_bf16, hipStream_t s);
hipError_t launch_distill_backward(const DistillGrad& a, int64_t rows, bool bf16, hipStream_t s);

// ---------------------------------------------------------------- product with an epilogue
struct LinearArgs {
  const uint8_t* packed;
  const float* alpha;
  int64_t n, k;              // gated: n counts the gate's and the values' rows
  int gran, group_sbs;
  const void* bias;          // [n] or null
  bool bias_bf16;
  int activation;
  bool gated;
  const uint16_t* residual;  // [tokens, outputs] or null
  float res_scale;
};
hipError_t launch_linear_decode(const LinearArgs& a, const uint16_t* x, int tokens, void* y, bool y_bf16,
                                hipStream_t s);
hipError_t launch_linear_tiles(const LinearArgs& a, const uint16_t* x, int64_t m, uint16_t* y, hipStream_t s);
GemmPlan plan_linear(int64_t n, int64_t k, int gran, int group_size, int64_t m, bool gated);
hipError_t launch_linear_gemm(const GemmPlan& p, const LinearArgs& a, const uint16_t* x, int64_t m, uint16_t* y,
                              float* ws, hipStream_t s);

// ---------------------------------------------------------------- mixture of experts
constexpr int kMoeExperts = 512, kMoeTopK = 16, kMoeShared = 4;
constexpr int kMoeParts = 8;                            // of the channels, in a launch for the logits
constexpr int kMoeSlots = 16 * kMoeTopK + kMoeShared;   // experts in use at most
struct MoeRoute {
  int count;                         // experts in use
  int list[kMoeSlots];
  int8_t place[kMoeSlots][16];       // among the token's choices; -1: not one of them
  float weight[kMoeSlots][16];
};
struct MoeArgs {
  const uint16_t* x;
  int tokens, experts, top_k, shared, slots;   // slots = top_k + shared
  int64_t dim, hidden;
  const void* router;
  bool router_bf16, softmax, normalize, gated;
  const float* bias;                           // [experts] or null
  float scale;
  int activation;
  const uint8_t *up, *down;                    // [experts + shared] packed weights, one after another
  const float *up_alpha, *down_alpha;
  int64_t up_bytes, down_bytes, up_scales, down_scales;
  int up_gran, up_group_sbs, down_gran, down_group_sbs;
  const uint16_t* residual;
  MoeRoute* route;
  float* logits;                               // [parts][tokens, experts]
  int parts;                                   // 0: the routing makes them itself
  __bf16* h;                                   // [bf16 terms][tokens, slots, hidden]
  int64_t h_plane;
  float* partial;                              // [ranges][tokens, dim]
  int ranges;
};
struct MoePlan {
  int used;                                    // experts in use at most
  int ranges;                                  // of the second products
  bool narrow;                                 // they take 16 rows a workgroup
  int parts;                                   // of the logits' channels
  int64_t h_plane;
  size_t logits_offset, h_offset, partial_offset, workspace_bytes;
};
MoePlan plan_moe(int tokens, int64_t dim, int64_t hidden, int experts, int shared, int top_k, bool router_bf16);
hipError_t launch_moe(const MoePlan& p, MoeArgs a, void* y, bool y_bf16, hipStream_t s);

}  // namespace sherry
