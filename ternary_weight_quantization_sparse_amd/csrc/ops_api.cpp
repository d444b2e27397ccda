// C-ABI entry points of the operators around the packed layer
// (include/sherry_ops.h): argument checks, plans, launches.  Every check runs
// on the host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ops_internal.h"

using namespace sherry;

namespace {

bool multiple_of(const void* p, uintptr_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }
bool aligned16(const void* p) { return multiple_of(p, 16); }
int hip_status(hipError_t e) { return e == hipSuccess ? SHERRY_OK : SHERRY_ERR_HIP; }

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1, kMaxDim = (int64_t)1 << 24;

int check_norm_shape(int64_t rows, int64_t dim, int32_t kind, int64_t gate_rows) {
  if (rows < 1 || rows > kMaxRows || dim < 1 || dim > kMaxDim) return SHERRY_ERR_ARG;
  if (kind < SHERRY_GATE_NONE || kind > SHERRY_GATE_ROWS) return SHERRY_ERR_ARG;
  if (kind == SHERRY_GATE_ROWS && (gate_rows < 1 || rows % gate_rows != 0)) return SHERRY_ERR_ARG;
  return SHERRY_OK;
}

int check_norm(int64_t rows, int64_t dim, const void* h, const void* y, int32_t dtype, const void* w_post,
               const void* w_pre, int32_t w_dtype, const void* gate, int32_t kind, int64_t gate_rows,
               float res_scale, float eps) {
  const int st = check_norm_shape(rows, dim, kind, gate_rows);
  if (st != SHERRY_OK) return st;
  if (dtype != SHERRY_F32 && dtype != SHERRY_BF16) return SHERRY_ERR_DTYPE;
  if (w_dtype != SHERRY_F32 && w_dtype != SHERRY_BF16) return SHERRY_ERR_DTYPE;
  if (!h || (kind != SHERRY_GATE_NONE && !gate)) return SHERRY_ERR_NULL;
  if (!y && !w_pre) return SHERRY_ERR_NULL;
  if (!y && (w_post || kind != SHERRY_GATE_NONE || res_scale != 1.0f)) return SHERRY_ERR_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(res_scale)) return SHERRY_ERR_ARG;
  const uintptr_t item = dtype == SHERRY_F32 ? 4 : 2, w_item = w_dtype == SHERRY_F32 ? 4 : 2;
  if (!multiple_of(h, item) || !multiple_of(y, item) || !multiple_of(gate, item) || !multiple_of(w_post, w_item) ||
      !multiple_of(w_pre, w_item))
    return SHERRY_ERR_ALIGN;
  return SHERRY_OK;
}

int check_adapted(int64_t n, int64_t k, int32_t gran, int32_t group_size, int64_t tokens, int32_t rank, bool decode) {
  const int32_t op = decode ? SHERRY_OP_GEMV : SHERRY_OP_GEMM;
  if (decode ? (tokens < 1 || tokens > 16) : tokens < 1) return SHERRY_ERR_BATCH;
  if (rank < 8 || rank > 256 || rank % 8 != 0) return SHERRY_ERR_ARG;
  // the packed product's own limits
  return sherry_workspace_bytes(op, n, k, gran, group_size, tokens, 1) == (size_t)-1 ? SHERRY_ERR_SHAPE : SHERRY_OK;
}

int check_adapters(const void* a, const void* b, const float* scale, const int32_t* ranks, const int32_t* ids,
                   int32_t adapters) {
  if (adapters < 1) return SHERRY_ERR_ARG;
  if (!a || !b || !scale || !ids) return SHERRY_ERR_NULL;
  if (!aligned16(a) || !aligned16(b) || !multiple_of(scale, 4) || !multiple_of(ranks, 4) || !multiple_of(ids, 4))
    return SHERRY_ERR_ALIGN;
  return SHERRY_OK;
}

constexpr int64_t kMuonMaxSide = 16384;

int check_muon_shape(int32_t count, int64_t n, int64_t k) {
  return count < 1 || count > 65535 || n < 1 || k < 1 || n > kMuonMaxSide || k > kMuonMaxSide ? SHERRY_ERR_ARG
                                                                                              : SHERRY_OK;
}

int run_muon(MuonArgs a, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != SHERRY_F32 && dtype != SHERRY_BF16) return SHERRY_ERR_DTYPE;
  if (a.steps < 1 || a.steps > 16 || !(a.eps >= 0.0f)) return SHERRY_ERR_ARG;
  const float args[] = {a.ca, a.cb, a.cc, a.eps, a.lr, a.momentum, a.decay, a.scale};
  for (float v : args)
    if (!std::isfinite(v)) return SHERRY_ERR_ARG;
  const uintptr_t item = dtype == SHERRY_F32 ? 4 : 2;
  if (!multiple_of(a.w, item) || !multiple_of(a.grad, item) || !multiple_of(a.buf, item) ||
      !multiple_of(a.w_out, item) || !multiple_of(a.buf_out, item))
    return SHERRY_ERR_ALIGN;
  // groups of steps: not for fp32 results, and only where the coefficients keep
  // a group's product in the range of its float16 planes
  const MuonRange range = muon_range(a.ca, a.cb, a.cc, a.steps);
  const bool loose = (dtype == SHERRY_BF16 || a.w) && range.groups;
  const MuonPlan plan = plan_muon(a.count, a.n, a.k, loose);
  if (!workspace || workspace_bytes < plan.workspace_bytes) return SHERRY_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SHERRY_ERR_ALIGN;
  if (!range.steps) return SHERRY_ERR_ARG;
  // an output is an input or apart from it; buf_out is written before w is read, and with w_out
  const uintptr_t bytes = (uintptr_t)a.count * (uintptr_t)a.n * (uintptr_t)a.k * item;
  auto apart = [&](const void* p, const void* q) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return !p || !q || (x < y ? y - x : x - y) >= bytes;
  };
  for (const void* in : {a.w, a.grad, a.buf})
    for (const void* out : {static_cast<const void*>(a.w_out), static_cast<const void*>(a.buf_out)})
      if (in != out && !apart(in, out)) return SHERRY_ERR_ARG;
  if (!apart(a.buf_out, a.w) || !apart(a.buf_out, a.w_out)) return SHERRY_ERR_ARG;
  return hip_status(launch_muon(plan, a, dtype == SHERRY_BF16, static_cast<char*>(workspace),
                                static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int32_t sherry_block_norm(int64_t rows, int64_t dim, const void* h, const void* y, int32_t dtype,
                          const void* w_post, const void* w_pre, int32_t w_dtype, const void* gate,
                          int32_t gate_kind, int64_t gate_rows, float res_scale, float eps, void* h_out,
                          void* n_out, void* stream) {
  const int st = check_norm(rows, dim, h, y, dtype, w_post, w_pre, w_dtype, gate, gate_kind, gate_rows, res_scale, eps);
  if (st != SHERRY_OK) return st;
  if ((y && !h_out) || (w_pre && !n_out)) return SHERRY_ERR_NULL;
  const uintptr_t item = dtype == SHERRY_F32 ? 4 : 2;
  if (!multiple_of(h_out, item) || !multiple_of(n_out, item)) return SHERRY_ERR_ALIGN;
  const NormArgs a{rows, (int)dim, h, y, w_post, w_pre, gate, gate_kind, gate_rows, res_scale, eps, h_out, n_out, 0};
  return hip_status(launch_norm_forward(a, dtype == SHERRY_BF16, w_dtype == SHERRY_BF16,
                                        static_cast<hipStream_t>(stream)));
}

size_t sherry_block_norm_backward_bytes(int64_t rows, int64_t dim, int32_t gate_kind, int64_t gate_rows) {
  if (check_norm_shape(rows, dim, gate_kind, gate_rows) != SHERRY_OK) return (size_t)-1;
  return norm_backward_ws(plan_norm_backward(rows, dim, gate_kind, gate_rows), rows, dim, gate_kind, gate_rows).bytes;
}

int32_t sherry_block_norm_backward(int64_t rows, int64_t dim, const void* h, const void* y, const void* dh_out,
                                   const void* dn_out, int32_t dtype, const void* w_post, const void* w_pre,
                                   int32_t w_dtype, const void* gate, int32_t gate_kind, int64_t gate_rows,
                                   float res_scale, float eps, void* dh, void* dy, void* dw_post, void* dw_pre,
                                   void* dgate, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_norm(rows, dim, h, y, dtype, w_post, w_pre, w_dtype, gate, gate_kind, gate_rows, res_scale, eps);
  if (st != SHERRY_OK) return st;
  if (!dh || (y && !dy) || (w_post && !dw_post) || (w_pre && !dw_pre) || (gate_kind != SHERRY_GATE_NONE && !dgate))
    return SHERRY_ERR_NULL;
  const uintptr_t item = dtype == SHERRY_F32 ? 4 : 2, w_item = w_dtype == SHERRY_F32 ? 4 : 2;
  if (!multiple_of(dh_out, item) || !multiple_of(dn_out, item) || !multiple_of(dh, item) || !multiple_of(dy, item) ||
      !multiple_of(dgate, item) || !multiple_of(dw_post, w_item) || !multiple_of(dw_pre, w_item))
    return SHERRY_ERR_ALIGN;
  const NormSplit sp = plan_norm_backward(rows, dim, gate_kind, gate_rows);
  const NormBackwardWs w = norm_backward_ws(sp, rows, dim, gate_kind, gate_rows);
  if (!workspace || workspace_bytes < w.bytes) return SHERRY_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SHERRY_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  // a norm that no gradient comes from takes no part: dw_pre is zero, and what h_out
  // holds (infinities among it) does not meet the other gradients
  const bool pre = w_pre && dn_out;
  const NormArgs a{rows,      (int)dim, h,       y,       w_post, pre ? w_pre : nullptr, gate, gate_kind,
                   gate_rows, res_scale, eps, nullptr, nullptr, 0};
  const NormGrads d{dh_out,
                    pre ? dn_out : nullptr,
                    dh,
                    dy,
                    dw_post,
                    w_pre ? dw_pre : nullptr,
                    dgate,
                    pre ? reinterpret_cast<float*>(ws + w.pre) : nullptr,
                    w_post ? reinterpret_cast<float*>(ws + w.post) : nullptr,
                    w.gate ? reinterpret_cast<float*>(ws + w.gate) : nullptr,
                    reinterpret_cast<float*>(ws + w.stats)};
  return hip_status(launch_norm_backward(a, d, sp, dtype == SHERRY_BF16, w_dtype == SHERRY_BF16,
                                         static_cast<hipStream_t>(stream)));
}

size_t sherry_adapter_workspace_bytes(int64_t n, int64_t k, int32_t granularity, int32_t group_size,
                                      int64_t tokens, int32_t rank, int32_t decode) {
  if (check_adapted(n, k, granularity, group_size, tokens, rank, decode != 0) != SHERRY_OK) return (size_t)-1;
  return plan_adapter(n, k, granularity, group_size, tokens, rank, decode != 0).workspace_bytes;
}

int32_t sherry_adapter_gemv(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                            const float* alpha, const void* x, int32_t batch, void* y, int32_t y_dtype,
                            const void* a, const void* b, const float* scale, const int32_t* ranks,
                            const int32_t* ids, int32_t adapters, int32_t rank, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int st = check_adapted(n, k, granularity, group_size, batch, rank, true);
  if (st == SHERRY_OK) st = check_adapters(a, b, scale, ranks, ids, adapters);
  if (st != SHERRY_OK) return st;
  if (y_dtype != SHERRY_BF16 && y_dtype != SHERRY_F32) return SHERRY_ERR_DTYPE;
  if (!packed || !alpha || !x || !y) return SHERRY_ERR_NULL;
  if (!aligned16(packed) || !aligned16(alpha) || !aligned16(x) || !aligned16(y)) return SHERRY_ERR_ALIGN;
  const AdapterPlan plan = plan_adapter(n, k, granularity, group_size, batch, rank, true);
  if (!workspace || workspace_bytes < plan.workspace_bytes) return SHERRY_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SHERRY_ERR_ALIGN;
  const AdapterArgs ad{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), scale, ranks, ids, adapters,
                       rank};
  return hip_status(launch_adapter_gemv(plan, n, k, granularity, group_size, static_cast<const uint8_t*>(packed), alpha,
                                        static_cast<const uint16_t*>(x), batch, y, y_dtype == SHERRY_BF16, ad,
                                        static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

int32_t sherry_adapter_gemm(int64_t n, int64_t k, int32_t granularity, int32_t group_size, const void* packed,
                            const float* alpha, const void* x, int64_t m, void* y, const void* a, const void* b,
                            const float* scale, const int32_t* ranks, const int32_t* ids, int32_t adapters,
                            int32_t rank, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_adapted(n, k, granularity, group_size, m, rank, false);
  if (st == SHERRY_OK) st = check_adapters(a, b, scale, ranks, ids, adapters);
  if (st != SHERRY_OK) return st;
  if (k > ((int64_t)1 << 21)) return SHERRY_ERR_UNSUPPORTED;   // as sherry_gemm
  if (m > ((int64_t)1 << 46) / k || (m + 127) / 128 > 65535) return SHERRY_ERR_BATCH;
  if (!packed || !alpha || !x || !y) return SHERRY_ERR_NULL;
  if (!aligned16(packed) || !aligned16(alpha) || !aligned16(x) || !aligned16(y)) return SHERRY_ERR_ALIGN;
  const AdapterPlan plan = plan_adapter(n, k, granularity, group_size, m, rank, false);
  if (!workspace || workspace_bytes < plan.workspace_bytes) return SHERRY_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SHERRY_ERR_ALIGN;
  const AdapterArgs ad{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), scale, ranks, ids, adapters,
                       rank};
  return hip_status(launch_adapter_gemm(plan, n, k, granularity, group_size, static_cast<const uint8_t*>(packed), alpha,
                                        static_cast<const uint16_t*>(x), m, static_cast<uint16_t*>(y), ad,
                                        static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sherry_muon_workspace_bytes(int32_t count, int64_t n, int64_t k) {
  return check_muon_shape(count, n, k) == SHERRY_OK ? plan_muon(count, n, k, false).workspace_bytes : (size_t)-1;
}

int32_t sherry_orthogonalize(int32_t count, int64_t n, int64_t k, const void* g, int32_t dtype, void* out,
                             int32_t steps, float a, float b, float c, float eps, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const int st = check_muon_shape(count, n, k);
  if (st != SHERRY_OK) return st;
  if (!g || !out) return SHERRY_ERR_NULL;
  const MuonArgs m{count, n, k, nullptr, g, nullptr, out, nullptr, 0.f, 0.f, 0.f, 1.f, eps, false, steps, a, b, c};
  return run_muon(m, dtype, workspace, workspace_bytes, stream);
}

int32_t sherry_muon_step(int32_t count, int64_t n, int64_t k, const void* w, const void* grad, const void* buf,
                         int32_t dtype, void* w_out, void* buf_out, float lr, float momentum, int32_t nesterov,
                         float weight_decay, float scale, int32_t steps, float a, float b, float c, float eps,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_muon_shape(count, n, k);
  if (st != SHERRY_OK) return st;
  if (!w || !grad || !buf || !w_out || !buf_out) return SHERRY_ERR_NULL;
  const MuonArgs m{count, n, k, w, grad, buf, w_out, buf_out, lr, momentum, weight_decay, scale, eps, nesterov != 0,
                   steps, a, b, c};
  return run_muon(m, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
