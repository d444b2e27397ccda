// Norms before and after a block, fused with the block's gate and the residual
// scale, and their gradients.
//
// Forward, for a row of D channels with the block's output y and the residual
// stream h (x^ = x / sqrt(mean(x^2) + eps)):
//   p = w_post * y^                  (p = y without w_post)
//   h' = res_scale * h + gate * p    (h' = h without y)
//   n  = w_pre * h'^                 (the next block's input; none without w_pre)
// Backward, from dh' and dn:
//   u = w_pre * dn,  t = dh' + (u - h'^ mean(u h'^)) / rms(h'),  dh = res_scale * t
//   dgate = t * p over the gate's broadcast,  q = gate * t,  v = w_post * q
//   dy = (v - y^ mean(v y^)) / rms(y)
//   dw_pre = sum_rows dn h'^,  dw_post = sum_rows q y^
// Everything is held in fp32 and rounded once, at the stores.  The backward
// pass recomputes p and h' from y and h: reading those costs the same bytes as
// reading a saved h', which would carry the rounding of its type.
//
// HBM bounds all of it: 4 row passes forward (y, h -> h', n), 6 backward (y, h,
// dh', dn -> dy, dh).  A row stays in the registers of one group of threads
// from its loads to its stores, so every byte moves once.  8192 x 2048 bf16
// (fp32 norm weights): forward 134 MB in 25.6 us (5.2 TB/s; a copy of 1 GB
// reaches 5.1), backward 201 MB in 47.5 us (4.2 TB/s) and 5 us for the column
// sums; one row 2.6 us.
#include <algorithm>
#include <type_traits>

#include "ops_internal.h"

namespace sherry {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------- element access
template <typename T, int V> struct Raw;
template <> struct Raw<uint16_t, 8> { typedef uint4 type; };
template <> struct Raw<float, 4> { typedef float4 type; };
template <> struct Raw<uint16_t, 1> { typedef uint16_t type; };
template <> struct Raw<float, 1> { typedef float type; };

__device__ inline void widen(const uint4& r, float (&v)[8]) {
  const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(d[i] << 16);
    v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
  }
}
__device__ inline void widen(const float4& r, float (&v)[4]) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ inline void widen(const uint16_t& r, float (&v)[1]) { v[0] = bf16_to_f32(r); }
__device__ inline void widen(const float& r, float (&v)[1]) { v[0] = r; }

__device__ inline uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

template <int V> __device__ inline void store_vec(uint16_t* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = (uint16_t)bf16_bits(v[i]);
  }
}
template <int V> __device__ inline void store_vec(float* p, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += (V % 4 == 0 ? 4 : 1)) {
    if constexpr (V % 4 == 0) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    else p[i] = v[i];
  }
}

// V consecutive parameters (norm weights, gates), fp32 or bf16
template <int V> __device__ inline void load_param(const float* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += (V % 4 == 0 ? 4 : 1)) {
    if constexpr (V % 4 == 0) {
      const float4 r = *reinterpret_cast<const float4*>(p + i);
      v[i] = r.x; v[i + 1] = r.y; v[i + 2] = r.z; v[i + 3] = r.w;
    } else {
      v[i] = p[i];
    }
  }
}
template <int V> __device__ inline void load_param(const uint16_t* p, float (&v)[V]) {
  if constexpr (V == 8) {
    widen(*reinterpret_cast<const uint4*>(p), v);
  } else if constexpr (V == 4) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xFFFF0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = bf16_to_f32(p[i]);
  }
}

// ------------------------------------------------------------------ reductions
// Sum over the wave, the same value in every lane: four steps inside rows of
// 16 lanes on the VALU, then the four rows' sums in order.
__device__ inline float wave_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));   // lane ^ 1
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));   // lane ^ 2
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, true));  // mirror in 8
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, true));  // mirror in 16
  const int i = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

// Sum over a thread group of 64 (one wave) or 256 (the workgroup).  A slot is
// written again only after another slot's barrier, which every wave reaches
// after its reads of this one: kernels that walk several rows take the slots
// of even and odd rows in turn.
template <int TPR>
__device__ inline float group_sum(float v, float (*slot)[4]) {
  v = wave_sum(v);
  if constexpr (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) (*slot)[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((*slot)[0] + (*slot)[1]) + ((*slot)[2] + (*slot)[3]);
}
template <int TPR>
__device__ inline void group_sum2(float& a, float& b, float (*slot)[8]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR == 64) return;
  if ((threadIdx.x & 63) == 0) {
    (*slot)[threadIdx.x >> 6] = a;
    (*slot)[4 + (threadIdx.x >> 6)] = b;
  }
  __syncthreads();
  a = ((*slot)[0] + (*slot)[1]) + ((*slot)[2] + (*slot)[3]);
  b = ((*slot)[4] + (*slot)[5]) + ((*slot)[6] + (*slot)[7]);
}

template <int TPR>
__device__ inline void group_sum3(float& a, float& b, float& c, float (*slot)[12]) {
  a = wave_sum(a);
  b = wave_sum(b);
  c = wave_sum(c);
  if constexpr (TPR == 64) return;
  if ((threadIdx.x & 63) == 0) {
    (*slot)[threadIdx.x >> 6] = a;
    (*slot)[4 + (threadIdx.x >> 6)] = b;
    (*slot)[8 + (threadIdx.x >> 6)] = c;
  }
  __syncthreads();
  a = ((*slot)[0] + (*slot)[1]) + ((*slot)[2] + (*slot)[3]);
  b = ((*slot)[4] + (*slot)[5]) + ((*slot)[6] + (*slot)[7]);
  c = ((*slot)[8] + (*slot)[9]) + ((*slot)[10] + (*slot)[11]);
}

__device__ inline float rnorm(float sum, float rdim, float eps) { return 1.0f / sqrtf(sum * rdim + eps); }
// r^3 m for a mean m of products with a row of norm 1 / r: r m is of the
// order of the other factor, r^3 alone would leave fp32's range at 2^43.
__device__ inline float cubed(float r, float m) { return r * (r * (r * m)); }

// Gate of (row, col): the address of its first element and whether it varies
// with the column.
struct GateAt {
  int kind;
  int64_t per;   // rows that share a gate row (SHERRY_GATE_ROWS)
};
__device__ inline int64_t gate_row(const GateAt& g, int64_t row) {
  return g.kind == SHERRY_GATE_CHANNEL ? 0 : row / g.per;
}

// --------------------------------------------------------------------- forward
template <typename T, typename W, int V, int NPT, int TPR>
__global__ __launch_bounds__(kThreads) void norm_forward(NormArgs a) {
  typedef typename Raw<T, V>::type R;
  __shared__ float red[2][4];
  const int t = threadIdx.x % TPR;
  const int64_t row = a.row0 + (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;   // whole waves; a 256-thread group always has its row
  const int dim = a.dim;
  const T* h = static_cast<const T*>(a.h) + row * dim;
  const T* y = static_cast<const T*>(a.y) + (a.y ? row * dim : 0);
  const float rdim = 1.0f / (float)dim;

  float hv[NPT][V], yv[NPT][V];
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    const int col = (j * TPR + t) * V;
    R rh{}, ry{};
    if (col < dim) {
      rh = *reinterpret_cast<const R*>(h + col);
      if (a.y) ry = *reinterpret_cast<const R*>(y + col);
    }
    widen(rh, hv[j]);
    widen(ry, yv[j]);
  }
  if (a.y) {
    float ry = 1.f;
    if (a.w_post) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NPT; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s += yv[j][e] * yv[j][e];
      ry = rnorm(group_sum<TPR>(s, &red[0]), rdim, a.eps);
    }
    const GateAt ga{a.gate_kind, a.gate_rows};
    float g1[1] = {1.f};
    if (a.gate_kind == SHERRY_GATE_TOKEN) load_param(static_cast<const T*>(a.gate) + row, g1);
    const T* grow = static_cast<const T*>(a.gate) +
                    (a.gate_kind >= SHERRY_GATE_CHANNEL ? gate_row(ga, row) * dim : 0);
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int col = (j * TPR + t) * V;
      float g[V], w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) { g[e] = g1[0]; w[e] = 1.f; }
      if (col < dim) {
        if (a.gate_kind >= SHERRY_GATE_CHANNEL) load_param(grow + col, g);
        if (a.w_post) load_param(static_cast<const W*>(a.w_post) + col, w);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) hv[j][e] = a.res_scale * hv[j][e] + g[e] * (yv[j][e] * ry * w[e]);
      if (col < dim) store_vec(static_cast<T*>(a.h_out) + row * dim + col, hv[j]);
    }
  }
  if (!a.w_pre) return;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NPT; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) s += hv[j][e] * hv[j][e];
  const float rh = rnorm(group_sum<TPR>(s, &red[1]), rdim, a.eps);
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    const int col = (j * TPR + t) * V;
    if (col >= dim) continue;
    float w[V], o[V];
    load_param(static_cast<const W*>(a.w_pre) + col, w);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = hv[j][e] * rh * w[e];
    store_vec(static_cast<T*>(a.n_out) + row * dim + col, o);
  }
}

// -------------------------------------------------------------------- backward
// Rows of one workgroup: [r0, r1) of gate sequences [q0, q1).  With one gate
// sequence (no per-sequence gate) a workgroup holds a range of its rows; with
// several it holds a part of one or some whole ones.
struct Share {
  int64_t q0, q1;
};
__device__ inline Share share_of(const NormSplit& s, int64_t b) {
  if (s.seqs_per_block == 1) return {b / s.blocks_per_seq, b / s.blocks_per_seq + 1};
  const int64_t q0 = b * s.seqs_per_block;
  return {q0, q0 + s.seqs_per_block < s.seqs ? q0 + s.seqs_per_block : s.seqs};
}
__device__ inline void rows_of(const NormSplit& s, int64_t b, int64_t q, int64_t& r0, int64_t& r1) {
  r0 = q * s.seq_rows;
  r1 = r0 + s.seq_rows;
  if (s.seqs_per_block == 1) {
    r0 += b % s.blocks_per_seq * s.block_rows;
    r1 = r0 + s.block_rows < r1 ? r0 + s.block_rows : r1;
  }
}

// Rows of up to 16 channels a thread keep the norm weights in registers and
// load the next row while the current one is worked on.
template <typename T, typename W, int V, int NPT, int TPR>
__global__ __launch_bounds__(kThreads) void norm_backward(NormArgs a, NormGrads d, NormSplit sp) {
  typedef typename Raw<T, V>::type R;
  constexpr int kGroups = kThreads / TPR;
  constexpr bool kHold = NPT * V <= 16;
  __shared__ float red1[2][4], red2[4][8], red3[2][12];
  __shared__ float join[kGroups > 1 ? kGroups : 1][kGroups > 1 ? TPR * V : 1];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int dim = a.dim;
  const float rdim = 1.0f / (float)dim;
  const bool post = a.w_post != nullptr, has_y = a.y != nullptr, pre = a.w_pre != nullptr;
  const bool col_gate = a.gate_kind >= SHERRY_GATE_CHANNEL;
  const bool elem_gate = a.gate_kind == SHERRY_GATE_ROWS && a.gate_rows == 1;
  const bool sum_gate = col_gate && !elem_gate;   // summed over rows
  const GateAt ga{a.gate_kind, a.gate_rows};

  auto load_weights = [&](int j, float (&w)[V], float (&wp)[V]) {
    const int col = (j * TPR + t) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) { w[e] = 1.f; wp[e] = 0.f; }
    if (col < dim) {
      if (post) load_param(static_cast<const W*>(a.w_post) + col, w);
      if (pre) load_param(static_cast<const W*>(a.w_pre) + col, wp);
    }
  };
  float w_held[kHold ? NPT : 1][V], wp_held[kHold ? NPT : 1][V];
  if constexpr (kHold)
#pragma unroll
    for (int j = 0; j < NPT; ++j) load_weights(j, w_held[j], wp_held[j]);

  struct Row {
    R h[NPT], y[NPT], d[NPT], n[NPT];
    T tok;
  };
  auto load_row = [&](Row& x, int64_t row) {
    const int64_t at = row * dim;
    if (a.gate_kind == SHERRY_GATE_TOKEN) x.tok = static_cast<const T*>(a.gate)[row];
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int col = (j * TPR + t) * V;
      x.h[j] = R{}; x.y[j] = R{}; x.d[j] = R{}; x.n[j] = R{};
      if (col < dim) {
        x.h[j] = *reinterpret_cast<const R*>(static_cast<const T*>(a.h) + at + col);
        if (has_y) x.y[j] = *reinterpret_cast<const R*>(static_cast<const T*>(a.y) + at + col);
        if (d.dh_out) x.d[j] = *reinterpret_cast<const R*>(static_cast<const T*>(d.dh_out) + at + col);
        if (d.dn_out) x.n[j] = *reinterpret_cast<const R*>(static_cast<const T*>(d.dn_out) + at + col);
      }
    }
  };

  float dwpre[NPT][V], dwpost[NPT][V], dgate[NPT][V];
#pragma unroll
  for (int j = 0; j < NPT; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dwpre[j][e] = dwpost[j][e] = dgate[j][e] = 0.f;

  // sums over the workgroup's row groups, in group order, into dst[col]
  auto flush = [&](float (&acc)[NPT][V], auto* dst) {
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int col = (j * TPR + t) * V;
      if constexpr (kGroups > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) join[group][t * V + e] = acc[j][e];
        __syncthreads();
        if (group == 0)
#pragma unroll
          for (int g = 1; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[j][e] += join[g][t * V + e];
      }
      if (group == 0 && col < dim) store_vec(dst + col, acc[j]);
    }
  };

  auto y_squares = [&](const Row& x) {   // this thread's part of sum(y^2)
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      float yv[V];
      widen(x.y[j], yv);
#pragma unroll
      for (int e = 0; e < V; ++e) s += yv[e] * yv[e];
    }
    return s;
  };
  auto load_gate = [&](int j, int64_t row, float (&g)[V]) {   // of a column gate
    const int col = (j * TPR + t) * V;
    if (col_gate && col < dim) load_param(static_cast<const T*>(a.gate) + gate_row(ga, row) * dim + col, g);
  };

  const int64_t b = blockIdx.x;
  const Share sh = share_of(sp, b);
  int odd = 0;
  for (int64_t q = sh.q0; q < sh.q1; ++q) {
    int64_t r0, r1;
    rows_of(sp, b, q, r0, r1);
    Row x;
    float gate[kHold ? NPT : 1][V];   // the same for all rows of a sequence
#pragma unroll
    for (int j = 0; j < (kHold ? NPT : 1); ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) gate[j][e] = 1.f;
    float s_yy = 0.f;                 // kHold: sum(y^2) of the row at hand, taken with the last row's sums
    if (kHold && r0 + group < r1) {
      load_row(x, r0 + group);
#pragma unroll
      for (int j = 0; j < NPT; ++j) load_gate(j, r0, gate[kHold ? j : 0]);
      if (post) {
        s_yy = group_sum<TPR>(y_squares(x), &red1[odd]);
        odd ^= 1;
      }
    }
    for (int64_t base = r0; base < r1; base += kGroups, odd ^= 1) {
      const int64_t row = base + group;
      if (kGroups > 1 && row >= r1) continue;   // a wave by itself: no barrier in its row
      Row ahead;
      const bool more = row + kGroups < r1;
      if constexpr (kHold) {
        if (more) load_row(ahead, row + kGroups);
      } else {
        load_row(x, row);
        if (post) s_yy = group_sum<TPR>(y_squares(x), &red1[odd]);
      }
      const int64_t at = row * dim;
      const float r_y = post ? rnorm(s_yy, rdim, a.eps) : 1.f;
      float tok[1] = {1.f};
      if (a.gate_kind == SHERRY_GATE_TOKEN) load_param(&x.tok, tok);

      // h' and the sums of its norm's gradient
      float h2[NPT][V];
      float s_hh = 0.f, s_uh = 0.f;
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        float w_[V], wp_[V], yv[V], nv[V];
        float (&g)[V] = gate[kHold ? j : 0];
        if constexpr (!kHold) {
          load_gate(j, row, g);
          load_weights(j, w_, wp_);
        }
        const float (&w)[V] = kHold ? w_held[kHold ? j : 0] : w_;
        const float (&wp)[V] = kHold ? wp_held[kHold ? j : 0] : wp_;
        widen(x.h[j], h2[j]);
        widen(x.y[j], yv);
        widen(x.n[j], nv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (has_y) h2[j][e] = a.res_scale * h2[j][e] + tok[0] * g[e] * (yv[e] * r_y * w[e]);
          s_hh += h2[j][e] * h2[j][e];
          s_uh += wp[e] * nv[e] * h2[j][e];
        }
      }
      float r_h = 0.f, c_h = 0.f;
      if (pre) {
        group_sum2<TPR>(s_hh, s_uh, &red2[odd]);
        r_h = rnorm(s_hh, rdim, a.eps);
        c_h = cubed(r_h, s_uh * rdim);
      }
      // t and what follows from it
      float v[NPT][V];
      float s_vy = 0.f, s_tp = 0.f;
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        const int col = (j * TPR + t) * V;
        float w_[V], wp_[V], yv[V], nv[V], dv[V], tv[V], eg[V];
        float (&g)[V] = gate[kHold ? j : 0];
        if constexpr (!kHold) {
          load_gate(j, row, g);
          load_weights(j, w_, wp_);
        }
        const float (&w)[V] = kHold ? w_held[kHold ? j : 0] : w_;
        const float (&wp)[V] = kHold ? wp_held[kHold ? j : 0] : wp_;
        widen(x.y[j], yv);
        widen(x.n[j], nv);
        widen(x.d[j], dv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float yh = yv[e] * r_y;
          tv[e] = dv[e];
          if (pre) {
            tv[e] += r_h * (wp[e] * nv[e]) - c_h * h2[j][e];
            dwpre[j][e] += nv[e] * (h2[j][e] * r_h);
          }
          const float tp = tv[e] * (yh * w[e]);
          eg[e] = tp;
          dgate[j][e] += tp;
          s_tp += tp;
          const float qv = tv[e] * (tok[0] * g[e]);
          dwpost[j][e] += qv * yh;
          v[j][e] = qv * w[e];
          s_vy += v[j][e] * yv[e];
          tv[e] *= a.res_scale;
        }
        if (col < dim) {
          store_vec(static_cast<T*>(d.dh) + at + col, tv);
          if (elem_gate) store_vec(static_cast<T*>(d.dgate) + at + col, eg);
        }
      }
      if (has_y) {
        if constexpr (kHold) {
          s_yy = post && more ? y_squares(ahead) : 0.f;
          group_sum3<TPR>(s_vy, s_tp, s_yy, &red3[odd]);
        } else {
          group_sum2<TPR>(s_vy, s_tp, &red2[2 + odd]);
        }
        if (a.gate_kind == SHERRY_GATE_TOKEN && t == 0) {
          const float g1[1] = {s_tp};
          store_vec(static_cast<T*>(d.dgate) + row, g1);
        }
        const float c_y = post ? cubed(r_y, s_vy * rdim) : 0.f;
#pragma unroll
        for (int j = 0; j < NPT; ++j) {
          const int col = (j * TPR + t) * V;
          float yv[V];
          widen(x.y[j], yv);
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (post) v[j][e] = r_y * v[j][e] - c_y * yv[e];
          if (col < dim) store_vec(static_cast<T*>(d.dy) + at + col, v[j]);
        }
      }
      if constexpr (kHold) x = ahead;
    }
    if (sum_gate && (sp.seqs_per_block > 1 || sp.blocks_per_seq == 1)) {   // this workgroup holds all its rows
      flush(dgate, static_cast<T*>(d.dgate) + q * dim);
#pragma unroll
      for (int j = 0; j < NPT; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) dgate[j][e] = 0.f;
    }
  }
  if (pre) flush(dwpre, d.part_pre + b * dim);
  if (post) flush(dwpost, d.part_post + b * dim);
  if (sum_gate && sp.seqs_per_block == 1 && sp.blocks_per_seq > 1) flush(dgate, d.part_gate + b * dim);
}

// Column sums of the workgroups' partials, in workgroup order: 32 columns by 8
// slices of the workgroups.  blockIdx.y: dw_pre, dw_post, then the gate's
// sequences.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_join(NormArgs a, NormGrads d, NormSplit sp) {
  __shared__ float part[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int slice = threadIdx.x >> 5;
  const int which = blockIdx.y;
  const float* src = which == 0 ? d.part_pre : which == 1 ? d.part_post : d.part_gate;
  if (!src) {   // no gradient came from the norm before the next block
    if (which == 0 && d.dw_pre && slice == 0 && col < a.dim) store_vec(static_cast<W*>(d.dw_pre) + col, {0.f});
    return;
  }
  const int64_t q = which < 2 ? 0 : which - 2;
  const int64_t blocks = which < 2 ? sp.blocks : sp.blocks_per_seq;
  src += q * sp.blocks_per_seq * a.dim;
  const int64_t per = (blocks + 7) / 8;
  const int64_t b0 = slice * per, b1 = b0 + per < blocks ? b0 + per : blocks;
  float s = 0.f;
  if (col < a.dim) {
    int64_t b = b0;
    for (; b + 8 <= b1; b += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[(b + i) * a.dim + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; b < b1; ++b) s += src[b * a.dim + col];
  }
  part[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice != 0 || col >= a.dim) return;
  for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
  const float v[1] = {s};
  if (which == 0) store_vec(static_cast<W*>(d.dw_pre) + col, v);
  else if (which == 1) store_vec(static_cast<W*>(d.dw_post) + col, v);
  else store_vec(static_cast<T*>(d.dgate) + q * a.dim + col, v);
}

// ------------------------------------------------- rows longer than registers
// One workgroup a row, each pass reading the row again (from L2 after the first).
template <typename T>
__device__ inline float at1(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <typename T>
__device__ inline void put1(void* p, int64_t i, float v) {
  if constexpr (sizeof(T) == 2) static_cast<uint16_t*>(p)[i] = (uint16_t)bf16_bits(v);
  else static_cast<float*>(p)[i] = v;
}
template <typename T>
__device__ inline float gate_at(const NormArgs& a, int64_t row, int64_t col) {
  if (a.gate_kind == SHERRY_GATE_NONE) return 1.f;
  if (a.gate_kind == SHERRY_GATE_TOKEN) return at1<T>(a.gate, row);
  return at1<T>(a.gate, gate_row(GateAt{a.gate_kind, a.gate_rows}, row) * a.dim + col);
}
template <typename T, typename W>
__device__ inline float h2_at(const NormArgs& a, int64_t row, int64_t col, float r_y) {
  const float h = at1<T>(a.h, row * a.dim + col);
  if (!a.y) return h;
  const float w = a.w_post ? at1<W>(a.w_post, col) : 1.f;
  return a.res_scale * h + gate_at<T>(a, row, col) * (at1<T>(a.y, row * a.dim + col) * r_y * w);
}

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_forward_long(NormArgs a) {
  __shared__ float red[2][4];
  const int64_t row = a.row0 + blockIdx.x;
  const float rdim = 1.0f / (float)a.dim;
  float r_y = 1.f;
  if (a.w_post) {
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
      const float v = at1<T>(a.y, row * a.dim + c);
      s += v * v;
    }
    r_y = rnorm(group_sum<256>(s, &red[0]), rdim, a.eps);
  }
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
    const float v = h2_at<T, W>(a, row, c, r_y);
    s += v * v;
    if (a.y) put1<T>(a.h_out, row * a.dim + c, v);
  }
  if (!a.w_pre) return;
  const float r_h = rnorm(group_sum<256>(s, &red[1]), rdim, a.eps);
  for (int64_t c = threadIdx.x; c < a.dim; c += kThreads)
    put1<T>(a.n_out, row * a.dim + c, h2_at<T, W>(a, row, c, r_y) * r_h * at1<W>(a.w_pre, c));
}

template <typename T, typename W>
__device__ inline float t_at(const NormArgs& a, const NormGrads& d, int64_t row, int64_t c, float h2, float r_h,
                             float c_h) {
  const int64_t i = row * a.dim + c;
  float t = d.dh_out ? at1<T>(d.dh_out, i) : 0.f;
  if (a.w_pre) t += r_h * (at1<W>(a.w_pre, c) * (d.dn_out ? at1<T>(d.dn_out, i) : 0.f)) - c_h * h2;
  return t;
}

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_backward_long(NormArgs a, NormGrads d) {
  __shared__ float red1[1][4], red2[2][8];
  const int64_t row = a.row0 + blockIdx.x;
  const float rdim = 1.0f / (float)a.dim;
  float r_y = 1.f, r_h = 0.f, c_h = 0.f;
  if (a.w_post) {
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
      const float v = at1<T>(a.y, row * a.dim + c);
      s += v * v;
    }
    r_y = rnorm(group_sum<256>(s, &red1[0]), rdim, a.eps);
  }
  if (a.w_pre) {
    float s_hh = 0.f, s_uh = 0.f;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
      const float h2 = h2_at<T, W>(a, row, c, r_y);
      s_hh += h2 * h2;
      if (d.dn_out) s_uh += at1<W>(a.w_pre, c) * at1<T>(d.dn_out, row * a.dim + c) * h2;
    }
    group_sum2<256>(s_hh, s_uh, &red2[0]);
    r_h = rnorm(s_hh, rdim, a.eps);
    c_h = cubed(r_h, s_uh * rdim);
  }
  float s_vy = 0.f, s_tp = 0.f;
  for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
    const float t = t_at<T, W>(a, d, row, c, h2_at<T, W>(a, row, c, r_y), r_h, c_h);
    put1<T>(d.dh, row * a.dim + c, a.res_scale * t);
    if (a.y) {
      const float y = at1<T>(a.y, row * a.dim + c), w = a.w_post ? at1<W>(a.w_post, c) : 1.f;
      s_tp += t * (y * r_y * w);
      s_vy += t * gate_at<T>(a, row, c) * w * y;
      if (a.gate_kind == SHERRY_GATE_ROWS && a.gate_rows == 1) put1<T>(d.dgate, row * a.dim + c, t * (y * r_y * w));
    }
  }
  if (a.y) {
    group_sum2<256>(s_vy, s_tp, &red2[1]);
    if (a.gate_kind == SHERRY_GATE_TOKEN && threadIdx.x == 0) put1<T>(d.dgate, row, s_tp);
    const float c_y = a.w_post ? cubed(r_y, s_vy * rdim) : 0.f;
    for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
      const float t = t_at<T, W>(a, d, row, c, h2_at<T, W>(a, row, c, r_y), r_h, c_h);
      const float w = a.w_post ? at1<W>(a.w_post, c) : 1.f;
      const float v = t * gate_at<T>(a, row, c) * w;
      put1<T>(d.dy, row * a.dim + c, a.w_post ? r_y * v - c_y * at1<T>(a.y, row * a.dim + c) : v);
    }
  }
  if (threadIdx.x == 0) {
    d.stats[row * 3] = r_y;
    d.stats[row * 3 + 1] = r_h;
    d.stats[row * 3 + 2] = c_h;
  }
}

// Column sums for those rows: a thread a column, a workgroup a share of rows.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_columns_long(NormArgs a, NormGrads d, NormSplit sp) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.dim) return;
  const int64_t b = blockIdx.y;
  const bool sum_gate = a.gate_kind == SHERRY_GATE_CHANNEL || (a.gate_kind == SHERRY_GATE_ROWS && a.gate_rows > 1);
  const float w = a.w_post ? at1<W>(a.w_post, c) : 1.f;
  float dwpre = 0.f, dwpost = 0.f, dgate = 0.f;
  const Share sh = share_of(sp, b);
  for (int64_t q = sh.q0; q < sh.q1; ++q) {
    int64_t r0, r1;
    rows_of(sp, b, q, r0, r1);
    for (int64_t row = r0; row < r1; ++row) {
      const float r_y = d.stats[row * 3], r_h = d.stats[row * 3 + 1], c_h = d.stats[row * 3 + 2];
      const float h2 = h2_at<T, W>(a, row, c, r_y);
      if (d.dn_out) dwpre += at1<T>(d.dn_out, row * a.dim + c) * (h2 * r_h);
      if (a.y) {
        const float t = t_at<T, W>(a, d, row, c, h2, r_h, c_h);
        const float yh = at1<T>(a.y, row * a.dim + c) * r_y;
        dgate += t * (yh * w);
        dwpost += t * gate_at<T>(a, row, c) * yh;
      }
    }
    if (sum_gate && (sp.seqs_per_block > 1 || sp.blocks_per_seq == 1)) {
      put1<T>(d.dgate, q * a.dim + c, dgate);
      dgate = 0.f;
    }
  }
  if (a.w_pre) d.part_pre[b * a.dim + c] = dwpre;
  if (a.w_post) d.part_post[b * a.dim + c] = dwpost;
  if (sum_gate && sp.seqs_per_block == 1 && sp.blocks_per_seq > 1) d.part_gate[b * a.dim + c] = dgate;
}

// -------------------------------------------------------------------- dispatch
// Thread groups by the row's load count: a wave for up to two 64-lane loads
// (no barrier in a row), else the workgroup with up to 32 channels a thread, 16
// where a load is one channel.  The backward kernel keeps these in 512 registers, one
// wave a SIMD, from 16 channels a thread on, and spills 60 (bf16) or 232 (fp32) bytes
// at 16 of one channel a load; the kernels of long rows, which read a row again in
// each pass, take twice that (4096 x 3001: 110 us against 215 in fp32, 84 against 206 in bf16).
template <typename T, typename W, int V, typename F>
bool with_shape(int64_t dim, F&& f) {
  const int64_t vecs = (dim + V - 1) / V;
  if (vecs <= 64) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 64>{});
  else if (vecs <= 128) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 64>{});
  else if (vecs <= 256) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 256>{});
  else if (vecs <= 512) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 256>{});
  else if (vecs <= 1024) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 256>{});
  else if (V < 8 && vecs <= 2048) f(std::integral_constant<int, V < 8 ? 8 : 4>{}, std::integral_constant<int, 256>{});
  else if (V < 4 && vecs <= 4096) f(std::integral_constant<int, V < 4 ? 16 : 4>{}, std::integral_constant<int, 256>{});
  else return false;
  return true;
}

// Kernels with a workgroup for every `per` rows: launches of at most 2^22
// workgroups each, since a launch holds fewer than 2^32 threads.
template <typename F>
hipError_t over_rows(NormArgs a, int64_t per, F&& launch) {
  constexpr int64_t kMost = (int64_t)1 << 22;
  for (; a.row0 < a.rows; a.row0 += kMost * per) {
    launch(a, dim3((unsigned)std::min(kMost, (a.rows - a.row0 + per - 1) / per)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, typename W, int V>
hipError_t forward_v(const NormArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  const bool ok = with_shape<T, W, V>(a.dim, [&](auto npt, auto tpr) {
    e = over_rows(a, kThreads / decltype(tpr)::value, [&](const NormArgs& part, dim3 grid) {
      hipLaunchKernelGGL((norm_forward<T, W, V, decltype(npt)::value, decltype(tpr)::value>), grid, dim3(kThreads), 0,
                         s, part);
    });
  });
  if (ok) return e;
  return over_rows(a, 1, [&](const NormArgs& part, dim3 grid) {
    hipLaunchKernelGGL((norm_forward_long<T, W>), grid, dim3(kThreads), 0, s, part);
  });
}

template <typename T, typename W, int V>
hipError_t backward_v(const NormArgs& a, const NormGrads& d, const NormSplit& sp, hipStream_t s) {
  if (a.rows > 0) {
    const bool ok = with_shape<T, W, V>(a.dim, [&](auto npt, auto tpr) {
      hipLaunchKernelGGL((norm_backward<T, W, V, decltype(npt)::value, decltype(tpr)::value>),
                         dim3((unsigned)sp.blocks), dim3(kThreads), 0, s, a, d, sp);
    });
    if (!ok) {
      const hipError_t e = over_rows(a, 1, [&](const NormArgs& part, dim3 grid) {
        hipLaunchKernelGGL((norm_backward_long<T, W>), grid, dim3(kThreads), 0, s, part, d);
      });
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((norm_columns_long<T, W>),
                         dim3((unsigned)((a.dim + kThreads - 1) / kThreads), (unsigned)sp.blocks), dim3(kThreads), 0,
                         s, a, d, sp);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!d.dw_pre && !a.w_post && !d.part_gate) return hipSuccess;
  hipLaunchKernelGGL((norm_join<T, W>), dim3((unsigned)((a.dim + 31) / 32), (unsigned)(2 + (d.part_gate ? sp.seqs : 0))),
                     dim3(kThreads), 0, s, a, d, sp);
  return hipGetLastError();
}

template <typename T, int V, typename F>
hipError_t by_weight(bool w_bf16, F&& f) {
  return w_bf16 ? f((uint16_t*)nullptr) : f((float*)nullptr);
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// Shares of rows for the column sums.  About 512 workgroups of 256 threads,
// each holding its columns' sums over all its rows, so the partials stay small
// against the rows themselves (8192 x 2048 bf16, 8 channels a thread, two
// workgroups a CU: 47.5 us and 5 us of joining; with 1024 workgroups 51 and 8.5).
// From 16 channels a thread on a CU holds one, and they run in two rounds.
NormSplit plan_norm_backward(int64_t rows, int64_t dim, int gate_kind, int64_t gate_rows) {
  constexpr int64_t kBlocks = 512;
  NormSplit s{};
  s.seq_rows = gate_kind == SHERRY_GATE_ROWS ? gate_rows : rows;
  s.seqs = s.seq_rows > 0 ? rows / s.seq_rows : 0;
  if (rows == 0) return s;
  const int64_t want = (rows + kBlocks - 1) / kBlocks;
  s.block_rows = std::max<int64_t>(want, dim <= 1024 ? 4 : 1);   // one row a wave for short rows
  if (s.seq_rows >= s.block_rows) {
    s.seqs_per_block = 1;
    s.blocks_per_seq = (s.seq_rows + s.block_rows - 1) / s.block_rows;
    s.blocks = s.seqs * s.blocks_per_seq;
  } else {
    s.seqs_per_block = s.block_rows / s.seq_rows;
    s.blocks_per_seq = 1;
    s.blocks = (s.seqs + s.seqs_per_block - 1) / s.seqs_per_block;
  }
  return s;
}

NormBackwardWs norm_backward_ws(const NormSplit& s, int64_t rows, int64_t dim, int gate_kind, int64_t gate_rows) {
  NormBackwardWs w{};
  const size_t part = (((size_t)s.blocks * (size_t)dim * sizeof(float)) + 15) & ~(size_t)15;
  const bool gate = (gate_kind == SHERRY_GATE_CHANNEL || (gate_kind == SHERRY_GATE_ROWS && gate_rows > 1)) &&
                    s.seqs_per_block == 1 && s.blocks_per_seq > 1;
  w.pre = 0;
  w.post = part;
  w.gate = gate ? 2 * part : 0;
  w.stats = (gate ? 3 : 2) * part;
  w.bytes = w.stats + (size_t)rows * 3 * sizeof(float);
  return w;
}

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool w_bf16, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int vec = bf16 ? 8 : 4;
  const bool v = a.dim % vec == 0 && aligned(a.h) && aligned(a.y) && aligned(a.w_post) && aligned(a.w_pre) &&
                 aligned(a.gate) && aligned(a.h_out) && aligned(a.n_out);
#define SHERRY_NORM_FWD(T, VV)                                                            \
  return by_weight<T, VV>(w_bf16, [&](auto* w) {                                          \
    return forward_v<T, typename std::remove_pointer<decltype(w)>::type, VV>(a, s); })
  if (bf16) {
    if (v) SHERRY_NORM_FWD(uint16_t, 8);
    SHERRY_NORM_FWD(uint16_t, 1);
  }
  if (v) SHERRY_NORM_FWD(float, 4);
  SHERRY_NORM_FWD(float, 1);
#undef SHERRY_NORM_FWD
}

hipError_t launch_norm_backward(const NormArgs& a, const NormGrads& d, const NormSplit& sp, bool bf16, bool w_bf16,
                                hipStream_t s) {
  const int vec = bf16 ? 8 : 4;
  const bool v = a.dim % vec == 0 && aligned(a.h) && aligned(a.y) && aligned(a.w_post) && aligned(a.w_pre) &&
                 aligned(a.gate) && aligned(d.dh_out) && aligned(d.dn_out) && aligned(d.dh) && aligned(d.dy) &&
                 aligned(d.dgate);
#define SHERRY_NORM_BWD(T, VV)                                                            \
  return by_weight<T, VV>(w_bf16, [&](auto* w) {                                          \
    return backward_v<T, typename std::remove_pointer<decltype(w)>::type, VV>(a, d, sp, s); })
  if (bf16) {
    if (v) SHERRY_NORM_BWD(uint16_t, 8);
    SHERRY_NORM_BWD(uint16_t, 1);
  }
  if (v) SHERRY_NORM_BWD(float, 4);
  SHERRY_NORM_BWD(float, 1);
#undef SHERRY_NORM_BWD
}

}  // namespace sherry
