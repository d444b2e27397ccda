// Packed products of 1..16 tokens with what follows them in one launch, and a
// mixture-of-experts layer of packed experts.
//
// One tile product serves them: a wave multiplies the tokens (the 16 rows of
// v_mfma_f32_16x16x32_bf16's A operand) with 16-row tiles of a packed weight
// (the B operand, decoded through a 32-entry LDS table as in the decode
// product), lane (r, q) of it holding row r's nibble dword q, sign dword and
// scale: 12 bytes a tile and superblock, straight from memory into registers.
// The waves of a workgroup split K (or the experts' K) and join through LDS in
// wave order, so a call needs neither partials in memory nor a second launch,
// and its sums have one order.
#include <algorithm>
#include <cfloat>

#include "epilogue.h"

namespace sherry {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A packed weight as the tile product reads it.
struct Planes {
  const uint8_t *nib, *sgn;
  const float* alpha;
  int64_t n;
  int group_sbs;      // superblocks of a scale group; 0: scales of a row or of the weight
  uint32_t row_step;  // scales: 1 a row, 0 one for the weight
};
__device__ inline Planes planes(const uint8_t* packed, const float* alpha, int64_t n, int64_t k, int gran,
                                int group_sbs) {
  return Planes{packed, packed + nibble_plane_bytes(n, k), alpha, n, gran == SHERRY_PER_GROUP ? group_sbs : 0,
                gran == SHERRY_PER_TENSOR ? 0u : 1u};
}

// Records of one superblock of TR row tiles.
template <int TR>
struct Records {
  uint32_t nib[TR], sgn[TR];
  float al[TR];
};
template <int TR>
__device__ inline void load_records(const Planes& p, int sb, const uint32_t (&row)[TR], int q, Records<TR>& r) {
  const uint8_t* nib = p.nib + (int64_t)sb * p.n * 16;
  const uint8_t* sgn = p.sgn + (int64_t)sb * p.n * 4;
  const int group = p.group_sbs == 0 ? 0 : p.group_sbs == 1 ? sb : sb / p.group_sbs;
  const float* al = p.alpha + group * p.n;
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    r.nib[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(nib + (row[i] * 16u + q * 4u)));
    r.sgn[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(sgn + row[i] * 4u));
    r.al[i] = al[row[i] * p.row_step];
  }
}

// acc += scale * weight * (tokens x tile) over one superblock; the tokens'
// values are the sum of TERMS bf16 terms.
template <int TR, int TERMS>
__device__ inline void multiply(const Records<TR>& r, const u32x4 (&x)[TERMS][4], const char* dtab, int q,
                                const f32x4 weight, f32x4 (&acc)[TR]) {
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const uint32_t lo = quad_offsets8(r.nib[i], r.sgn[i], 2 * q), hi = quad_offsets8(r.nib[i], r.sgn[i], 2 * q + 1);
    f32x4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint2 e0 = *reinterpret_cast<const uint2*>(dtab + __builtin_amdgcn_ubfe(lo, 8 * t, 8));
      const uint2 e1 = *reinterpret_cast<const uint2*>(dtab + __builtin_amdgcn_ubfe(hi, 8 * t, 8));
      const bf16x8 w = __builtin_bit_cast(bf16x8, u32x4{e0.x, e0.y, e1.x, e1.y});
#pragma unroll
      for (int m = TERMS - 1; m >= 0; --m)
        g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[m][t]), w, g, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] += r.al[i] * weight[e] * g[e];
  }
}

// Items [j0, j1) of a wave, DEPTH at a time, the next ones' loads under the
// current ones' products.  load(j, records, x) and weight(j); items past the
// end are not loaded.
template <int TR, int TERMS, int DEPTH, typename Load, typename Weight>
__device__ inline void run_items(int j0, int j1, const char* dtab, int q, Load load, Weight weight,
                                 f32x4 (&acc)[TR]) {
  Records<TR> rec[2][DEPTH];
  u32x4 x[2][DEPTH][TERMS][4];
  auto fetch = [&](int buf, int j) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (j + d < j1) load(j + d, rec[buf][d], x[buf][d]);
  };
  auto use = [&](int buf, int j) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (j + d < j1) multiply<TR, TERMS>(rec[buf][d], x[buf][d], dtab, q, weight(j + d), acc);
  };
  fetch(0, j0);
  for (int j = j0; j < j1; j += 2 * DEPTH) {
    fetch(1, j + DEPTH);
    use(0, j);
    fetch(0, j + 2 * DEPTH);
    use(1, j + DEPTH);
  }
}

// ------------------------------------------------------------ linear, 1..16 tokens
// Workgroup: TR row tiles (gated: the first half of them gate rows, the others
// the same outputs' rows of the second half), WAVES ranges of K.
template <int TR, int WAVES, bool GATED>
__global__ __launch_bounds__(64 * WAVES) void linear_decode(LinearArgs a, const uint16_t* __restrict__ x, int tokens,
                                                            void* __restrict__ y, bool y_bf16) {
  static_assert(!GATED || TR % 2 == 0, "a gate tile and its other half");
  constexpr int kOut = GATED ? TR / 2 : TR;   // output tiles
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  const int64_t outs = GATED ? a.n / 2 : a.n;
  const int64_t col0 = (int64_t)blockIdx.x * (16 * kOut);
  const Planes p = planes(a.packed, a.alpha, a.n, a.k, a.gran, a.group_sbs);
  uint32_t row[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int64_t col = min(col0 + (i % kOut) * 16 + r, outs - 1);   // (repeated rows are not stored)
    row[i] = (uint32_t)(i < kOut ? col : outs + col);
  }
  f32x4 acc[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const int sbs = (int)(a.k / kSuperblock);
  const int j0 = sbs * wave / WAVES, j1 = sbs * (wave + 1) / WAVES;
  const uint16_t* xr = x + (int64_t)r * a.k + 8 * q;
  run_items<TR, 1, TR == 1 ? 2 : 1>(
      j0, j1, reinterpret_cast<const char*>(dtab), q,
      [&](int j, Records<TR>& rec, u32x4 (&xf)[1][4]) {
        load_records<TR>(p, j, row, q, rec);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          xf[0][t] = r < tokens ? *reinterpret_cast<const u32x4*>(xr + (int64_t)j * kSuperblock + 32 * t)
                                : u32x4{0u, 0u, 0u, 0u};
      },
      [](int) { return f32x4{1.f, 1.f, 1.f, 1.f}; }, acc);
#pragma unroll
  for (int i = 0; i < TR; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int o = tid; o < tokens * 16 * kOut; o += 64 * WAVES) {
    const int tile = o / (16 * tokens), token = o / 16 % tokens, c = o % 16;
    const int64_t col = col0 + tile * 16 + c;
    if (col >= outs) continue;
    const int at = (token >> 2) * 16 + c, e = token & 3;
    float z = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      z += part[w][tile][at][e];
      if constexpr (GATED) u += part[w][kOut + tile][at][e];
    }
    if (a.bias) {
      z += load_float(a.bias, col, a.bias_bf16);
      if constexpr (GATED) u += load_float(a.bias, outs + col, a.bias_bf16);
    }
    z = activate(z, a.activation);
    if constexpr (GATED) z *= u;
    const int64_t to = (int64_t)token * outs + col;
    if (a.residual) z += a.res_scale * bf16_to_f32(a.residual[to]);
    if (y_bf16) static_cast<__bf16*>(y)[to] = (__bf16)z;
    else static_cast<float*>(y)[to] = z;
  }
}

// ------------------------------------------------------------ mixture of experts
// Selection keys as ordered integers: 0 taken or no expert, 1 an expert that is
// off (-infinity), 2 not a number, then the numbers in order (-0 as 0).
__device__ inline uint32_t order(float f) {
  if (f != f) return 2u;
  const uint32_t u = __float_as_uint(f + 0.f);
  if (u == 0xFF800000u) return 1u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kOff = 1u;

template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// The largest of a wave's values (in every lane): within rows of 16, then across them.
__device__ inline uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0x111>(v);   // row_shr 1, 2, 4, 8
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);   // row_bcast 15, 31
  v = dpp_max<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline float wave_maxf(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ inline float wave_sumf(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A token's keys: lane l holds experts l, l + 64, ...  Without a bias the
// logits themselves, whose order is that of their scores.
// R is the least of 1, 2 and 8 that holds the experts.
template <int R>
struct Keys {
  uint32_t key[R];
  float logit[R];
};
template <int R>
__device__ inline void load_keys(const MoeArgs& a, int token, int lane, Keys<R>& k) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 64 + lane;
    k.logit[i] = e < a.experts ? a.logits[(int64_t)token * a.experts + e] : -INFINITY;
    k.key[i] = e < a.experts ? order(k.logit[i]) : 0u;
  }
  if (!a.bias) return;
  float top = -INFINITY, sum = 0.f;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < R; ++i) top = fmaxf(top, k.logit[i]);
    top = wave_maxf(top);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 64 + lane < a.experts) sum += expf(k.logit[i] - top);
    sum = wave_sumf(sum);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 64 + lane;
    if (e >= a.experts) continue;
    const float score = a.softmax ? expf(k.logit[i] - top) / sum : 1.f / (1.f + expf(-k.logit[i]));
    k.key[i] = order(score + a.bias[e]);
  }
}
// The largest key's expert (the lowest index of equal ones), which is then
// taken; -1 where only experts that are off are left.
template <int R>
__device__ inline int take_best(Keys<R>& k, int lane) {
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) v = max(v, k.key[i]);
  const uint32_t best = wave_max_u32(v);
  if (best <= kOff) return -1;
  int e = -1;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint64_t who = __ballot(k.key[i] == best);
    if (e < 0 && who) {
      const int l = __builtin_ctzll(who);
      e = i * 64 + l;
      if (lane == l) k.key[i] = 0u;
    }
  }
  return e;
}
// Where expert e stands in the token's order; -1 beyond the top_k or off.
template <int R>
__device__ inline int rank_of(const MoeArgs& a, const Keys<R>& k, int e, int lane) {
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i == e / 64) mine = (uint32_t)__builtin_amdgcn_readlane((int)k.key[i], e & 63);
  int rank = 0;
#pragma unroll
  for (int i = 0; i < R; ++i)
    rank += __popcll(__ballot(k.key[i] > mine || (k.key[i] == mine && i * 64 + lane < e)));
  return mine > kOff && rank < a.top_k ? rank : -1;
}

// Router logits [tokens, experts]: 16 experts a workgroup on MFMA (A: the
// tokens, B: the router's rows), waves split the channels.  A float32 router
// goes in as three bf16 terms (24 bits).
constexpr int kLogitWaves = 8;
template <bool R_BF16>
__global__ __launch_bounds__(64 * kLogitWaves) void moe_logits(MoeArgs a) {
  constexpr int kAhead = 4;
  __shared__ f32x4 part[kLogitWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int e0 = blockIdx.x * 16, expert = min(e0 + r, a.experts - 1);
  const int steps = (int)(a.dim / 32);
  const uint16_t* xr = a.x + (int64_t)r * a.dim + 8 * q;
  const int64_t rr = (int64_t)expert * a.dim + 8 * q;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < steps; s += kAhead * kLogitWaves) {
    u32x4 xv[kAhead], w[kAhead][R_BF16 ? 1 : 2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = s + u * kLogitWaves;
      const bool in = at < steps;
      xv[u] = in && r < a.tokens ? *reinterpret_cast<const u32x4*>(xr + (int64_t)at * 32) : u32x4{0u, 0u, 0u, 0u};
      if constexpr (R_BF16) {
        w[u][0] = in ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.router) + rr + (int64_t)at * 32)
                     : u32x4{0u, 0u, 0u, 0u};
      } else {
        const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const float*>(a.router) + rr + (int64_t)at * 32);
        w[u][0] = in ? src[0] : u32x4{0u, 0u, 0u, 0u};
        w[u][R_BF16 ? 0 : 1] = in ? src[1] : u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u * kLogitWaves >= steps) continue;
      const bf16x8 xb = __builtin_bit_cast(bf16x8, xv[u]);
      if constexpr (R_BF16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, __builtin_bit_cast(bf16x8, w[u][0]), acc, 0, 0, 0);
      } else {
        bf16x8 term[3];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float rest = __uint_as_float(w[u][R_BF16 ? 0 : i / 4][i % 4]);
#pragma unroll
          for (int t = 0; t < 3; ++t) {
            term[t][i] = (__bf16)rest;
            rest -= (float)term[t][i];
          }
        }
#pragma unroll
        for (int t = 2; t >= 0; --t) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, term[t], acc, 0, 0, 0);
      }
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (tid < 256) {
    const int token = tid / 16, c = tid % 16;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kLogitWaves; ++w) s += part[w][(token >> 2) * 16 + c][token & 3];
    if (token < a.tokens && e0 + c < a.experts) a.logits[(int64_t)token * a.experts + e0 + c] = s;
  }
}

// First products and the activation: h[token, slot] of one expert's TR / 2 (or TR) output tiles
// for its tokens.  blockIdx.y names the expert (every expert, where the tokens' choices are as
// many), or a (token, rank) whose expert it is: the first token that chose an expert stands for
// all.  h is kept as two bf16 terms (16 bits, 2^-17 of the value, beside y's 2^-9 or the float32 sums').
template <int TR, int WAVES, bool GATED, int R>
__global__ __launch_bounds__(64 * WAVES) void moe_up(MoeArgs a) {
  constexpr int kOut = GATED ? TR / 2 : TR;
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  __shared__ int rank[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  const int y = blockIdx.y;
  int expert;
  if (y >= a.choices) {          // a shared expert: every token's
    expert = a.experts + y - a.choices;
    if (tid < 16) rank[tid] = tid < a.tokens ? a.top_k + y - a.choices : -1;
  } else {
    int first = 0;
    if (a.by_choice) {
      first = y / a.top_k;
      Keys<R> k;
      load_keys(a, first, lane, k);
      for (int j = 0; j < y % a.top_k; ++j) take_best(k, lane);
      expert = take_best(k, lane);
      if (expert < 0) return;    // (every wave finds the same)
    } else {
      expert = y;
    }
    for (int t = wave; t < 16; t += WAVES) {
      int at = -1;
      if (t < a.tokens) {
        Keys<R> k;
        load_keys(a, t, lane, k);
        at = rank_of(a, k, expert, lane);
      }
      if (lane == 0) rank[t] = at;
    }
    __syncthreads();
    bool any = false;
    for (int t = 0; t < 16; ++t) {
      if (rank[t] < 0) continue;
      if (a.by_choice && t < first) return;   // an earlier token's workgroup does it
      any = true;
    }
    if (!any) return;
  }
  __syncthreads();
  const int64_t outs = a.hidden, n = GATED ? 2 * outs : outs;
  const int64_t col0 = (int64_t)blockIdx.x * (16 * kOut);
  const Planes p = planes(a.up + expert * a.up_bytes, a.up_alpha + expert * a.up_scales, n, a.dim, a.up_gran, a.up_group_sbs);
  uint32_t row[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int64_t col = min(col0 + (i % kOut) * 16 + r, outs - 1);
    row[i] = (uint32_t)(i < kOut ? col : outs + col);
  }
  f32x4 acc[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int sbs = (int)(a.dim / kSuperblock);
  const int j0 = sbs * wave / WAVES, j1 = sbs * (wave + 1) / WAVES;
  const uint16_t* xr = a.x + (int64_t)r * a.dim + 8 * q;
  const bool mine = rank[r] >= 0;
  run_items<TR, 1, 2>(
      j0, j1, reinterpret_cast<const char*>(dtab), q,
      [&](int j, Records<TR>& rec, u32x4 (&xf)[1][4]) {
        load_records<TR>(p, j, row, q, rec);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          xf[0][t] = mine ? *reinterpret_cast<const u32x4*>(xr + (int64_t)j * kSuperblock + 32 * t)
                          : u32x4{0u, 0u, 0u, 0u};
      },
      [](int) { return f32x4{1.f, 1.f, 1.f, 1.f}; }, acc);
#pragma unroll
  for (int i = 0; i < TR; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int o = tid; o < 256 * kOut; o += 64 * WAVES) {
    const int tile = o / 256, token = o / 16 % 16, c = o % 16;
    const int64_t col = col0 + tile * 16 + c;
    if (rank[token] < 0 || col >= outs) continue;
    const int at = (token >> 2) * 16 + c, e = token & 3;
    float z = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      z += part[w][tile][at][e];
      if constexpr (GATED) u += part[w][kOut + tile][at][e];
    }
    z = activate(z, a.activation);
    if constexpr (GATED) z *= u;
    const __bf16 hi = (__bf16)z;
    const float rest = z - (float)hi;
    const int64_t to = ((int64_t)token * a.slots + rank[token]) * a.hidden + col;
    a.h[to] = hi;
    a.h[a.h_plane + to] = __builtin_isfinite(rest) ? (__bf16)rest : (__bf16)0.f;
  }
}

// Second products, weighted and added over a token's experts, 16 output
// channels a workgroup: its waves first choose (a token each), list the experts in
// use, and then share their superblocks evenly.  A token's row of the A operand is its h of
// the expert at hand, or zeros.
constexpr int kDownWaves = 16;
template <int R>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down(MoeArgs a, void* __restrict__ y, bool y_bf16) {
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[kDownWaves][64];
  __shared__ uint32_t used[kMoeExperts / 32];
  __shared__ int list[16 * kMoeTopK + kMoeShared];     // the experts in use
  __shared__ int8_t slot[16 * kMoeTopK + kMoeShared][16];
  __shared__ __attribute__((aligned(16))) float weight[16 * kMoeTopK + kMoeShared][16];
  __shared__ int chosen[16][kMoeTopK];
  __shared__ float chosen_w[16][kMoeTopK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  if (tid < kMoeExperts / 32) used[tid] = 0u;
  __syncthreads();
  if (wave < a.tokens) {
    Keys<R> k;
    load_keys(a, wave, lane, k);
    float logit[R];   // (the keys lose theirs)
#pragma unroll
    for (int i = 0; i < R; ++i) logit[i] = k.logit[i];
    int mine = -1;        // lane j: the j-th expert and its logit
    float l = -INFINITY;
    for (int j = 0; j < a.top_k; ++j) {
      const int e = take_best(k, lane);
      float v = -INFINITY;
      if (e >= 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i == e / 64) v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_int(logit[i]), e & 63));
      }
      if (lane == j) {
        mine = e;
        l = v;
      }
    }
    // weights by their logarithms, so that none is lost to the others' size
    const float g = a.softmax ? l : fminf(l, 0.f) - log1pf(expf(-fabsf(l)));
    float w;
    if (a.normalize) {
      const float top = wave_maxf(mine >= 0 ? g : -INFINITY);
      w = mine >= 0 ? expf(g - top) : 0.f;
      w /= wave_sumf(w);
    } else if (a.softmax) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) top = fmaxf(top, logit[i]);
      top = wave_maxf(top);
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i * 64 + lane < a.experts) sum += expf(logit[i] - top);
      w = expf(l - top) / wave_sumf(sum);
    } else {
      w = 1.f / (1.f + expf(-l));
    }
    if (lane < a.top_k) {
      chosen[wave][lane] = mine;
      chosen_w[wave][lane] = w * a.scale;
      if (mine >= 0) atomicOr(&used[mine / 32], 1u << (mine & 31));
    }
  }
  __syncthreads();
  // the experts in use, in rising order, then the shared ones
  int count = 0;
  for (int w = 0; w < (a.experts + 31) / 32; ++w) {
    const uint32_t bits = used[w];
    if (wave == 0 && lane < 32 && (bits >> lane & 1u)) list[count + __popc(bits & ((1u << lane) - 1u))] = w * 32 + lane;
    count += __popc(bits);
  }
  if (tid < a.shared) list[count + tid] = a.experts + tid;
  const int total = count + a.shared;
  __syncthreads();
  for (int i = tid; i < total * 16; i += 64 * kDownWaves) {
    const int at = i / 16, token = i % 16, e = list[at];
    int s = -1;
    float w = 0.f;
    if (token < a.tokens) {
      if (at >= count) {
        s = a.top_k + at - count;
        w = 1.f;
      }
      for (int j = 0; j < a.top_k && at < count; ++j)
        if (chosen[token][j] == e) {
          s = j;
          w = chosen_w[token][j];
        }
    }
    slot[at][token] = (int8_t)s;
    weight[at][token] = w;
  }
  __syncthreads();
  const int64_t col0 = (int64_t)blockIdx.x * 16;
  const uint32_t row[1] = {(uint32_t)(col0 + r)};
  const int sbs = (int)(a.hidden / kSuperblock);
  const int items = total * sbs;
  f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
  run_items<1, 2, 1>(
      items * wave / kDownWaves, items * (wave + 1) / kDownWaves, reinterpret_cast<const char*>(dtab), q,
      [&](int j, Records<1>& rec, u32x4 (&xf)[2][4]) {
        const int at = j / sbs, sb = j % sbs, e = __builtin_amdgcn_readfirstlane(list[at]);
        const Planes p = planes(a.down + e * a.down_bytes, a.down_alpha + e * a.down_scales, a.dim, a.hidden, a.down_gran,
                                a.down_group_sbs);
        load_records<1>(p, sb, row, q, rec);
        const int s = slot[at][r];
        const __bf16* h = a.h + ((int64_t)r * a.slots + s) * a.hidden + sb * kSuperblock + 8 * q;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          xf[0][t] = s >= 0 ? *reinterpret_cast<const u32x4*>(h + 32 * t) : u32x4{0u, 0u, 0u, 0u};
          xf[1][t] = s >= 0 ? *reinterpret_cast<const u32x4*>(h + a.h_plane + 32 * t) : u32x4{0u, 0u, 0u, 0u};
        }
      },
      [&](int j) { return *reinterpret_cast<const f32x4*>(&weight[j / sbs][4 * q]); }, acc);
  part[wave][lane] = acc[0];
  __syncthreads();
  if (tid < 256) {
    const int token = tid / 16, c = tid % 16;
    if (token >= a.tokens) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) s += part[w][(token >> 2) * 16 + c][token & 3];
    const int64_t to = (int64_t)token * a.dim + col0 + c;
    if (a.residual) s += bf16_to_f32(a.residual[to]);
    if (y_bf16) static_cast<__bf16*>(y)[to] = (__bf16)s;
    else static_cast<float*>(y)[to] = s;
  }
}

}  // namespace

// Tiles of a workgroup and its ranges of K: a wave takes about two tiles'
// superblocks at once, and 16 waves at most share them.
hipError_t launch_linear_decode(const LinearArgs& a, const uint16_t* x, int tokens, void* y, bool y_bf16,
                                hipStream_t s) {
  const int64_t outs = a.gated ? a.n / 2 : a.n;
  const int sbs = (int)(a.k / kSuperblock);
#define SHERRY_LINEAR(TR, W, G)                                                                             \
  hipLaunchKernelGGL((linear_decode<TR, W, G>), dim3((unsigned)((outs + 16 * (G ? TR / 2 : TR) - 1) / (16 * (G ? TR / 2 : TR)))), \
                     dim3(64 * W), 0, s, a, x, tokens, y, y_bf16)
#define SHERRY_LINEAR_W(TR, G)            \
  do {                                    \
    if (sbs >= 16) SHERRY_LINEAR(TR, 8, G);  \
    else SHERRY_LINEAR(TR, 4, G);         \
  } while (0)
  if (a.gated) SHERRY_LINEAR_W(2, true);
  else SHERRY_LINEAR_W(1, false);
#undef SHERRY_LINEAR_W
#undef SHERRY_LINEAR
  return hipGetLastError();
}

MoePlan plan_moe(int tokens, int experts, int slots, int64_t hidden) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  MoePlan p{};
  p.h_offset = up((size_t)tokens * experts * 4);
  p.h_plane = (int64_t)tokens * slots * hidden;
  p.workspace_bytes = p.h_offset + up((size_t)p.h_plane * 4);
  return p;
}

hipError_t launch_moe(MoeArgs a, void* y, bool y_bf16, hipStream_t s) {
  const dim3 routers((unsigned)((a.experts + 15) / 16));
  if (a.router_bf16) hipLaunchKernelGGL(moe_logits<true>, routers, dim3(64 * kLogitWaves), 0, s, a);
  else hipLaunchKernelGGL(moe_logits<false>, routers, dim3(64 * kLogitWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.by_choice = a.tokens * a.top_k < a.experts;
  a.choices = a.by_choice ? a.tokens * a.top_k : a.experts;
  const unsigned depth = (unsigned)(a.choices + a.shared);
#define SHERRY_MOE(R)                                                                                                    \
  do {                                                                                                                  \
    if (a.gated) hipLaunchKernelGGL((moe_up<2, 4, true, R>), dim3((unsigned)(a.hidden / 16), depth), dim3(256), 0, s, a); \
    else hipLaunchKernelGGL((moe_up<1, 4, false, R>), dim3((unsigned)(a.hidden / 16), depth), dim3(256), 0, s, a);        \
    e = hipGetLastError();                                                                                              \
    if (e != hipSuccess) return e;                                                                                      \
    hipLaunchKernelGGL(moe_down<R>, dim3((unsigned)(a.dim / 16)), dim3(64 * kDownWaves), 0, s, a, y, y_bf16);            \
  } while (0)
  if (a.experts <= 64) SHERRY_MOE(1);
  else if (a.experts <= 128) SHERRY_MOE(2);
  else SHERRY_MOE(8);
#undef SHERRY_MOE
  return hipGetLastError();
}

}  // namespace sherry
