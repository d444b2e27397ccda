// Packed products of few tokens with what follows them in one launch, and a
// mixture-of-experts layer of packed experts.
//
// One tile product serves them: a wave multiplies the tokens (the 16 rows of
// v_mfma_f32_16x16x32_bf16's A operand) with 16-row tiles of a packed weight
// (the B operand, decoded through a 32-entry LDS table as in the decode
// product), lane (r, q) of it holding row r's nibble dword q, sign dword and
// scale, straight from memory into registers.  The waves of a workgroup split
// K (or the experts' K) and join through LDS in wave order, so sums have one
// order and a product needs neither partials in memory nor a second launch;
// only the experts' second products, past 64 superblocks, are split over
// workgroups too and joined by a launch of their own.
//
// Latency bounds nearly all of it: the weights of 1 x 2048 x 2048 are read in
// 0.15 us at a copy's rate, and a launch that waits for one load from memory
// takes 3.5 us.  What carries it is many short workgroups whose loads are all
// issued at once, and few launches.
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
  uint32_t row_step;  // bytes from one row's scale to the next: 4, or 0 (one for the weight)
};
__device__ inline Planes planes(const uint8_t* packed, const float* alpha, int64_t n, int64_t k, int gran,
                                int group_sbs) {
  return Planes{packed, packed + nibble_plane_bytes(n, k), alpha, n, gran == SHERRY_PER_GROUP ? group_sbs : 0,
                gran == SHERRY_PER_TENSOR ? 0u : 4u};
}

__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kBufferWord3);
}
constexpr uint32_t kNowhere = 1u << 31;   // an offset outside every buffer here: reads zeros, without traffic

struct Block {   // one superblock's slices of the planes and scales
  __amdgpu_buffer_rsrc_t nib, sgn, al;
};
__device__ inline Block block(const Planes& p, int sb) {
  const uint32_t n = (uint32_t)p.n;
  const int group = p.group_sbs == 0 ? 0 : p.group_sbs == 1 ? sb : sb / p.group_sbs;
  return Block{buffer(p.nib + (int64_t)sb * p.n * 16, n * 16u), buffer(p.sgn + (int64_t)sb * p.n * 4, n * 4u),
               buffer(p.alpha + group * p.n, n * 4u)};   // (one scale for the weight: only the first is read)
}

// Records of one superblock of TR row tiles, as loaded and as the products take them: lane (r, q) of tile i has
// nibble dword q, the sign dword and the scale of its row r.  Buffer loads, so that the loads of
// an item past the end (rows nowhere) are issued like any other and cost no
// traffic: the compiler can then count what is in flight, which a branch around them prevents.
template <int TR>
struct TileRecords {
  uint32_t nib[TR], sgn[TR];
  float al[TR];
};
// One and two tiles: each lane loads its own words.
template <int TR>
struct Records {
  uint32_t nib[TR], sgn[TR];
  float al[TR];
  __device__ void load(const Block& b, const uint32_t (&row)[TR], uint32_t row_step, int q) {
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      nib[i] = __builtin_amdgcn_raw_buffer_load_b32(b.nib, row[i] * 16u + q * 4u, 0, 0);
      sgn[i] = __builtin_amdgcn_raw_buffer_load_b32(b.sgn, row[i] * 4u, 0, 0);
      al[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b.al, row[i] * row_step, 0, 0));
    }
  }
  __device__ TileRecords<TR> tiles() const {
    TileRecords<TR> r;
#pragma unroll
    for (int i = 0; i < TR; ++i) r.nib[i] = nib[i], r.sgn[i] = sgn[i], r.al[i] = al[i];
    return r;
  }
};
// Four tiles: lane (r, q) loads the whole record of row r of tile q (three loads of 1 KB and 256 bytes instead of
// twelve), and the 4 x 4 words of four lanes change places: M[q][word] to M[tile][q].
template <>
struct Records<4> {
  u32x4 nib;
  uint32_t sgn, al;
  __device__ void load(const Block& b, const uint32_t (&row)[1], uint32_t row_step, int) {
    nib = __builtin_amdgcn_raw_buffer_load_b128(b.nib, row[0] * 16u, 0, 0);
    sgn = __builtin_amdgcn_raw_buffer_load_b32(b.sgn, row[0] * 4u, 0, 0);
    al = __builtin_amdgcn_raw_buffer_load_b32(b.al, row[0] * row_step, 0, 0);
  }
  // halves, and odd with even rows of 16 lanes, change places
  __device__ static void swap32(uint32_t& a, uint32_t& b) {
    const auto v = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = v[0], b = v[1];
  }
  __device__ static void swap16(uint32_t& a, uint32_t& b) {
    const auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = v[0], b = v[1];
  }
  __device__ static void spread(uint32_t v, uint32_t (&w)[4]) {   // row q of 16 lanes to every row of w[q]
    w[0] = w[2] = v;
    swap32(w[0], w[2]);
    w[1] = w[0], w[3] = w[2];
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
  }
  __device__ TileRecords<4> tiles() const {
    TileRecords<4> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.nib[i] = nib[i];
    swap32(r.nib[0], r.nib[2]);
    swap32(r.nib[1], r.nib[3]);
    swap16(r.nib[0], r.nib[1]);
    swap16(r.nib[2], r.nib[3]);
    spread(sgn, r.sgn);
    uint32_t a[4];
    spread(al, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.al[i] = __uint_as_float(a[i]);
    return r;
  }
};
// A lane's rows of TR tiles whose row of tile i is row_of(i, r); kNoRow: its offsets lie outside every plane.
constexpr uint32_t kNoRow = 1u << 27;
template <int TR> constexpr int kRowsOf = TR == 4 ? 1 : TR;
template <int TR, typename F>
__device__ inline void lane_rows(F row_of, int r, int q, uint32_t (&row)[kRowsOf<TR>]) {
#pragma unroll
  for (int i = 0; i < kRowsOf<TR>; ++i) row[i] = row_of(TR == 4 ? q : i, r);
}
// A superblock of one token's bf16 values: lane (r, q)'s k = 32 t + 8 q .. + 7.
__device__ inline void load_tokens(__amdgpu_buffer_rsrc_t x, uint32_t at, u32x4 (&xf)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) xf[t] = __builtin_amdgcn_raw_buffer_load_b128(x, at + 64u * t, 0, 0);
}

// v as the sum of bf16 terms, each the upper 8 bits of what is left: fp32's 24 bits exactly.  So what lies beyond the
// largest bf16 stays finite, and an infinity has no further terms.
constexpr int kTerms = 3;
__device__ inline void split_terms(float v, __bf16 (&term)[kTerms]) {
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    const uint32_t upper = __float_as_uint(v) & 0xFFFF0000u;
    term[t] = __builtin_bit_cast(__bf16, (uint16_t)(upper >> 16));
    v = v == __uint_as_float(upper) ? 0.f : v - __uint_as_float(upper);
  }
}

// A row's scale times the tokens' weights of an expert; One: no weights.  A weight of zero (a token that the expert
// does not serve) gives zero also where the scale is not finite: that is what the legacy product is for, at an
// ordinary one's cost (a comparison and selections took 0.4 us of moe_down's 13, with two terms of h).
struct One {};
__device__ inline float weighted(float scale, One, int) { return scale; }
__device__ inline float weighted(float scale, const f32x4& weight, int e) {
  float v;
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(v) : "v"(scale), "v"(weight[e]));
  return v;
}

// acc += scale * weight * (tokens x tile) over one superblock; the tokens' values are the sum of TERMS bf16
// terms.  Tiles take turns, so that a tile's products are not a chain that each waits for.
template <int TR, int TERMS, typename W>
__device__ inline void multiply(const Records<TR>& rec, const u32x4 (&x)[TERMS][4], const char* dtab, int q,
                                const W weight, f32x4 (&acc)[TR]) {
  const TileRecords<TR> r = rec.tiles();
  uint32_t lo[TR], hi[TR];
  f32x4 g[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    lo[i] = quad_offsets8(r.nib[i], r.sgn[i], 2 * q);
    hi[i] = quad_offsets8(r.nib[i], r.sgn[i], 2 * q + 1);
    g[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      const uint2 e0 = *reinterpret_cast<const uint2*>(dtab + __builtin_amdgcn_ubfe(lo[i], 8 * t, 8));
      const uint2 e1 = *reinterpret_cast<const uint2*>(dtab + __builtin_amdgcn_ubfe(hi[i], 8 * t, 8));
      const bf16x8 w = __builtin_bit_cast(bf16x8, u32x4{e0.x, e0.y, e1.x, e1.y});
#pragma unroll
      for (int m = TERMS - 1; m >= 0; --m)
        g[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[m][t]), w, g[i], 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < TR; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] += weighted(r.al[i], weight, e) * g[i][e];
}

// Items [j0, j1) of a wave: records through a ring of RING register sets, tokens through one of XRING; an item's
// loads are issued as soon as its set is free.  records(j, live, set), tokens(j, live, set), weight(j).
template <int TR, int TERMS, int RING, int XRING, typename R, typename X, typename W>
__device__ inline void run_items(int j0, int j1, const char* dtab, int q, R records, X tokens, W weight,
                                 f32x4 (&acc)[TR]) {
  static_assert(RING % XRING == 0, "sets of one item in step");
  if (j0 >= j1) return;
  Records<TR> rec[RING];
  u32x4 x[XRING][TERMS][4];
  const int last = j1 - 1;
#pragma unroll
  for (int d = 0; d < RING; ++d) {
    if (d < XRING) tokens(min(j0 + d, last), j0 + d < j1, x[d < XRING ? d : 0]);
    records(min(j0 + d, last), j0 + d < j1, rec[d]);
  }
  for (int j = j0;; j += RING) {
#pragma unroll
    for (int d = 0; d < RING; ++d) {
      const int at = j + d;
      multiply<TR, TERMS>(rec[d], x[d % XRING], dtab, q, weight(at), acc);
      if (at + 1 >= j1) return;
      tokens(min(at + XRING, last), at + XRING < j1, x[d % XRING]);
      records(min(at + RING, last), at + RING < j1, rec[d]);
    }
  }
}

// One output tile of a packed weight: TR row tiles (GATED: half gate rows, half the same outputs' rows of the
// weight's second half).  The waves split K; a wave issues all its loads at once where it has up to XS superblocks
// (0: more, through a ring), and the waves join through LDS: wave_sums adds them in order.  Short workgroups, eight
// waves a SIMD, hide the latency better than ones that walk several tiles and load ahead (mixture of experts, 16
// tokens, 56 experts of 2048 x 2048, both before sets past a wave's range were left out: 18 us against 20 to 25).
template <int TR, int WAVES, bool GATED, int XS>
__device__ inline void tile_product(const Planes& p, int64_t outs, int sbs, __amdgpu_buffer_rsrc_t x, uint32_t x_lane,
                                    int64_t tile, const char* dtab, f32x4 (&part)[WAVES][TR][64]) {
  constexpr int kOut = GATED ? TR / 2 : TR, kHeld = XS > 0 ? XS : 1;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j0 = sbs * wave / WAVES, j1 = sbs * (wave + 1) / WAVES;
  uint32_t row[kRowsOf<TR>];
  lane_rows<TR>(
      [&](int i, int rr) {
        const int64_t col = tile * (16 * kOut) + (i % kOut) * 16 + rr;
        return col < outs ? (uint32_t)(i < kOut ? col : outs + col) : kNoRow;
      },
      r, q, row);
  f32x4 acc[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (XS > 0) {
    Records<TR> rec[kHeld];
    u32x4 xs[kHeld][1][4];
    // (a set past the wave's range repeats a superblock, without tokens, and is left out)
#pragma unroll
    for (int d = 0; d < kHeld; ++d) {
      rec[d].load(block(p, max(min(j0 + d, j1 - 1), 0)), row, p.row_step, q);
      load_tokens(x, j0 + d < j1 ? x_lane + (uint32_t)(j0 + d) * (2 * kSuperblock) : kNowhere, xs[d][0]);
    }
    lds_barrier();   // the table is written
#pragma unroll
    for (int d = 0; d < kHeld; ++d)
      if (j0 + d < j1) multiply<TR, 1>(rec[d], xs[d], dtab, q, One{}, acc);
  } else {
    lds_barrier();
    run_items<TR, 1, 2, 2>(
        j0, j1, dtab, q,
        [&](int j, bool live, Records<TR>& to) { if (live) to.load(block(p, j), row, p.row_step, q); },
        [&](int j, bool live, u32x4 (&to)[1][4]) {
          if (live) load_tokens(x, x_lane + (uint32_t)j * (2 * kSuperblock), to[0]);
        },
        [](int) { return One{}; }, acc);
  }
#pragma unroll
  for (int i = 0; i < TR; ++i) part[wave][i][lane] = acc[i];
  lds_barrier();
}
template <int TR, int WAVES>
__device__ inline float wave_sums(const f32x4 (&part)[WAVES][TR][64], int which, int token, int c) {
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += part[w][which][(token >> 2) * 16 + c][token & 3];
  return sum;
}

// Bias, activation, gate and residual of one output; `to` its place in y.
template <bool GATED>
__device__ inline float finish_output(const LinearArgs& a, float z, float u, int64_t col, int64_t outs, int64_t to) {
  if (a.bias) z += load_float(a.bias, col, a.bias_bf16);
  z = activate(z, a.activation);
  if constexpr (GATED) {
    if (a.bias) u += load_float(a.bias, outs + col, a.bias_bf16);
    z *= u;
  }
  if (a.residual) z += a.res_scale * bf16_to_f32(a.residual[to]);
  return z;
}

// ------------------------------------------------------------ linear, 1..16 tokens
// 1 x 2048 x 2048: 3.7 us; 16 x 16384 x 2048 gated, 6.6 MB: 5.4 us (1.2 TB/s); 5 x 1001 x 8192: 7.7 us.
template <int TR, int WAVES, bool GATED, int XS>
__global__ __launch_bounds__(64 * WAVES) void linear_decode(LinearArgs a, const uint16_t* __restrict__ x, int tokens,
                                                            void* __restrict__ y, bool y_bf16) {
  static_assert(!GATED || TR % 2 == 0, "a gate tile and its other half");
  constexpr int kOut = GATED ? TR / 2 : TR;   // output tiles
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  const int64_t outs = GATED ? a.n / 2 : a.n;
  const Planes p = planes(a.packed, a.alpha, a.n, a.k, a.gran, a.group_sbs);
  // consecutive workgroups land on different XCDs: give each XCD neighbouring tiles, which share memory lines
  const int xcd = blockIdx.x & 7, share = gridDim.x >> 3, more = gridDim.x & 7;
  const int64_t tile = xcd * share + min(xcd, more) + (blockIdx.x >> 3);
  const uint32_t x_lane = r < tokens ? (uint32_t)(r * a.k + 8 * q) * 2u : kNowhere;
  tile_product<TR, WAVES, GATED, XS>(p, outs, (int)(a.k / kSuperblock), buffer(x, (uint32_t)(tokens * a.k * 2)), x_lane,
                                     tile, reinterpret_cast<const char*>(dtab), part);
  for (int o = tid; o < tokens * 16 * kOut; o += 64 * WAVES) {
    const int token = o / (16 * kOut), which = o / 16 % kOut, c = o % 16;
    const int64_t col = tile * (16 * kOut) + which * 16 + c;
    if (col >= outs) continue;
    const int64_t to = (int64_t)token * outs + col;
    const float u = GATED ? wave_sums<TR, WAVES>(part, kOut * GATED + which, token, c) : 1.f;
    const float z = finish_output<GATED>(a, wave_sums<TR, WAVES>(part, which, token, c), u, col, outs, to);
    if (y_bf16) static_cast<__bf16*>(y)[to] = (__bf16)z;
    else static_cast<float*>(y)[to] = z;
  }
}

// ------------------------------------------------------------ linear, prompts of few tiles
// More tokens than 16, in tiles of 16 by 64 weight rows a workgroup: no staging of the tokens and no partials in
// memory, so a launch of many short workgroups instead of a few long ones and a second launch (517 x 2048 x 2048:
// 15.4 us against 20.1; 64 x 2048 x 2048: 6.5 against 10.2).  A superblock's loads are waited for: the other waves of
// the SIMD cover them (loads a superblock ahead 17.0 us, two tiles of tokens a workgroup 18.6); what bounds many
// tiles is the tokens' traffic, each row block's own.
template <int WAVES, bool GATED>
__global__ __launch_bounds__(64 * WAVES) void linear_tiles(LinearArgs a, const uint16_t* __restrict__ x, int64_t m,
                                                           __bf16* __restrict__ y, int tiles_m) {
  constexpr int TR = 4, kOut = GATED ? TR / 2 : TR;
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  const int64_t outs = GATED ? a.n / 2 : a.n;
  const Planes p = planes(a.packed, a.alpha, a.n, a.k, a.gran, a.group_sbs);
  // each XCD takes neighbouring workgroups: all the tokens of a few rows
  const int xcd = blockIdx.x & 7, share = gridDim.x >> 3, more = gridDim.x & 7;
  const int id = xcd * share + min(xcd, more) + (blockIdx.x >> 3), tm = id % tiles_m, tn = id / tiles_m;
  const int64_t m0 = (int64_t)tm * 16, col0 = (int64_t)tn * (16 * kOut);
  uint32_t row[kRowsOf<TR>];
  lane_rows<TR>(
      [&](int i, int rr) {
        const int64_t col = col0 + (i % kOut) * 16 + rr;
        return col < outs ? (uint32_t)(i < kOut ? col : outs + col) : kNoRow;
      },
      r, q, row);
  const uint32_t x_lane = m0 + r < m ? (uint32_t)((m0 + r) * a.k + 8 * q) * 2u : kNowhere;
  const auto xb = buffer(x, (uint32_t)(m * a.k * 2));
  f32x4 acc[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int sbs = (int)(a.k / kSuperblock), j0 = sbs * wave / WAVES, j1 = sbs * (wave + 1) / WAVES;
  Records<TR> rec;
  u32x4 xf[4];
  auto load = [&](int j) {
    rec.load(block(p, j), row, p.row_step, q);
    load_tokens(xb, x_lane + (uint32_t)j * (2 * kSuperblock), xf);
  };
  if (j0 < j1) load(j0);
  lds_barrier();   // the table is written
  for (int j = j0; j < j1; ++j) {
    const TileRecords<TR> rt = rec.tiles();
    const char* tab = reinterpret_cast<const char*>(dtab);
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      const uint32_t lo = quad_offsets8(rt.nib[i], rt.sgn[i], 2 * q), hi = quad_offsets8(rt.nib[i], rt.sgn[i], 2 * q + 1);
      f32x4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint2 e0 = *reinterpret_cast<const uint2*>(tab + __builtin_amdgcn_ubfe(lo, 8 * s, 8));
        const uint2 e1 = *reinterpret_cast<const uint2*>(tab + __builtin_amdgcn_ubfe(hi, 8 * s, 8));
        const bf16x8 w = __builtin_bit_cast(bf16x8, u32x4{e0.x, e0.y, e1.x, e1.y});
        g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xf[s]), w, g, 0, 0, 0);
      }
      acc[i] += rt.al[i] * g;
    }
    if (j + 1 < j1) load(j + 1);
  }
#pragma unroll
  for (int i = 0; i < TR; ++i) part[wave][i][lane] = acc[i];
  lds_barrier();
  for (int i = wave; i < kOut; i += WAVES) {   // four tokens of an output a lane
    const int64_t col = col0 + i * 16 + r;
    if (col >= outs) continue;
    f32x4 z = part[0][i][lane], u = {1.f, 1.f, 1.f, 1.f};
    if constexpr (GATED) u = part[0][kOut + i][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      z += part[w][i][lane];
      if constexpr (GATED) u += part[w][kOut + i][lane];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t token = m0 + 4 * q + e;
      if (token < m) y[token * outs + col] = (__bf16)finish_output<GATED>(a, z[e], u[e], col, outs, token * outs + col);
    }
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

// Reductions over a wave (the result in every lane): within rows of 16 lanes, then across them.
template <int CTRL, typename F>
__device__ inline uint32_t dpp_step(uint32_t v, uint32_t none, F f) {
  return f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, 0xF, 0xF, false));
}
template <typename F>
__device__ inline uint32_t wave_reduce(uint32_t v, uint32_t none, F f) {
  v = dpp_step<0x111>(v, none, f);   // row_shr 1, 2, 4, 8
  v = dpp_step<0x112>(v, none, f);
  v = dpp_step<0x114>(v, none, f);
  v = dpp_step<0x118>(v, none, f);
  v = dpp_step<0x142>(v, none, f);   // row_bcast 15, 31
  v = dpp_step<0x143>(v, none, f);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline uint32_t wave_max_u32(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ inline float wave_maxf(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0xFF800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ inline float wave_sumf(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
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
__device__ inline void load_keys(const MoeArgs& a, const float* logits, int parts, int64_t part_step, int lane,
                                 Keys<R>& k) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 64 + lane;
    float v[kMoeParts], sum = 0.f;
#pragma unroll
    for (int p = 0; p < kMoeParts; ++p) v[p] = e < a.experts && p < parts ? logits[p * part_step + e] : 0.f;
#pragma unroll
    for (int p = 0; p < kMoeParts; ++p) sum += v[p];
    k.logit[i] = e < a.experts ? sum : -INFINITY;
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
// Router logits of a tile of 16 experts on MFMA (A: the tokens, B: the router's rows): 32-channel steps [s0, s1),
// consecutive ones, so that a row's memory lines are read whole.  A float32 router goes in as three bf16 terms (24
// bits).
template <bool R_BF16>
__device__ inline f32x4 logit_tile(const MoeArgs& a, int tile, int s0, int s1, int lane) {
  constexpr int kAhead = R_BF16 ? 8 : 4;
  const int r = lane & 15, q = lane >> 4;
  const uint16_t* xr = a.x + (int64_t)r * a.dim + 8 * q;
  const int64_t rr = (int64_t)min(tile * 16 + r, a.experts - 1) * a.dim + 8 * q;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; s += kAhead) {
    u32x4 xv[kAhead], w[kAhead][R_BF16 ? 1 : 2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = s + u < s1;
      xv[u] = in && r < a.tokens ? *reinterpret_cast<const u32x4*>(xr + (int64_t)(s + u) * 32) : u32x4{0u, 0u, 0u, 0u};
      const int64_t at = rr + (int64_t)(s + u) * 32;
      if constexpr (R_BF16) {
        w[u][0] = in ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.router) + at) : u32x4{0u, 0u, 0u, 0u};
      } else {
        const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const float*>(a.router) + at);
        w[u][0] = in ? src[0] : u32x4{0u, 0u, 0u, 0u};
        w[u][R_BF16 ? 0 : 1] = in ? src[1] : u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u >= s1) continue;
      const bf16x8 xb = __builtin_bit_cast(bf16x8, xv[u]);
      if constexpr (R_BF16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, __builtin_bit_cast(bf16x8, w[u][0]), acc, 0, 0, 0);
      } else {
        bf16x8 term[kTerms];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __bf16 of[kTerms];
          split_terms(__uint_as_float(w[u][R_BF16 ? 0 : e / 4][e % 4]), of);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) term[t][e] = of[t];
        }
#pragma unroll
        for (int t = kTerms - 1; t >= 0; --t) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, term[t], acc, 0, 0, 0);
      }
    }
  }
  return acc;
}

// Logits of many experts, in parts over the channels [part, tokens, experts]: one CU alone reads a cold router slowly
// (64 experts of 2048 channels and 16 tokens, 320 KB: 12 us), so a tile and a part a workgroup.
constexpr int kLogitWaves = 4;
template <bool R_BF16>
__global__ __launch_bounds__(64 * kLogitWaves) void moe_logits(MoeArgs a) {
  __shared__ f32x4 part[kLogitWaves][1][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int steps = (int)(a.dim / 32), share = a.parts * kLogitWaves, mine = blockIdx.y * kLogitWaves + wave;
  part[wave][0][lane] = logit_tile<R_BF16>(a, blockIdx.x, steps * mine / share, steps * (mine + 1) / share, lane);
  __syncthreads();
  const int token = tid / 16, c = tid % 16, e = blockIdx.x * 16 + c;
  if (token < a.tokens && e < a.experts)
    a.logits[((int64_t)blockIdx.y * a.tokens + token) * a.experts + e] = wave_sums<1, kLogitWaves>(part, 0, token, c);
}

// The routing of a workgroup of WAVES waves: each token's experts and weights, a token a wave, and from them the
// experts in use.  OWN: the logits (of up to 64 experts) are made here.
struct Routing {
  __attribute__((aligned(16))) int chosen[16][kMoeTopK];
  float weight[16][kMoeTopK];
  uint32_t used[kMoeExperts / 32];
};
// Logits of up to 64 experts: the waves take the tiles in turn and share the channels of each.
template <int WAVES>
__device__ inline void own_logits(const MoeArgs& a, f32x4 (*part)[64], float (*logits)[64], int tid, int wave) {
  const int tiles = a.experts <= 16 ? 1 : a.experts <= 32 ? 2 : 4, shares = WAVES / tiles;
  const int steps = (int)(a.dim / 32), tile = wave % tiles, share = wave / tiles, lane = tid & 63;
  const int s0 = steps * share / shares, s1 = steps * (share + 1) / shares;
  part[wave][lane] = a.router_bf16 ? logit_tile<true>(a, tile, s0, s1, lane) : logit_tile<false>(a, tile, s0, s1, lane);
  lds_barrier();
  for (int o = tid; o < 256 * tiles; o += 64 * WAVES) {
    const int token = o / (16 * tiles), e = o % (16 * tiles);
    float v[WAVES], sum = 0.f;   // (loaded together)
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      v[w] = w < shares ? part[w * tiles + e / 16][(token >> 2) * 16 + e % 16][token & 3] : 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += v[w];
    logits[token][e] = sum;
  }
}
// One token's experts and their weights, from its keys.
template <int R>
__device__ inline void choose(const MoeArgs& a, Keys<R>& k, int token, int lane, Routing& to) {
  int mine = -1;        // lane j: the j-th expert and its logit
  float l = -INFINITY;
  for (int j = 0; j < a.top_k; ++j) {
    const int e = take_best(k, lane);
    float v = -INFINITY;
    if (e >= 0) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i == e / 64) v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(k.logit[i]), e & 63));
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
    for (int i = 0; i < R; ++i) top = fmaxf(top, k.logit[i]);
    top = wave_maxf(top);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 64 + lane < a.experts) sum += expf(k.logit[i] - top);
    w = expf(l - top) / wave_sumf(sum);
  } else {
    w = 1.f / (1.f + expf(-l));
  }
  if (a.softmax) {   // a logit that is not a number leaves no softmax
    bool bad = false;
#pragma unroll
    for (int i = 0; i < R; ++i) bad = bad || k.logit[i] != k.logit[i];
    if (__any(bad)) w = NAN;
  }
  if (lane < a.top_k) {
    to.chosen[token][lane] = mine;
    to.weight[token][lane] = w * a.scale;
    if (mine >= 0) atomicOr(&to.used[mine / 32], 1u << (mine & 31));
  }
}
// The routing, into LDS.  scratch, logits: OWN's.
template <int R, bool OWN, int WAVES>
__device__ inline void route_tokens(const MoeArgs& a, Routing& to, f32x4 (*scratch)[64], float (*logits)[64], int tid,
                                   int wave) {
  static_assert(!OWN || R == 1, "logits of up to 64 experts");
  const int lane = tid & 63;
  if (tid < kMoeExperts / 32) to.used[tid] = 0u;
  if constexpr (OWN) own_logits<WAVES>(a, scratch, logits, tid, wave);
  lds_barrier();
  for (int token = wave; token < a.tokens; token += WAVES) {
    Keys<R> k;
    if constexpr (OWN) load_keys(a, logits[token], 1, 0, lane, k);
    else load_keys(a, a.logits + (int64_t)token * a.experts, a.parts, (int64_t)a.tokens * a.experts, lane, k);
    choose(a, k, token, lane, to);
  }
  lds_barrier();
}
// An expert's place among a token's choices (-1: not chosen) and its weight.
__device__ inline int place_of(const MoeArgs& a, const Routing& from, int expert, int token, float& w) {
  int s = -1;
  w = 0.f;
  if (token >= a.tokens) return s;
  if (expert >= a.experts) {
    w = 1.f;
    return a.top_k + expert - a.experts;
  }
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {   // (choices past top_k are not looked at)
    const int4 c = *reinterpret_cast<const int4*>(&from.chosen[token][j0]);
    if (c.x == expert) s = j0;
    if (c.y == expert && j0 + 1 < a.top_k) s = j0 + 1;
    if (c.z == expert && j0 + 2 < a.top_k) s = j0 + 2;
    if (c.w == expert && j0 + 3 < a.top_k) s = j0 + 3;
  }
  if (s >= 0) w = from.weight[token][s];
  return s;
}

// The routing in a launch of its own, one workgroup: 5.4 us for 16 tokens, 8 of 64 experts (logits made before), a
// chain of the choices, their weights and three barriers.
constexpr int kRouteWaves = 16;
template <int R, bool OWN>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route(MoeArgs a) {
  __shared__ Routing rt;
  __shared__ f32x4 part[OWN ? kRouteWaves : 1][64];
  __shared__ float logits[OWN ? 16 : 1][64];
  const int tid = threadIdx.x;
  __shared__ int list[kMoeSlots];   // the experts in use, in rising order, then the shared ones
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  route_tokens<R, OWN, kRouteWaves>(a, rt, part, logits, tid, wave);
  int count = 0;
  for (int w = 0; w < (a.experts + 31) / 32; ++w) {
    const uint32_t bits = rt.used[w];
    if (wave == 0 && lane < 32 && (bits >> lane & 1u)) list[count + __popc(bits & ((1u << lane) - 1u))] = w * 32 + lane;
    count += __popc(bits);
  }
  if (tid < a.shared) list[count + tid] = a.experts + tid;
  lds_barrier();
  const int total = count + a.shared;
  if (tid == 0) a.route->count = total;
  for (int i = tid; i < total * 16; i += 64 * kRouteWaves) {
    const int at = i / 16, token = i % 16;
    float w;
    const int s = place_of(a, rt, list[at], token, w);
    if (token == 0) a.route->list[at] = list[at];
    a.route->place[at][token] = (int8_t)s;
    a.route->weight[at][token] = w;
  }
}

// First products and the activation: h[token, place] of the blockIdx.y-th expert in use, for its tokens. h is kept as
// three bf16 terms, which together are the fp32 value: two (2^-17 of it) left a float32 y 2.5e-6 from its definition,
// three 2.2e-7 (16 tokens, 8 of 64 experts). 16 tokens, 56 of 64 experts of 2048 x 2 x 1024, 43 MB: 16.2 us (2.7
// TB/s).  Of that the LDS lookups take 6 us; without any product it took 13, without the records' loads 12.
template <int TR, int WAVES, bool GATED, int XS, bool OWN>
__global__ __launch_bounds__(64 * WAVES) void moe_up(MoeArgs a) {
  constexpr int kOut = GATED ? TR / 2 : TR;
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  __shared__ int place[16];
  __shared__ float weight[16];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int at = blockIdx.y;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  int expert, mine;
  float w;
  if constexpr (OWN) {
    __shared__ Routing rt;
    __shared__ float logits[16][64];
    route_tokens<1, true, WAVES>(a, rt, part[0], logits, tid, __builtin_amdgcn_readfirstlane(tid >> 6));
    uint32_t bits[2] = {(uint32_t)__builtin_amdgcn_readfirstlane((int)rt.used[0]),
                        (uint32_t)__builtin_amdgcn_readfirstlane((int)rt.used[1])};
    const int low = __popc(bits[0]), count = low + __popc(bits[1]);
    if (blockIdx.x == 0 && at == 0 && tid == 0) a.route->count = count + a.shared;   // (the route is for moe_down)
    if (at >= count + a.shared) return;
    if (at >= count) {
      expert = a.experts + at - count;
    } else {   // the at-th expert in use
      uint32_t left = at < low ? bits[0] : bits[1];
      for (int i = at < low ? at : at - low; i > 0; --i) left &= left - 1u;
      expert = __builtin_ctz(left) + (at < low ? 0 : 32);
    }
    mine = place_of(a, rt, expert, r, w);
    if (blockIdx.x == 0 && tid < 16) {
      if (tid == 0) a.route->list[at] = expert;
      a.route->place[at][tid] = (int8_t)mine;
      a.route->weight[at][tid] = w;
    }
  } else {
    const MoeRoute& route = *a.route;
    const int count = route.count;
    expert = route.list[at], mine = route.place[at][r], w = route.weight[at][r];   // (loaded together)
    if (at >= count) return;
  }
  if (tid < 16) place[tid] = mine, weight[tid] = w;
  const int64_t outs = a.hidden, n = GATED ? 2 * outs : outs, tile = blockIdx.x;
  const Planes p = planes(a.up + expert * a.up_bytes, a.up_alpha + expert * a.up_scales, n, a.dim, a.up_gran, a.up_group_sbs);
  const uint32_t x_lane = mine >= 0 ? (uint32_t)(r * a.dim + 8 * q) * 2u : kNowhere;
  tile_product<TR, WAVES, GATED, XS>(p, outs, (int)(a.dim / kSuperblock), buffer(a.x, (uint32_t)(a.tokens * a.dim * 2)),
                                     x_lane, tile, reinterpret_cast<const char*>(dtab), part);
  for (int o = tid; o < 256 * kOut; o += 64 * WAVES) {
    const int which = o / 256, token = o / 16 % 16, c = o % 16;
    const int to_place = place[token];
    if (to_place < 0) continue;
    float z = activate(wave_sums<TR, WAVES>(part, which, token, c), a.activation);
    if constexpr (GATED) z *= wave_sums<TR, WAVES>(part, kOut + which, token, c);
    if (weight[token] != weight[token]) z = NAN;   // also for the outputs whose scale is zero (`weighted`)
    __bf16 term[kTerms];
    split_terms(z, term);
    const int64_t to = ((int64_t)token * a.slots + to_place) * a.hidden + tile * (16 * kOut) + which * 16 + c;
#pragma unroll
    for (int t = 0; t < kTerms; ++t) a.h[t * a.h_plane + to] = term[t];
  }
}

// Second products, weighted and added over the experts in use: TR row tiles of y, one of gridDim.y ranges of the
// (expert, superblock) items; the waves share a range evenly.  A token's row of the A operand is its h of the expert
// at hand, or zeros.  Several ranges leave fp32 partials for moe_join. 16 tokens, 56 experts of 1024 x 2048, 25 MB:
// 15.7 us (1.6 TB/s; with two terms of h 13.4), each item's h (three terms of 4 KB) beside the weights' 11 KB.
__device__ inline void store_moe(const MoeArgs& a, int64_t to, float s, void* y, bool y_bf16) {
  if (a.residual) s += bf16_to_f32(a.residual[to]);
  if (y_bf16) static_cast<__bf16*>(y)[to] = (__bf16)s;
  else static_cast<float*>(y)[to] = s;
}
template <int TR, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void moe_down(MoeArgs a, void* __restrict__ y, bool y_bf16) {
  __shared__ __attribute__((aligned(16))) uint2 dtab[32];
  __shared__ f32x4 part[WAVES][TR][64];
  __shared__ int list[kMoeSlots];
  __shared__ int8_t place[kMoeSlots][16];
  __shared__ __attribute__((aligned(16))) float weight[kMoeSlots][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  if (tid < 32) dtab[tid] = decode_bf16(tid);
  const MoeRoute& route = *a.route;
  const int sbs = (int)(a.hidden / kSuperblock), items = route.count * sbs;
  const int i0 = (int)((int64_t)items * blockIdx.y / gridDim.y), i1 = (int)((int64_t)items * (blockIdx.y + 1) / gridDim.y);
  const int a0 = i0 / sbs, a1 = (i1 + sbs - 1) / sbs;
  for (int i = tid; i < (a1 - a0) * 16; i += 64 * WAVES) {
    const int at = i / 16, t = i % 16;
    place[at][t] = route.place[a0 + at][t];
    weight[at][t] = route.weight[a0 + at][t];
    if (t == 0) list[at] = route.list[a0 + at];
  }
  __syncthreads();
  const int64_t col0 = (int64_t)blockIdx.x * (16 * TR);
  uint32_t row[kRowsOf<TR>];
  lane_rows<TR>([&](int i, int rr) { return (uint32_t)col0 + i * 16 + rr; }, r, q, row);   // (dim is whole blocks of 64 rows)
  f32x4 acc[TR];
#pragma unroll
  for (int i = 0; i < TR; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto h = buffer(a.h, (uint32_t)(kTerms * a.h_plane * 2));
  run_items<TR, kTerms, 1, 1>(
      i0 + (i1 - i0) * wave / WAVES, i0 + (i1 - i0) * (wave + 1) / WAVES, reinterpret_cast<const char*>(dtab), q,
      [&](int j, bool live, Records<TR>& rec) {
        const int e = __builtin_amdgcn_readfirstlane(list[j / sbs - a0]);
        const Planes p = planes(a.down + e * a.down_bytes, a.down_alpha + e * a.down_scales, a.dim, a.hidden, a.down_gran,
                                a.down_group_sbs);
        if (live) rec.load(block(p, j % sbs), row, p.row_step, q);
      },
      [&](int j, bool live, u32x4 (&xf)[kTerms][4]) {
        const int s = place[j / sbs - a0][r];
        const uint32_t from = (uint32_t)((r * a.slots + s) * a.hidden + j % sbs * kSuperblock + 8 * q) * 2u;
        if (!live) return;
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          load_tokens(h, s >= 0 ? from + t * (uint32_t)a.h_plane * 2u : kNowhere, xf[t]);
      },
      [&](int j) { return *reinterpret_cast<const f32x4*>(&weight[j / sbs - a0][4 * q]); }, acc);
#pragma unroll
  for (int i = 0; i < TR; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  const int64_t size = (int64_t)a.tokens * a.dim;
  float* mine = a.partial + (int64_t)blockIdx.y * size;
  for (int o = tid; o < a.tokens * 16 * TR; o += 64 * WAVES) {
    const int token = o / (16 * TR), c = o % (16 * TR);
    const float s = wave_sums<TR, WAVES>(part, c / 16, token, c % 16);
    const int64_t to = (int64_t)token * a.dim + col0 + c;
    if (gridDim.y == 1) store_moe(a, to, s, y, y_bf16);
    else mine[to] = s;
  }
}
// The ranges' partials, added in their order.  A launch of its own: letting the last range of each row block do it
// (a count that the routing clears) costs a write-back of the L2 (8 to 19 us), or saves 2 us of 22 with stores past
// the L2 whose order rests on a wait alone.
__global__ __launch_bounds__(256) void moe_join(MoeArgs a, void* __restrict__ y, bool y_bf16) {
  const int64_t size = (int64_t)a.tokens * a.dim, to = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (to >= size) return;
  float s = 0.f;
  for (int z = 0; z < a.ranges; z += 8) {   // 8 loads ahead of their adds
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = z + i < a.ranges ? a.partial[(z + i) * size + to] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (z + i < a.ranges) s += t[i];
  }
  store_moe(a, to, s, y, y_bf16);
}

}  // namespace

// Waves by the superblocks of K, one to four of them each at once.
#define SHERRY_TILES(RUN, SBS)          \
  do {                                  \
    if ((SBS) <= 4) RUN(4, 1);          \
    else if ((SBS) <= 8) RUN(4, 2);     \
    else if ((SBS) <= 16) RUN(8, 2);    \
    else if ((SBS) <= 32) RUN(16, 2);   \
    else if ((SBS) <= 64) RUN(16, 4);   \
    else RUN(16, 0);                    \
  } while (0)
// 64 weight rows a workgroup where that leaves work for every CU (16 x 16384 x 2048 gated: 5.4 us, with 16 + 16 rows
// 7.7); 16 (16 + 16: gate and values) where it does not (1 x 2048 x 2048: 3.7 us in 128 workgroups).
bool wide_tiles(int64_t blocks64) { return blocks64 >= 256; }

hipError_t launch_linear_decode(const LinearArgs& a, const uint16_t* x, int tokens, void* y, bool y_bf16,
                                hipStream_t s) {
  const int64_t outs = a.gated ? a.n / 2 : a.n;
  const bool wide = wide_tiles((a.n + 63) / 64);
  const int64_t tile = wide ? (a.gated ? 32 : 64) : 16;
  const dim3 grid((unsigned)((outs + tile - 1) / tile));
#define SHERRY_LINEAR_T(TR, W, G, XS) \
  hipLaunchKernelGGL((linear_decode<TR, W, G, XS>), grid, dim3(64 * W), 0, s, a, x, tokens, y, y_bf16)
#define SHERRY_LINEAR(W, XS)                          \
  do {                                                \
    if (wide && a.gated) SHERRY_LINEAR_T(4, W, true, XS);  \
    else if (wide) SHERRY_LINEAR_T(4, W, false, XS);  \
    else if (a.gated) SHERRY_LINEAR_T(2, W, true, XS);\
    else SHERRY_LINEAR_T(1, W, false, XS);            \
  } while (0)
  SHERRY_TILES(SHERRY_LINEAR, a.k / kSuperblock);
#undef SHERRY_LINEAR
#undef SHERRY_LINEAR_T
  return hipGetLastError();
}

// Workgroups of 16 tokens by 64 rows, of 8 waves where there is at most one a CU (64 x 2048 x 8192: 12.2 us, with 4
// waves 15.4), otherwise of 4 (517 x 2048 x 2048: 15.4 us, with 8 17.5).
hipError_t launch_linear_tiles(const LinearArgs& a, const uint16_t* x, int64_t m, uint16_t* y, hipStream_t s) {
  const int64_t outs = a.gated ? a.n / 2 : a.n, tile = a.gated ? 32 : 64;
  const int tiles_m = (int)((m + 15) / 16);
  const dim3 grid((unsigned)(tiles_m * ((outs + tile - 1) / tile)));
  __bf16* to = reinterpret_cast<__bf16*>(y);
#define SHERRY_LINEAR_TILES(W, G) \
  hipLaunchKernelGGL((linear_tiles<W, G>), grid, dim3(64 * W), 0, s, a, x, m, to, tiles_m)
  if (grid.x <= 256 && a.gated) SHERRY_LINEAR_TILES(8, true);
  else if (grid.x <= 256) SHERRY_LINEAR_TILES(8, false);
  else if (a.gated) SHERRY_LINEAR_TILES(4, true);
  else SHERRY_LINEAR_TILES(4, false);
#undef SHERRY_LINEAR_TILES
  return hipGetLastError();
}

// Router and tokens that the routing's one workgroup reads itself (64 KB: 5.4 us; 320 KB took 15.5 against 3.5 + 5.9
// with the logits in a launch of their own).
constexpr int64_t kRouteBytes = 65536;

// Up to this many workgroups the first products make a small router's routing each for itself, which saves its
// launch.  At 512, in a graph 17.6 us against 18.3 and called from Python 19.6 against 21.9 (4 tokens, 2 of 16 experts
// of 1024 x 2048); at 256, 16.6 against 18.1 and 17.2 against 19.5 (4 tokens, 4 of 32 of 512 x 512).  Many tokens are
// routed a few a wave one after another, which costs a graph more than the launch and Python less: 16 tokens, 2 of 16
// of 512 x 1024, 18.7 against 17.5 and 19.5 against 21.9; 4 of 30 of 512 x 384, 21.9 against 18.6 and 22.6 against
// 23.0.  At 1024 workgroups 22.4 against 21.3 in a graph, at 2048 32 against 25.5.
constexpr int64_t kOwnRouting = 512;

// The second products in one range of 16 waves and 16 rows a workgroup up to kNarrowItems items (4 a wave), which
// saves the joining launch (1 token; 2 of 16 experts of 4096 x 2048, 32 items: in a graph 19.5 us against 20.9; 8 of 64
// of 2048 x 1024, 64 items: 22.8 against 20.4, but called from Python 23.2 against 26.8; 2 of 8 of 2048 x 8192, 128
// items: 29.4 against 20.5).  Past it 64 rows, 8 waves and ranges of about two items a wave (2 of 8 of 2048 x 8192:
// 20.5 us, with one a wave 20.6, with four 23.4), at most 512 workgroups (16 tokens, 8 of 64 of 2048 x 1024: 40.6, with
// 256 41.6, with 1024, whose partials are twice as many, 43.9).
constexpr int kNarrowItems = 64, kDownTiles = 4, kDownWaves = 8;
MoePlan plan_moe(int tokens, int64_t dim, int64_t hidden, int experts, int shared, int top_k, bool router_bf16) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const int slots = top_k + shared;
  MoePlan p{};
  p.used = std::min(experts, tokens * top_k) + shared;
  const int64_t items = p.used * (hidden / kSuperblock);
  const int64_t blocks = dim / (16 * kDownTiles);
  p.narrow = items <= kNarrowItems;
  p.ranges = 1;
  if (!p.narrow) p.ranges = (int)std::min((items + 2 * kDownWaves - 1) / (2 * kDownWaves), (512 + blocks - 1) / blocks);
  p.h_plane = (int64_t)tokens * slots * hidden;
  p.logits_offset = up(sizeof(MoeRoute));
  const int64_t read = (experts * (router_bf16 ? 2 : 4) + tokens * 2) * dim;
  p.parts = experts <= 64 && read <= kRouteBytes ? 0 : (int)std::min<int64_t>(kMoeParts, (dim + 511) / 512);
  p.h_offset = p.logits_offset + up((size_t)p.parts * tokens * experts * 4);
  p.partial_offset = p.h_offset + up((size_t)p.h_plane * 2 * kTerms);
  p.workspace_bytes = p.partial_offset + (p.ranges > 1 ? up((size_t)p.ranges * tokens * dim * 4) : 0);
  return p;
}

hipError_t launch_moe(const MoePlan& p, MoeArgs a, void* y, bool y_bf16, hipStream_t s) {
  const dim3 wg(64 * kRouteWaves);
  hipError_t e;
  a.ranges = p.ranges;
  a.parts = p.parts;
  const bool wide = wide_tiles((a.gated ? 2 : 1) * a.hidden / 64 * p.used);
  const dim3 first((unsigned)(a.hidden / (wide ? (a.gated ? 32 : 64) : 16)), (unsigned)p.used);
  const bool own = p.parts == 0 && (int64_t)first.x * first.y <= kOwnRouting;
  if (p.parts > 0) {
    const dim3 tiles((unsigned)((a.experts + 15) / 16), (unsigned)p.parts);
    if (a.router_bf16) hipLaunchKernelGGL(moe_logits<true>, tiles, dim3(64 * kLogitWaves), 0, s, a);
    else hipLaunchKernelGGL(moe_logits<false>, tiles, dim3(64 * kLogitWaves), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!own) {
    if (p.parts == 0) hipLaunchKernelGGL((moe_route<1, true>), dim3(1), wg, 0, s, a);
    else if (a.experts <= 64) hipLaunchKernelGGL((moe_route<1, false>), dim3(1), wg, 0, s, a);
    else if (a.experts <= 128) hipLaunchKernelGGL((moe_route<2, false>), dim3(1), wg, 0, s, a);
    else hipLaunchKernelGGL((moe_route<8, false>), dim3(1), wg, 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#define SHERRY_UP_T(TR, W, G, XS)                                                                     \
  do {                                                                                                \
    if (own) hipLaunchKernelGGL((moe_up<TR, W, G, XS, true>), first, dim3(64 * W), 0, s, a);          \
    else hipLaunchKernelGGL((moe_up<TR, W, G, XS, false>), first, dim3(64 * W), 0, s, a);             \
  } while (0)
#define SHERRY_UP(W, XS)                              \
  do {                                                \
    if (wide && a.gated) SHERRY_UP_T(4, W, true, XS); \
    else if (wide) SHERRY_UP_T(4, W, false, XS);      \
    else if (a.gated) SHERRY_UP_T(2, W, true, XS);    \
    else SHERRY_UP_T(1, W, false, XS);                \
  } while (0)
  SHERRY_TILES(SHERRY_UP, a.dim / kSuperblock);
#undef SHERRY_UP
#undef SHERRY_UP_T
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.narrow)
    hipLaunchKernelGGL((moe_down<1, 16>), dim3((unsigned)(a.dim / 16)), dim3(64 * 16), 0, s, a, y, y_bf16);
  else
    hipLaunchKernelGGL((moe_down<kDownTiles, kDownWaves>), dim3((unsigned)(a.dim / (16 * kDownTiles)), (unsigned)p.ranges),
                       dim3(64 * kDownWaves), 0, s, a, y, y_bf16);
  e = hipGetLastError();
  if (e != hipSuccess || p.ranges == 1) return e;
  hipLaunchKernelGGL(moe_join, dim3((unsigned)((a.tokens * a.dim + 255) / 256)), dim3(256), 0, s, a, y, y_bf16);
  return hipGetLastError();
}

}  // namespace sherry
