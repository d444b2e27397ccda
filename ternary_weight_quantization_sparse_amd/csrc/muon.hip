// Orthogonalised updates of latent weights by Newton-Schulz products.
//
// For u [N, K] (X the smaller side's rows: X = u or u^T, R x L with R <= L):
//   X <- u / (|u| + eps);   per step:  A = X X^T,  X <- a X + (b A + c A A) X
// Three products a step, all of the form C[i, j] = sum_k P[i, k] Q[j, k] with
// both operands' rows contiguous along k, so X is kept twice, as rows [R, L]
// and [L, R].  A and A A are symmetric: only tiles on and above the diagonal
// are computed, each written twice.
//
// Numbers.  The steps amplify what is small in X up to a^steps ~ 485 times, so
// one 16-bit product per step loses 1e-3 to 4e-2 of the result (measured on
// Gaussian and low-rank spectra).  Every value is kept as two float16 planes,
// value * 2^13 = hi + lo (22 bits), and a product is three matrix products,
// hi hi + hi lo + lo hi, summed in fp32: the result then differs from one in
// fp32 arithmetic by no more than that differs from 64 bits.  The power of two
// puts entries down to 1 / sqrt(L) well inside float16's range (lo parts stay
// normal numbers to 2^-27) and leaves room below 8 for X, A and b A + c A A, so
// singular values of an iterate below 2.82; muon_range refuses coefficients that can leave it.
//
// Steps in groups.  All factors of X are polynomials of one matrix and commute,
// so three steps need X only at their start and end: with A = X X^T, B = b A +
// c A A, P = a I + B, the next step's A is P A P, and X <- P'' P' P X.  P'' P' P is
// kept as q I + D (the large part apart), D at 2^9: it reaches a^3.  Where L >=
// 2 R the R x R products cost less than two passes over X: 38 R^3 against 65 R^3
// flops at L = 4 R (8192 x 2048: bf16 in 1.14 ms, fp32, step by step, in 1.65).  Their roundings reach
// the result larger, up to what fp32 arithmetic loses on the same steps.  Off from 64
// bits, of the result, grouped (single steps; fp32 products): Gaussian 512 x 2048
// 3.1e-6 (1.6e-6; 3.3e-6) and 2048 x 8192 5.2e-6 (2.3e-6; 5.3e-6), rank 8 and a tail
// 1.1e-5 (1.1e-5; 3.2e-5) and 5.3e-5 (4.1e-5; 6.4e-5), rank 256 and a tail of 2048 x 8192
// 3.6e-6 (1.5e-6; 3.0e-6).  So sherry_orthogonalize takes every step of fp32
// matrices by itself; bf16 results and the update of weights, where fp32's own
// error will do, take groups.  A caller who wants single steps in an update adds the former's result.
//
// The matrix cores bound the large sizes, at the clock that their power leaves:
// 2048 x 8192 runs its products with X at 1.1 PFLOP/s of float16 (185 us each),
// the matrix cores 70% busy at 1.8 GHz; a step of an 8192 x 2048 fp32 weight takes 1.19 to 1.25
// ms by card, 0.98 PFLOP of float16 (1.68 if every step went over X).  Small ones are bound by their 15 to 17
// launches of about 5 us (256 x 512: 82 us).
#include <algorithm>
#include <cmath>
#include <utility>

#include "ops_internal.h"

namespace sherry {
namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr float kScale = 8192.f, kRScale = 1.f / 8192.f, kScaleD = 512.f;
constexpr int kBK = 16;                 // k of an LDS stage: one 64-byte piece (hi, lo) of a row
constexpr int kRowB = kBK * 4;
constexpr int kSlots = 4;               // LDS stages: one read, up to three in flight
constexpr int kGroupSteps = 3;          // steps between two looks at X, where they are taken in groups

// A split matrix of `rows` rows is kept in the order of the MFMA's operands:
// for each 16 columns and 32 rows 2 KB, 1 KB of hi values and 1 KB of lo ones,
// each as lane 32 h + r holds them: 8 columns from 8 h of row r.  A fragment
// is 1 KB of consecutive memory, a stage of a tile one consecutive run, and
// both are read from LDS without bank conflicts as they lie.
constexpr int kLo = 512;   // from a hi value to its lo one
__device__ inline int64_t split_at(int64_t row, int64_t rows, int64_t c) {
  return ((c >> 4) * rows + (row & ~31)) * 32 + ((c >> 3) & 1) * 256 + (row & 31) * 8 + (c & 7);
}
__device__ inline void split8(const float (&v)[8], f16* at) {
  f16x8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (f16)v[e];
    lo[e] = (f16)(v[e] - (float)hi[e]);
  }
  *reinterpret_cast<f16x8*>(at) = hi;
  *reinterpret_cast<f16x8*>(at + kLo) = lo;
}

template <bool BF16> __device__ inline float get1(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16> __device__ inline void put1(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else static_cast<float*>(p)[i] = v;
}

template <bool BF16> __device__ inline void get8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(d[e] << 16);
      v[2 * e + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
    }
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  }
}
template <bool BF16> __device__ inline f32x4 get4(const void* p, int64_t i) {
  if constexpr (BF16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    return f32x4{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                 __uint_as_float(r.y & 0xFFFF0000u)};
  } else {
    return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
  }
}
template <bool BF16> __device__ inline void put8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      d[e] = __builtin_bit_cast(uint16_t, (__bf16)v[2 * e]) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * e + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// Momentum, and the sum of squares of u in doubles (no overflow or underflow
// for any fp32 gradient), one partial a workgroup.  Without momentum u is the
// gradient itself and is not written (u null).
template <bool BF16>
__global__ __launch_bounds__(kThreads) void muon_momentum(MuonArgs a, float* __restrict__ u,
                                                          double* __restrict__ sums) {
  __shared__ double part[kThreads / 64];
  const int64_t size = a.n * a.k, c = blockIdx.y;
  double s = 0.0;
  // eight elements a thread where everything is 16-byte aligned, else one
  const auto low = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  const bool wide = size % 8 == 0 && ((low(a.grad) | low(a.buf) | low(a.buf_out)) & 15) == 0;
  const int64_t step = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (wide) {
    for (int64_t i = first * 8; i < size; i += step * 8) {
      const int64_t at = c * size + i;
      float v[8];
      get8<BF16>(a.grad, at, v);
      if (a.buf) {
        float b[8];
        get8<BF16>(a.buf, at, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          b[e] = a.momentum * b[e] + v[e];
          v[e] = a.nesterov ? v[e] + a.momentum * b[e] : b[e];
        }
        put8<BF16>(a.buf_out, at, b);
      }
      if (u) put8<false>(u, at, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (double)v[e] * (double)v[e];
    }
  } else {
    for (int64_t i = first; i < size; i += step) {
      const int64_t at = c * size + i;
      float v = get1<BF16>(a.grad, at);
      if (a.buf) {
        const float b = a.momentum * get1<BF16>(a.buf, at) + v;
        put1<BF16>(a.buf_out, at, b);
        v = a.nesterov ? v + a.momentum * b : b;
      }
      if (u) u[at] = v;
      s += (double)v * (double)v;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[c * gridDim.x + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

constexpr int kPad = 36;   // floats of a scratch row: 32 and a pad, 16-byte aligned

struct SplitOut {
  f16* m;
  int64_t rows, size;   // rows and halves of one matrix
};

// u / (|u| + eps) as split rows and as split columns, zeros in the padding: a
// wave per 32 x 32 tile, transposed through LDS.  The first tile's values are
// on their way while the norm's partials are added.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void muon_split(const void* __restrict__ u, const double* __restrict__ sums,
                                                       int parts, float eps, int64_t n, int64_t k, int64_t np,
                                                       int64_t kp, SplitOut rows, SplitOut cols) {
  __shared__ double part[kThreads / 64];
  __shared__ __attribute__((aligned(16))) float scratch[4][32 * kPad];
  const int64_t c = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* mine = scratch[wave];
  const int64_t base = c * n * k;
  const bool vec = k % 4 == 0 && (reinterpret_cast<uintptr_t>(u) & (BF16 ? 7 : 15)) == 0;
  const int64_t tiles_k = kp / 32, tiles = np / 32 * tiles_k, step = (int64_t)gridDim.x * 4;
  int64_t t = (int64_t)blockIdx.x * 4 + wave;
  f32x4 in[4];
  auto load = [&](int64_t tile) {
    const int64_t n0 = tile / tiles_k * 32, k0 = tile % tiles_k * 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 3), q = (lane & 7) * 4;
      in[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (n0 + r < n) {
        const int64_t src = base + (n0 + r) * k + k0 + q;
        if (vec) {
          if (k0 + q < k) in[i] = get4<BF16>(u, src);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k0 + q + e < k) in[i][e] = get1<BF16>(u, src + e);
        }
      }
    }
  };
  if (t < tiles) load(t);
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += sums[c * parts + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) part[wave] = s;
  __syncthreads();
  s = (part[0] + part[1]) + (part[2] + part[3]);
  // kScale / (|u| + eps) in two factors, the first a power of two: alone it leaves
  // fp32's range for norms below 2^-115
  const double norm = sqrt(s) + (double)eps;
  const float pre = norm < 0x1p-60 ? 0x1p96f : norm > 0x1p60 ? 0x1p-64f : 1.f;
  const float mul = (float)((double)kScale / (norm * (double)pre));
  rows.m += c * rows.size;
  cols.m += c * cols.size;
  for (; t < tiles; t += step) {
    const int64_t n0 = t / tiles_k * 32, k0 = t % tiles_k * 32;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4*>(mine + (i * 8 + (lane >> 3)) * kPad + (lane & 7) * 4) = in[i] * pre * mul;
    if (t + step < tiles) load(t + step);
    __builtin_amdgcn_wave_barrier();
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float v[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = mine[r * kPad + p * 16 + h * 8 + e];
        w[e] = mine[(p * 16 + h * 8 + e) * kPad + r];
      }
      split8(v, rows.m + split_at(n0 + r, rows.rows, k0 + p * 16 + h * 8));
      split8(w, cols.m + split_at(k0 + r, cols.rows, n0 + p * 16 + h * 8));
    }
  }
}

enum { kSym, kApply, kLast };

// C = kp P Q^T + k1 own1 + k2 own2, split rows.  Scales are folded into the factors.
struct Product {
  const f16 *p, *q;          // split rows [rows of C, K], [columns of C, K]
  const f16 *own1, *own2;    // C's shape and orientation, or null
  f16 *out, *out_t;          // C and its transpose (kSym: one matrix)
  float kp, k1, k2;
};
struct ProductShape {
  int64_t p_size, q_size, c_size, ct_size;   // halves of one matrix
  int64_t kdim, p_rows, q_rows, c_rows, ct_rows;
  int64_t c_high, c_wide;           // C's padded size
  int count;                        // matrices of one product
  int splits;                       // K ranges of a tile, joined by muon_join
  int tiles_m, tiles_n, tiles;      // tiles of one matrix
};
struct ProductPair {
  Product g[2];                     // independent products of one shape
};

template <int TM_, int TN_, int WM_, int WN_>
struct Tile {   // WM x WN waves, each of TM x TN 32 x 32 products
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
  static constexpr int kRows = 32 * TM * WM, kCols = 32 * TN * WN, kWaves = WM * WN;
};

// Tile number -> (ti, tj); kSym: tiles that reach above the diagonal, row by
// row (tiles WIDE times as wide as high).
template <int EPI, int WIDE = 1>
__device__ inline void tile_at(const ProductShape& sh, int at, int& ti, int& tj) {
  if constexpr (EPI == kSym) {
    ti = 0;
    while (at >= sh.tiles_n - ti / WIDE) at -= sh.tiles_n - ti++ / WIDE;
    tj = ti / WIDE + at;
  } else if (sh.tiles_m < sh.tiles_n) {   // the shorter side inside: an XCD's run needs fewer rows of the longer one
    ti = at % sh.tiles_m;
    tj = at / sh.tiles_m;
  } else {
    ti = at / sh.tiles_n;
    tj = at % sh.tiles_n;
  }
}

// Workgroup -> (matrix, K range, tile).  Workgroups go to the eight XCDs in
// turn; each XCD gets a contiguous run, so its L2 fetches the rows that its
// tiles share once, and of few matrices.
__device__ inline int run_of_xcd(int id, int all) {
  const int per = all >> 3, rest = all & 7, x = id & 7;
  return x * per + (x < rest ? x : rest) + (id >> 3);
}

// Own values of a 32 x 32 product, as `finish` adds them: 8 columns of row r in
// each half of 16 columns.
struct Own {
  f16x8 hi[2], lo[2], hi2[2], lo2[2];
};
template <int EPI>
__device__ inline void load_own(const Product& g, const ProductShape& sh, int64_t c, int64_t row0, int64_t col0, Own& o) {
  if (EPI == kLast || (EPI == kSym && col0 < row0)) return;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t at = c * sh.c_size + split_at(row0 + r, sh.c_rows, col0 + p * 16 + h * 8);
    if (g.own1) {
      o.hi[p] = *reinterpret_cast<const f16x8*>(g.own1 + at);
      o.lo[p] = *reinterpret_cast<const f16x8*>(g.own1 + at + kLo);
    }
    if (EPI == kSym && g.own2) {
      o.hi2[p] = *reinterpret_cast<const f16x8*>(g.own2 + at);
      o.lo2[p] = *reinterpret_cast<const f16x8*>(g.own2 + at + kLo);
    }
  }
}

// Finish of one 32 x 32 product: its sums go through LDS (32 x kPad floats of
// this wave) so that own values are read and results written 16 bytes a lane,
// 1 KB of consecutive memory an instruction.  `acc` holds
// C[8 (e / 4) + 4 h + e % 4][r] in lane 32 h + r.
template <int EPI, bool BF16>
__device__ inline void finish(const Product& g, const ProductShape& sh, const MuonArgs& m, int64_t c, int64_t row0,
                              int64_t col0, const f32x16& acc, const Own& own, float* scratch) {
  if (EPI == kSym && col0 < row0) return;   // written by the product above the diagonal
  const bool mirror = EPI == kApply || (EPI == kSym && col0 > row0);
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    scratch[(8 * (e / 4) + 4 * (lane >> 5) + e % 4) * kPad + (lane & 31)] = acc[e] * g.kp;
  __builtin_amdgcn_wave_barrier();
  const int r = lane & 31, h = lane >> 5;
  auto take = [&](int row, int col, float (&v)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(scratch + row * kPad + col);
    const f32x4 b = *reinterpret_cast<const f32x4*>(scratch + row * kPad + col + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  };
  if constexpr (EPI == kLast) {
    const float keep = 1.f - m.lr * m.decay, lr = m.lr * m.scale;
    const bool wide = m.k % 8 == 0 && ((reinterpret_cast<uintptr_t>(m.w_out) | reinterpret_cast<uintptr_t>(m.w)) & 15) == 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int lr_ = t * 16 + (lane >> 2), lc = (lane & 3) * 8;
      const int64_t row = row0 + lr_, col = col0 + lc;
      float v[8];
      take(lr_, lc, v);
      const f16* o1 = g.own1 + c * sh.c_size + split_at(row, sh.c_rows, col);
      const f16x8 hi = *reinterpret_cast<const f16x8*>(o1), lo = *reinterpret_cast<const f16x8*>(o1 + kLo);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += g.k1 * ((float)hi[e] + (float)lo[e]);
      if (row >= m.n || col >= m.k) continue;
      const int64_t o = (c * m.n + row) * m.k + col;
      if (wide) {
        float w[8];
        if (m.w) {
          get8<BF16>(m.w, o, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = w[e] * keep - lr * v[e];
        }
        put8<BF16>(m.w_out, o, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < m.k) put1<BF16>(m.w_out, o + e, m.w ? get1<BF16>(m.w, o + e) * keep - lr * v[e] : v[e]);
      }
    }
    return;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int lc = p * 16 + h * 8;
    float v[8];
    take(r, lc, v);
    if (g.own1)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += g.k1 * ((float)own.hi[p][e] + (float)own.lo[p][e]);
    if (EPI == kSym && g.own2)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += g.k2 * ((float)own.hi2[p][e] + (float)own.lo2[p][e]);
    split8(v, g.out + c * sh.c_size + split_at(row0 + r, sh.c_rows, col0 + lc));
    if (mirror) {
      *reinterpret_cast<f32x4*>(scratch + r * kPad + lc) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(scratch + r * kPad + lc + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
  __builtin_amdgcn_wave_barrier();
  if (!mirror) return;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int lc = p * 16 + h * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = scratch[(lc + e) * kPad + r];
    split8(v, g.out_t + c * sh.ct_size + split_at(col0 + r, sh.ct_rows, row0 + lc));
  }
  __builtin_amdgcn_wave_barrier();
}

// K loop.  A stage is 16 k of both operands, both planes: one MFMA's depth.
// Copies go straight into LDS, three stages ahead.  The two halves of the
// waves (one of each on every SIMD) take turns, a barrier between the turns:
// while one reads its fragments from LDS and issues its copies, the other
// multiplies, so the matrix cores wait for neither.
template <class T, int EPI, bool BF16>
__global__ __launch_bounds__(64 * T::kWaves) void muon_product(ProductPair pair, ProductShape sh, MuonArgs m,
                                                              f32x4* __restrict__ partial) {
  constexpr int kRows = T::kRows;
  constexpr int kPieces = (T::kRows + T::kCols) / 16;   // 1 KB copies of a stage
  constexpr int kCopies = kPieces / T::kWaves;
  constexpr int kStageB = (T::kRows + T::kCols) * kRowB;
  static_assert(kPieces % T::kWaves == 0, "whole copies a wave");
  __shared__ __attribute__((aligned(16))) char lds[kSlots * kStageB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int per = sh.tiles * sh.splits, run = run_of_xcd(blockIdx.x, gridDim.x);
  const int z = run / per, tile = run % per % sh.tiles, split = run % per / sh.tiles;
  const Product& g = pair.g[z >= sh.count];
  const int64_t c = z >= sh.count ? z - sh.count : z;
  int ti, tj;
  tile_at<EPI, T::kCols / T::kRows>(sh, tile, ti, tj);
  const int64_t i0 = (int64_t)ti * T::kRows, j0 = (int64_t)tj * T::kCols;
  const int p_pitch = (int)(sh.p_rows * kRowB), q_pitch = (int)(sh.q_rows * kRowB);   // bytes of 16 columns
  const __amdgpu_buffer_rsrc_t pr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<f16*>(g.p + c * sh.p_size + i0 * 32), (short)0, (int)((sh.p_size - i0 * 32) * 2), kBufferWord3);
  const __amdgpu_buffer_rsrc_t qr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<f16*>(g.q + c * sh.q_size + j0 * 32), (short)0, (int)((sh.q_size - j0 * 32) * 2), kBufferWord3);

  auto issue = [&](int slot, int stage) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int piece = wave * kCopies + i;             // 16 rows: of P, then of Q
      const bool in_p = piece * 16 < kRows;
      const uint32_t off = (uint32_t)(in_p ? piece : piece - kRows / 16) * 1024 + (uint32_t)lane * 16;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(in_p ? pr : qr, (lds_void*)(lds + slot * kStageB + piece * 1024), 16,
                                               off, stage * (in_p ? p_pitch : q_pitch), 0, 0);
    }
  };

  f32x16 acc[T::TM][T::TN];
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  struct Frags {
    f16x8 ph[T::TM], pl[T::TM], qh[T::TN], ql[T::TN];
  };
  auto read = [&](Frags& f, int slot) {
    const char* pb = lds + slot * kStageB + wm * T::TM * 2048 + lane * 16;
    const char* qb = lds + slot * kStageB + kRows * kRowB + wn * T::TN * 2048 + lane * 16;
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
      f.qh[j] = *reinterpret_cast<const f16x8*>(qb + j * 2048);
      f.ql[j] = *reinterpret_cast<const f16x8*>(qb + j * 2048 + 1024);
    }
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
      f.ph[i] = *reinterpret_cast<const f16x8*>(pb + i * 2048);
      f.pl[i] = *reinterpret_cast<const f16x8*>(pb + i * 2048 + 1024);
    }
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
#pragma unroll
      for (int j = 0; j < T::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.ph[i], f.ql[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < T::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.pl[i], f.qh[j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < T::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.ph[i], f.qh[j], acc[i][j], 0, 0, 0);
    }
  };
  const int all = (int)(sh.kdim / kBK);
  const int s0 = (int)((int64_t)all * split / sh.splits), s1 = (int)((int64_t)all * (split + 1) / sh.splits);
  const int stages = s1 - s0;                           // at least 4 (the plan's K ranges)
  auto copy = [&](int t) { issue(t & (kSlots - 1), s0 + t); };
#pragma unroll
  for (int t = 0; t < kSlots - 1; ++t) copy(t);
  wait_vmcnt<2 * kCopies>();
  lds_barrier();                                        // stage 0 is here
  const bool second = wave >= T::kWaves / 2;
  if (second) lds_barrier();
  for (int t = 0; t < stages; ++t) {
    Frags f;
    read(f, t & (kSlots - 1));
    if (t + 3 < stages) copy(t + 3);                    // into the slot that both halves have read
    if (t + 3 < stages) wait_vmcnt<2 * kCopies>();      // this wave's part of stage t + 1 is here
    else wait_vmcnt<0>();
    lds_barrier();
    __builtin_amdgcn_s_setprio(1);
    multiply(f);
    __builtin_amdgcn_s_setprio(0);
    lds_barrier();
  }
  if (!second) lds_barrier();

  if (sh.splits > 1) {   // [z][tile][split][wave][product][4 rows][lane]
    partial += ((((int64_t)z * sh.tiles + tile) * sh.splits + split) * T::kWaves + wave) * (T::TM * T::TN * 4 * 64) + lane;
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
      for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4)
          partial[((i * T::TN + j) * 4 + e4) * 64] =
              f32x4{acc[i][j][4 * e4], acc[i][j][4 * e4 + 1], acc[i][j][4 * e4 + 2], acc[i][j][4 * e4 + 3]};
    return;
  }
  __syncthreads();   // every wave has read its last stage: LDS becomes scratch
  auto end = [&](int i, int j, const f32x16& v, float* scratch) {
    const int64_t row0 = i0 + (wm * T::TM + i) * 32, col0 = j0 + (wn * T::TN + j) * 32;
    Own own;
    load_own<EPI>(g, sh, c, row0, col0, own);
    finish<EPI, BF16>(g, sh, m, c, row0, col0, v, own, scratch);
  };
  float* scratch = reinterpret_cast<float*>(lds) + wave * (32 * kPad);
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) end(i, j, acc[i][j], scratch);
}

// Sums of a split tile's partials, in split order, and the product's finish:
// one wave per 32 x 32 product.
template <class T, int EPI, bool BF16>
__global__ __launch_bounds__(64) void muon_join(ProductPair pair, ProductShape sh, MuonArgs m,
                                                const f32x4* __restrict__ partial) {
  constexpr int kPer = T::TM * T::TN;
  __shared__ __attribute__((aligned(16))) float scratch[32 * kPad];
  const int z = blockIdx.z;
  const Product& g = pair.g[z >= sh.count];
  const int64_t c = z >= sh.count ? z - sh.count : z;
  const int tile = blockIdx.x / (T::kWaves * kPer), at = blockIdx.x % (T::kWaves * kPer);
  const int wave = at / kPer, i = at % kPer / T::TN, j = at % T::TN;
  int ti, tj;
  tile_at<EPI, T::kCols / T::kRows>(sh, tile, ti, tj);
  partial += (((int64_t)z * sh.tiles + tile) * sh.splits * T::kWaves + wave) * (kPer * 4 * 64) + at % kPer * 256 + threadIdx.x;
  const int64_t row0 = (int64_t)ti * T::kRows + (wave / T::WN * T::TM + i) * 32;
  const int64_t col0 = (int64_t)tj * T::kCols + (wave % T::WN * T::TN + j) * 32;
  Own own;
  load_own<EPI>(g, sh, c, row0, col0, own);
  f32x16 s;
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = 0.f;
  for (int k = 0; k < sh.splits; ++k)
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const f32x4 v = partial[(int64_t)k * T::kWaves * (kPer * 4 * 64) + e4 * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * e4 + e] += v[e];
    }
  finish<EPI, BF16>(g, sh, m, c, row0, col0, s, own, scratch);
}

// The same for small matrices, where a launch has few tiles and latency counts:
// every wave of the workgroup takes a part of K of one tile, its fragments
// straight from memory into registers (no LDS stage, no barrier in the loop),
// kAhead steps ahead; the parts are added through LDS in wave order.
template <int TM, int TN, int W, int EPI, bool BF16>
__global__ __launch_bounds__(64 * W) void muon_product_small(ProductPair pair, ProductShape sh, MuonArgs m) {
  constexpr int kAhead = TM * TN == 1 ? 8 : 4;
  constexpr int kProducts = TM * TN;
  __shared__ f32x4 part[W][kProducts][4][64];
  __shared__ __attribute__((aligned(16))) float scratch[kProducts][32 * kPad];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int run = run_of_xcd(blockIdx.x, gridDim.x), z = run / sh.tiles;
  const Product& g = pair.g[z >= sh.count];
  const int64_t c = z >= sh.count ? z - sh.count : z;
  int ti, tj;
  tile_at<EPI>(sh, run % sh.tiles, ti, tj);
  const int64_t i0 = (int64_t)ti * (32 * TM), j0 = (int64_t)tj * (32 * TN);
  const f16* pp = g.p + c * sh.p_size + i0 * 32 + lane * 8;
  const f16* qp = g.q + c * sh.q_size + j0 * 32 + lane * 8;
  const int64_t p_pitch = sh.p_rows * 32, q_pitch = sh.q_rows * 32;   // 16 columns
  const int all = (int)(sh.kdim / kBK);
  const int s0 = all * wave / W, s1 = all * (wave + 1) / W;

  struct Frags {
    f16x8 ph[TM], pl[TM], qh[TN], ql[TN];
  } f[kAhead];
  auto load = [&](Frags& x, int s) {
    const f16* p = pp + s * p_pitch;
    const f16* q = qp + s * q_pitch;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      x.ph[i] = *reinterpret_cast<const f16x8*>(p + i * 1024);
      x.pl[i] = *reinterpret_cast<const f16x8*>(p + i * 1024 + kLo);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      x.qh[j] = *reinterpret_cast<const f16x8*>(q + j * 1024);
      x.ql[j] = *reinterpret_cast<const f16x8*>(q + j * 1024 + kLo);
    }
  };
  // wave q finishes product q: its own values are on their way from the start
  const int64_t row0 = i0 + wave / TN * 32, col0 = j0 + wave % TN * 32;
  Own own;
  if (wave < kProducts) load_own<EPI>(g, sh, c, row0, col0, own);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (s0 + u < s1) load(f[u], s0 + u);
  for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u < s1) {
        const Frags& x = f[u];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x.ph[i], x.ql[j], acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x.pl[i], x.qh[j], acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x.ph[i], x.qh[j], acc[i][j], 0, 0, 0);
          }
        if (s + u + kAhead < s1) load(f[u], s + u + kAhead);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kProducts; ++q) {
    const f32x16& v = acc[q / TN][q % TN];
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][q][e][lane] = f32x4{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
  }
  __syncthreads();
  if (wave >= kProducts) return;
  f32x16 s;
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 v = part[w][wave][q][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * q + e] += v[e];
    }
  finish<EPI, BF16>(g, sh, m, c, row0, col0, s, own, scratch[wave]);
}

template <int EPI>
int tiles_of(const ProductShape& sh, int wide) {
  if (EPI != kSym) return sh.tiles_m * sh.tiles_n;
  int all = 0;
  for (int i = 0; i < sh.tiles_m; ++i) all += sh.tiles_n - i / wide;
  return all;
}

template <int TM, int TN, int W, int EPI, bool BF16>
hipError_t product_small(const ProductPair& g, int pairs, ProductShape sh, const MuonArgs& m, hipStream_t s) {
  sh.tiles = tiles_of<EPI>(sh, 1);
  hipLaunchKernelGGL((muon_product_small<TM, TN, W, EPI, BF16>),
                     dim3((unsigned)sh.tiles * (unsigned)(pairs * sh.count)), dim3(64 * W), 0, s, g, sh, m);
  return hipGetLastError();
}

typedef Tile<2, 2, 2, 4> TileBig;    // 128 x 256
typedef Tile<2, 2, 4, 2> TileTall;   // 256 x 128

template <class T, int EPI, bool BF16>
hipError_t product_t(const ProductPair& g, int pairs, ProductShape sh, const MuonArgs& m, f32x4* partial,
                     hipStream_t s) {
  sh.tiles = tiles_of<EPI>(sh, T::kCols / T::kRows);
  const unsigned z = (unsigned)(pairs * sh.count);
  hipLaunchKernelGGL((muon_product<T, EPI, BF16>), dim3((unsigned)(sh.tiles * sh.splits) * z),
                     dim3(64 * T::kWaves), 0, s, g, sh, m, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sh.splits == 1) return e;
  hipLaunchKernelGGL((muon_join<T, EPI, BF16>), dim3((unsigned)(sh.tiles * T::kWaves * T::TM * T::TN), 1, z),
                     dim3(64), 0, s, g, sh, m, partial);
  return hipGetLastError();
}

template <int EPI, bool BF16 = false>
hipError_t product(const ProductPair& g, int pairs, ProductShape sh, MuonCut cut, const MuonArgs& m, f32x4* partial,
                   hipStream_t s) {
  sh.tiles_m = (int)(sh.c_high / cut.rows);
  sh.tiles_n = (int)(sh.c_wide / cut.cols);
  sh.splits = cut.splits;
  if constexpr (EPI == kLast)
    if (cut.rows == 256) return product_t<TileTall, EPI, BF16>(g, pairs, sh, m, partial, s);
  if (cut.rows == 128) return product_t<TileBig, EPI, BF16>(g, pairs, sh, m, partial, s);
  if (cut.rows == 64) return product_small<2, 2, 4, EPI, BF16>(g, pairs, sh, m, s);
  return product_small<1, 1, 4, EPI, BF16>(g, pairs, sh, m, s);
}

hipError_t steps(const MuonPlan& p, const MuonArgs& m, bool bf16, char* ws, hipStream_t s) {
  auto at = [&](size_t o) { return reinterpret_cast<f16*>(ws + o); };
  f16 *x = at(p.x), *xt[2] = {at(p.xt0), at(p.xt1)}, *a = at(p.a), *b = at(p.b), *pa = at(p.pa);
  f16* d[2] = {at(p.d0), at(p.d1)};
  f32x4* partial = reinterpret_cast<f32x4*>(ws + p.partial);
  const int64_t xs = p.rp * p.lp * 2, as = p.rp * p.rp * 2, R = p.rp, L = p.lp;
  const ProductShape gram{xs, xs, as, as, L, R, R, R, R, R, R, m.count, 1, 0, 0, 0};
  const ProductShape sym{as, as, as, as, R, R, R, R, R, R, R, m.count, 1, 0, 0, 0};
  const ProductShape apply{as, xs, xs, xs, R, R, L, R, L, R, L, m.count, 1, 0, 0, 0};
  hipError_t e = hipSuccess;
  auto run = [&](const Product& g, const ProductShape& sh, MuonCut cut) {
    if (e == hipSuccess) e = product<kSym>(ProductPair{{g, g}}, 1, sh, cut, m, partial, s);
  };
  const float one = kRScale;   // a product of two values at kScale, back at kScale
  int now = 0;
  for (int done = 0; done < m.steps;) {
    const int group = std::min(p.group, m.steps - done);
    // Q = q I + D with X <- Q X after `group` steps; D at kScale for one step, kScaleD for more
    run({x, x, nullptr, nullptr, a, a, one, 0.f, 0.f}, gram, p.gram);
    float q = 1.f;
    int cur = 0;
    for (int i = 0; i < group; ++i) {
      f16* bi = i == 0 ? d[0] : b;      // B = b A + c A A; P = a I + B
      run({a, a, a, nullptr, bi, bi, m.cc * one, m.cb, 0.f}, sym, p.sym);
      // A <- P A P
      const Product half{bi, a, a, nullptr, pa, pa, one, m.ca, 0.f};
      // D <- a D + q B + B D, of the scale of the ones before (i == 1: D is the first step's B)
      const float sd = i == 1 ? kScale : kScaleD;
      const Product delta{bi, d[cur], d[cur], bi, d[cur ^ 1], d[cur ^ 1], kScaleD / (kScale * sd), m.ca * (kScaleD / sd),
                          q * (kScaleD / kScale)};
      const bool more = i + 1 < group;
      if (i > 0 && more) {
        if (e == hipSuccess) e = product<kSym>(ProductPair{{half, delta}}, 2, sym, p.pair, m, partial, s);
      } else if (i > 0) {
        run(delta, sym, p.sym);
      } else if (more) {
        run(half, sym, p.sym);
      }
      if (i > 0) cur ^= 1;
      if (more) run({bi, pa, pa, nullptr, a, a, one, m.ca, 0.f}, sym, p.sym);
      q *= m.ca;
    }
    done += group;
    const float kd = 1.f / (group > 1 ? kScaleD : kScale);
    if (e != hipSuccess) return e;
    if (done < m.steps) {
      const Product g{d[cur], xt[now], x, nullptr, x, xt[now ^ 1], kd, q, 0.f};
      e = product<kApply>(ProductPair{{g, g}}, 1, apply, p.apply, m, partial, s);
      now ^= 1;
    } else {
      // the result's own orientation: rows n, columns k; its values at 1
      Product g{d[cur], xt[now], x, nullptr, nullptr, nullptr, kd * kRScale, q * kRScale, 0.f};
      ProductShape sh = apply;
      if (m.n > m.k) {
        g = Product{xt[now], d[cur], xt[now], nullptr, nullptr, nullptr, kd * kRScale, q * kRScale, 0.f};
        sh = ProductShape{xs, as, xs, xs, R, L, R, L, R, L, R, m.count, 1, 0, 0, 0};
      }
      const ProductPair pair{{g, g}};
      e = bf16 ? product<kLast, true>(pair, 1, sh, p.last, m, partial, s)
               : product<kLast, false>(pair, 1, sh, p.last, m, partial, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The largest |u0 + u1 x + u2 x^2 + u3 x^3| of x in [0, top], at the ends or
// where the derivative is zero; `odd`: of s times that for x = s^2.
double largest(const double (&u)[4], double top, bool odd) {
  auto value = [&](double x) {
    const double v = u[0] + x * (u[1] + x * (u[2] + x * u[3]));
    return std::fabs(odd ? std::sqrt(x) * v : v);
  };
  double most = std::max(value(0.0), value(top));
  // (s v(s^2))' = u0 + 3 u1 x + 5 u2 x^2 (u3 = 0); v' = u1 + 2 u2 x + 3 u3 x^2
  const double p = odd ? u[0] : u[1], q = odd ? 3 * u[1] : 2 * u[2], r = odd ? 5 * u[2] : 3 * u[3];
  double at[2] = {-1.0, -1.0};
  if (r == 0.0) {
    if (q != 0.0) at[0] = -p / q;
  } else if (q * q >= 4 * p * r) {
    const double w = -0.5 * (q + std::copysign(std::sqrt(q * q - 4 * p * r), q));
    at[0] = w / r;
    if (w != 0.0) at[1] = p / w;
  }
  for (double x : at)
    if (x > 0.0 && x < top) most = std::max(most, value(x));
  return most;
}

}  // namespace

// p(s) = a s + b s^3 + c s^5 is 0 at 0 and continuous, so singular values of
// [0, m] go to [0, max |p|] of it, all of it: the ranges below are exact for
// single steps.  The product of a group is bounded by its factors' largest values.
MuonRange muon_range(double a, double b, double c, int steps) {
  constexpr double kMost = 65504.0 / kScale * 0.999, kMostD = 65504.0 / kScaleD * 0.999;
  MuonRange fit{true, true};
  double m = 1.0, product = 1.0, alone = 1.0;   // of a group: P's largest values, and q = a^steps
  for (int i = 0; i < steps; ++i) {
    const double top = m * m;
    if (!(top < kMost) || !(largest({0, b, c, 0}, top, false) < kMost)) fit.steps = false;   // A, B = b A + c A A
    const bool first = i % kGroupSteps == 0, last = i % kGroupSteps == kGroupSteps - 1 || i + 1 == steps;
    product = (first ? 1.0 : product) * largest({a, b, c, 0}, top, false);
    alone = (first ? 1.0 : alone) * std::fabs(a);
    if (!last && !(largest({0, a, b, c}, top, false) < kMost)) fit.groups = false;           // P A
    if (!first && !(product + alone < kMostD)) fit.groups = false;                           // D
    m = largest({a, b, c, 0}, top, true);
  }
  fit.groups = fit.groups && fit.steps;
  return fit;
}

static int64_t up_to(int64_t side, int64_t tile) { return (side + tile - 1) / tile * tile; }

// Tiles that a matrix's own sides admit, however many there are: the larger
// one's padding may not cost more products (r r l of the padded sides) than its rate gains.
// * 64 x 64 against 32 x 32, up to 1.3 times: 2000 x 128 x 128 (1.0) 1877 us
//   against 2023, 64 x 400 x 400 (1.25) 804 against 825; 300 x 288 x 288 (1.37)
//   2049 against 1800, 2000 x 96 x 96 (2.4) 1864 against 1133.
// * 128 x 256 against 64 x 64, up to 1.4 times, or where one matrix by itself is
//   enough work for it (cut_of): 20 x 1100 x 1100 (1.37) 2690 us against 3150, 256 x
//   256 x 256 (1.0) 876 against 1095; 64 x 400 x 400 (1.49) 875 against 804, 64 x 300
//   x 300 (4.1) 855 against 425, 2000 x 128 x 128 (8) 5229 against 1877.
struct MuonTiles {
  bool mid, big;
};
static MuonTiles tiles_for(int64_t r, int64_t l) {
  auto products = [&](int64_t t) { return (double)up_to(r, t) * (double)up_to(r, t) * (double)up_to(l, t); };
  return {products(64) <= 1.3 * products(32), products(256) <= 1.4 * products(64)};
}

// Tile and K ranges of a product of `z` matrices C [high, wide], K deep,
// symmetric or not.  Measured on single products from 128 to 8192 a side:
// * up to 320 tiles of 32 x 32 (one a CU and some): these.  C 512 x 512
//   symmetric, K 512 and 2048: 4.8 and 9.2 us against 6.8 and 14.7 us by 64 x
//   64 tiles; C 1024 x 1024 has 528 and takes 12.6 against 10.5 us.
// * up to 500 K tiles x k of 64 x 64: these.  C 1024 x 1024, K 1024: 10.5 us
//   against 17.8 by the big tile; C 1024 x 4096, K 1024 (1050 K): 46.8 against 38.3.
// * else 128 x 256 tiles through LDS, K split while the launch stays within 224
//   workgroups, 24 stages of 16 and 8 ranges: C 2048 x 2048 symmetric, K
//   2048: 59 us whole, 40 in 3 ranges, 51 in 4; C 1024 x 4096, K 1024: 38 whole, 41 in 2.
static MuonCut cut_of(const MuonTiles& admitted, int64_t high, int64_t wide, int64_t k, int64_t z, bool sym) {
  auto tiles = [&](int64_t h, int64_t w) {
    const int64_t m = (high + h - 1) / h, n = (wide + w - 1) / w;
    return sym ? m * (n + 1) / 2 : m * n;
  };
  constexpr int64_t kBigWork = 500000;
  if (tiles(32, 32) * z <= 320) return {32, 32, 1};
  const int64_t work = tiles(64, 64) * k;
  if (work > kBigWork || (work * z > kBigWork && admitted.big)) {
    const int64_t most = std::min<int64_t>(std::min<int64_t>(8, k / 16 / 24), 224 / (tiles(128, 256) * z));
    return {128, 256, (int)std::max<int64_t>(1, most)};
  }
  return admitted.mid ? MuonCut{64, 64, 1} : MuonCut{32, 32, 1};
}

MuonPlan plan_muon(int matrices, int64_t n, int64_t k, bool loose) {
  MuonPlan p{};
  p.r = std::min(n, k);
  p.l = std::max(n, k);
  // Matrices at a time: 2^26 elements keep every CU busy for many tiles, and the
  // workspace within about 2.5 GB (or one matrix's) and a launch within 2^32 threads for any count.
  constexpr int64_t kElements = (int64_t)1 << 26;
  p.count = (int)std::min<int64_t>(matrices, std::max<int64_t>(1, kElements / (up_to(p.r, 32) * up_to(p.l, 32))));
  const int count = p.count;
  const MuonTiles admitted = tiles_for(p.r, p.l);
  p.gram = cut_of(admitted, p.r, p.r, p.l, count, true);
  p.sym = cut_of(admitted, p.r, p.r, p.r, count, true);
  p.pair = cut_of(admitted, p.r, p.r, p.r, 2 * (int64_t)count, true);
  p.apply = cut_of(admitted, p.r, p.l, p.r, count, false);
  // the result of n > k has X's columns as its rows, so its tile stands upright: the shorter side is
  // padded to 128 either way (8000 x 600 update: 225 us against 298 with the 128 x 256 tile and 256)
  p.last = p.apply;
  if (n > k) std::swap(p.last.rows, p.last.cols);
  // two launches more, less work: not where launches are all there is (256 x 512)
  const bool grouped = p.l >= 2 * p.r && p.apply.rows > 32;
  p.group = loose && grouped ? kGroupSteps : 1;
  // sides padded so that the tiles of every product are whole (the same for
  // either `loose`: the workspace is asked for before the steps' form is known)
  int64_t pr = std::max(p.apply.rows, std::max(p.gram.cols, p.sym.cols)), pl = p.apply.cols;
  if (grouped) pr = std::max<int64_t>(pr, p.pair.cols);
  pr = std::max<int64_t>(pr, n > k ? p.last.cols : p.last.rows);
  pl = std::max<int64_t>(pl, n > k ? p.last.rows : p.last.cols);
  p.rp = up_to(p.r, pr);
  p.lp = up_to(p.l, pl);
  p.parts = std::min<int64_t>(1024, (n * k + 8 * kThreads - 1) / (8 * kThreads));
  const size_t c = (size_t)count;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  const size_t big = c * (size_t)(p.rp * p.lp) * 4, small = c * (size_t)(p.rp * p.rp) * 4;
  p.u = take(c * (size_t)(n * k) * 4);
  p.sums = take(c * (size_t)p.parts * 8);
  p.x = take(big);
  p.xt0 = take(big);
  p.xt1 = take(big);
  p.a = take(small);
  p.b = take(small);
  p.pa = take(small);
  p.d0 = take(small);
  p.d1 = take(small);
  // fp32 partials of the products with split K: a tile for each range
  auto part = [&](const MuonCut& cut, int64_t high, int64_t wide, bool sym, size_t pairs) -> size_t {
    if (cut.splits == 1) return 0;
    const int64_t tm = high / cut.rows, tn = wide / cut.cols;
    return (size_t)((sym ? tm * (tn + 1) / 2 : tm * tn) * cut.splits * cut.rows * cut.cols) * pairs * c * 4;
  };
  size_t most = part(p.gram, p.rp, p.rp, true, 1);
  most = std::max(most, part(p.sym, p.rp, p.rp, true, 1));
  if (grouped) most = std::max(most, part(p.pair, p.rp, p.rp, true, 2));
  most = std::max(most, part(p.apply, p.rp, p.lp, false, 1));
  most = std::max(most, part(p.last, p.lp, p.rp, false, 1));
  p.partial = take(most);
  p.workspace_bytes = at;
  return p;
}

// The plan's matrices at a time.
static hipError_t launch_part(const MuonPlan& p, const MuonArgs& a, bool bf16, char* ws, hipStream_t s) {
  float* u = a.buf ? reinterpret_cast<float*>(ws + p.u) : nullptr;
  double* sums = reinterpret_cast<double*>(ws + p.sums);
  const dim3 g1((unsigned)p.parts, (unsigned)a.count);
  if (bf16) hipLaunchKernelGGL((muon_momentum<true>), g1, dim3(kThreads), 0, s, a, u, sums);
  else hipLaunchKernelGGL((muon_momentum<false>), g1, dim3(kThreads), 0, s, a, u, sums);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool wide = a.n <= a.k;
  const int64_t np = wide ? p.rp : p.lp, kp = wide ? p.lp : p.rp;
  const SplitOut x{reinterpret_cast<f16*>(ws + p.x), p.rp, p.rp * p.lp * 2};
  const SplitOut xt{reinterpret_cast<f16*>(ws + p.xt0), p.lp, p.lp * p.rp * 2};
  const dim3 g2((unsigned)std::min<int64_t>(2048, (np / 32 * (kp / 32) + 3) / 4), (unsigned)a.count);
  if (!u && bf16)
    hipLaunchKernelGGL((muon_split<true>), g2, dim3(kThreads), 0, s, a.grad, sums, (int)p.parts, a.eps, a.n, a.k, np, kp,
                       wide ? x : xt, wide ? xt : x);
  else
    hipLaunchKernelGGL((muon_split<false>), g2, dim3(kThreads), 0, s, u ? u : a.grad, sums, (int)p.parts, a.eps, a.n, a.k,
                       np, kp, wide ? x : xt, wide ? xt : x);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return steps(p, a, bf16, ws, s);
}

hipError_t launch_muon(const MuonPlan& p, const MuonArgs& a, bool bf16, char* ws, hipStream_t s) {
  const int64_t item = bf16 ? 2 : 4;
  for (int at = 0; at < a.count; at += p.count) {
    auto from = [&](const void* t) { return t ? static_cast<const char*>(t) + at * a.n * a.k * item : nullptr; };
    MuonArgs part = a;
    part.count = std::min(p.count, a.count - at);
    part.w = from(a.w);
    part.grad = from(a.grad);
    part.buf = from(a.buf);
    part.w_out = const_cast<char*>(from(a.w_out));
    part.buf_out = const_cast<char*>(from(a.buf_out));
    const hipError_t e = launch_part(p, part, bf16, ws, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sherry
