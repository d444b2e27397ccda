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
// normal numbers to 2^-27) and leaves room to 4 for iterates and 7 for b A + c A A.
//
// The matrix cores bound it: 3 steps (3 R^2 L + R^3) multiply-adds of float16.
#include <algorithm>

#include "ops_internal.h"

namespace sherry {
namespace {

typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr float kScale = 8192.f, kRScale = 1.f / 8192.f;
constexpr int kBK = 32;                 // k of an LDS stage: one 128-byte piece (hi, lo) of a row
constexpr int kRowB = kBK * 4;

// A split matrix holds a row's values in pieces of 32: 32 hi, then 32 lo.
__device__ inline int64_t split_at(int64_t row, int64_t cols, int64_t c) {
  return row * (2 * cols) + (c >> 5) * 64 + (c & 31);
}
__device__ inline void split_put(f16* m, int64_t at, float v) {
  const f16 hi = (f16)v;
  m[at] = hi;
  m[at + 32] = (f16)(v - (float)hi);
}
__device__ inline float split_get(const f16* m, int64_t at) { return (float)m[at] + (float)m[at + 32]; }

template <bool BF16> __device__ inline float get1(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16> __device__ inline void put1(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else static_cast<float*>(p)[i] = v;
}

// Momentum, and the sum of squares of u in doubles (no overflow or underflow
// for any fp32 gradient), one partial a workgroup.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void muon_momentum(MuonArgs a, float* __restrict__ u,
                                                          double* __restrict__ sums) {
  __shared__ double part[kThreads / 64];
  const int64_t size = a.n * a.k, c = blockIdx.y;
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < size; i += (int64_t)gridDim.x * kThreads) {
    const int64_t at = c * size + i;
    float v = get1<BF16>(a.grad, at);
    if (a.buf) {
      const float b = a.momentum * get1<BF16>(a.buf, at) + v;
      put1<BF16>(a.buf_out, at, b);
      v = a.nesterov ? v + a.momentum * b : b;
    }
    u[at] = v;
    s += (double)v * (double)v;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[c * gridDim.x + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// u / (|u| + eps) as split rows and as split columns, zeros in the padding:
// 32 x 32 tiles, transposed through LDS.
__global__ __launch_bounds__(kThreads) void muon_split(const float* __restrict__ u, const double* __restrict__ sums,
                                                       int parts, float eps, int64_t n, int64_t k, int64_t np,
                                                       int64_t kp, f16* __restrict__ rows, f16* __restrict__ cols) {
  __shared__ double part[kThreads];
  __shared__ float tile[32][33];
  const int64_t c = blockIdx.z;
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += sums[c * parts + i];
  part[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
    __syncthreads();
  }
  const float mul = (float)((double)kScale / (sqrt(part[0]) + (double)eps));
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t n0 = (int64_t)blockIdx.y * 32, k0 = (int64_t)blockIdx.x * 32;
  u += c * n * k;
  rows += c * np * kp * 2;
  cols += c * np * kp * 2;
  for (int i = y; i < 32; i += 8) {
    const float v = n0 + i < n && k0 + x < k ? u[(n0 + i) * k + k0 + x] * mul : 0.f;
    split_put(rows, split_at(n0 + i, kp, k0 + x), v);
    tile[i][x] = v;
  }
  __syncthreads();
  for (int i = y; i < 32; i += 8) split_put(cols, split_at(k0 + i, np, n0 + x), tile[x][i]);
}

enum { kGram, kSquare, kApply, kLast };

struct ProductArgs {
  const f16 *p, *q;        // split rows [rows of C, K], [columns of C, K]
  const f16* own;          // kSquare: A; kApply, kLast: X in C's orientation
  f16 *out, *out_t;        // C and its transpose (kGram, kSquare: the same matrix)
  int64_t p_size, q_size, c_size;   // halves of one matrix
  int64_t kdim, c_cols, ct_cols;
  int tiles_m, tiles_n;
  float ca, cb, cc;
};

// C = P Q^T by TILE x TILE tiles: four waves of TILE/2 x TILE/2, stages of 32 k
// (both planes of both operands) copied straight into LDS one stage ahead.
// The 16-byte chunks of a 128-byte LDS row are XORed with half the row's
// number, so the 16 rows of a fragment read cover every bank once.
template <int TILE, int EPI, bool BF16>
__global__ __launch_bounds__(kThreads) void muon_product(ProductArgs g, MuonArgs m) {
  constexpr int W = TILE / 2, S = W / 32;           // wave tile, 32 x 32 products of it
  constexpr int kCopies = TILE * 2 / 8 / 4;         // 1 KB copies a wave and stage
  __shared__ __attribute__((aligned(16))) char lds[2][2 * TILE * kRowB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t c = blockIdx.z;

  int ti, tj;
  if constexpr (EPI == kGram || EPI == kSquare) {   // tiles on and above the diagonal, row by row
    int left = blockIdx.x;
    ti = 0;
    while (left >= g.tiles_m - ti) left -= g.tiles_m - ti++;
    tj = ti + left;
  } else {
    ti = blockIdx.x / g.tiles_n;
    tj = blockIdx.x % g.tiles_n;
  }
  const int64_t i0 = (int64_t)ti * TILE, j0 = (int64_t)tj * TILE;
  const int64_t pitch = g.kdim * 4;                 // bytes of a split row
  const __amdgpu_buffer_rsrc_t pr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<f16*>(g.p + c * g.p_size + i0 * g.kdim * 2), (short)0, (int)(TILE * pitch), kBufferWord3);
  const __amdgpu_buffer_rsrc_t qr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<f16*>(g.q + c * g.q_size + j0 * g.kdim * 2), (short)0, (int)(TILE * pitch), kBufferWord3);

  auto issue = [&](int slot, int stage) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int piece = wave * kCopies + i;         // 8 rows: of P, then of Q
      const int row = (piece * 8) % TILE + (lane >> 3);
      const uint32_t chunk = (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
      const uint32_t off = (uint32_t)(row * pitch) + chunk * 16u + (uint32_t)stage * kRowB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(piece * 8 < TILE ? pr : qr, (lds_void*)(lds[slot] + piece * 1024), 16,
                                               off, 0, 0, 0);
    }
  };

  f32x16 acc[S][S];
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  const int r = lane & 31, h = lane >> 5;
  auto frag = [&](const char* base, int row, int chunk) {
    return *reinterpret_cast<const f16x8*>(base + row * kRowB + ((chunk ^ ((row >> 1) & 7)) << 4));
  };
  const int stages = (int)(g.kdim / kBK);
  issue(0, 0);
  for (int s = 0; s < stages; ++s) {
    wait_vmcnt<0>();
    lds_barrier();                                  // stage s is here, and stage s - 1 has been read
    if (s + 1 < stages) issue((s + 1) & 1, s + 1);
    const char* pb = lds[s & 1];
    const char* qb = pb + TILE * kRowB;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      f16x8 ph[S], pl[S], qh[S], ql[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        ph[i] = frag(pb, wm * W + i * 32 + r, kk * 2 + h);
        pl[i] = frag(pb, wm * W + i * 32 + r, 4 + kk * 2 + h);
        qh[i] = frag(qb, wn * W + i * 32 + r, kk * 2 + h);
        ql[i] = frag(qb, wn * W + i * 32 + r, 4 + kk * 2 + h);
      }
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[i], ql[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[i], qh[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[i], qh[j], acc[i][j], 0, 0, 0);
        }
    }
  }

  // lane holds C[8 (e / 4) + 4 h + e % 4][r] of each 32 x 32 product
  const f16* own = g.own + c * g.c_size;
  f16* out = g.out + c * g.c_size;
  f16* out_t = g.out_t + c * g.c_size;
  const float lr = m.lr * m.scale, keep = 1.f - m.lr * m.decay;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int64_t row = i0 + wm * W + i * 32 + e4 * 8 + h * 4;
        const int64_t col = j0 + wn * W + j * 32 + r;
        f16x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = acc[i][j][e4 * 4 + e] * kRScale;
          const int64_t at = split_at(row + e, g.c_cols, col);
          if constexpr (EPI == kSquare) v = g.cb * split_get(own, at) + g.cc * v;
          if constexpr (EPI == kApply || EPI == kLast) v = g.ca * split_get(own, at) + v;
          if constexpr (EPI == kLast) {
            if (row + e < m.n && col < m.k) {
              const int64_t o = (c * m.n + row + e) * m.k + col;
              const float w = v * kRScale;
              put1<BF16>(m.w_out, o, m.w ? get1<BF16>(m.w, o) * keep - lr * w : w);
            }
          } else {
            hi[e] = (f16)v;
            lo[e] = (f16)(v - (float)hi[e]);
            out[at] = hi[e];
            out[at + 32] = lo[e];
          }
        }
        if constexpr (EPI != kLast) {
          if (EPI == kApply || ti != tj) {
            f16* t = out_t + split_at(col, g.ct_cols, row);
            *reinterpret_cast<f16x4*>(t) = hi;
            *reinterpret_cast<f16x4*>(t + 32) = lo;
          }
        }
      }
}

template <int TILE, int EPI, bool BF16 = false>
hipError_t product(const ProductArgs& g, const MuonArgs& m, hipStream_t s) {
  const int tiles = EPI == kGram || EPI == kSquare ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
  hipLaunchKernelGGL((muon_product<TILE, EPI, BF16>), dim3((unsigned)tiles, 1, (unsigned)m.count), dim3(kThreads), 0,
                     s, g, m);
  return hipGetLastError();
}

template <int TILE>
hipError_t steps(const MuonPlan& p, const MuonArgs& m, bool bf16, char* ws, hipStream_t s) {
  f16* x = reinterpret_cast<f16*>(ws + p.x);
  f16* xt[2] = {reinterpret_cast<f16*>(ws + p.xt0), reinterpret_cast<f16*>(ws + p.xt1)};
  f16* a = reinterpret_cast<f16*>(ws + p.a);
  f16* b = reinterpret_cast<f16*>(ws + p.b);
  const int64_t xs = p.rp * p.lp * 2, as = p.rp * p.rp * 2;
  const int tr = (int)(p.rp / TILE), tl = (int)(p.lp / TILE);
  for (int i = 0; i < m.steps; ++i) {
    const bool last = i + 1 == m.steps;
    f16 *now = xt[i & 1], *next = xt[(i + 1) & 1];
    hipError_t e;
    const ProductArgs gram{x, x, x, a, a, xs, xs, as, p.lp, p.rp, p.rp, tr, tr, m.ca, m.cb, m.cc};
    if ((e = product<TILE, kGram>(gram, m, s)) != hipSuccess) return e;
    const ProductArgs square{a, a, a, b, b, as, as, as, p.rp, p.rp, p.rp, tr, tr, m.ca, m.cb, m.cc};
    if ((e = product<TILE, kSquare>(square, m, s)) != hipSuccess) return e;
    if (!last) {
      const ProductArgs apply{b, now, x, x, next, as, xs, xs, p.rp, p.lp, p.rp, tr, tl, m.ca, m.cb, m.cc};
      e = product<TILE, kApply>(apply, m, s);
    } else {
      // the result's own orientation: rows n, columns k
      ProductArgs end{b, now, x, x, x, as, xs, xs, p.rp, p.lp, p.rp, tr, tl, m.ca, m.cb, m.cc};
      if (m.n > m.k) end = ProductArgs{now, b, now, x, x, xs, as, xs, p.rp, p.rp, p.lp, tl, tr, m.ca, m.cb, m.cc};
      e = bf16 ? product<TILE, kLast, true>(end, m, s) : product<TILE, kLast, false>(end, m, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

MuonPlan plan_muon(int count, int64_t n, int64_t k) {
  MuonPlan p{};
  p.r = std::min(n, k);
  p.l = std::max(n, k);
  p.tile = p.r > 256 ? 128 : 64;
  p.rp = (p.r + p.tile - 1) / p.tile * p.tile;
  p.lp = (p.l + p.tile - 1) / p.tile * p.tile;
  p.parts = std::min<int64_t>(1024, (n * k + 4 * kThreads - 1) / (4 * kThreads));
  const size_t c = (size_t)count;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  p.u = take(c * (size_t)(n * k) * 4);
  p.sums = take(c * (size_t)p.parts * 8);
  p.x = take(c * (size_t)(p.rp * p.lp) * 4);
  p.xt0 = take(c * (size_t)(p.rp * p.lp) * 4);
  p.xt1 = take(c * (size_t)(p.rp * p.lp) * 4);
  p.a = take(c * (size_t)(p.rp * p.rp) * 4);
  p.b = take(c * (size_t)(p.rp * p.rp) * 4);
  p.workspace_bytes = at;
  return p;
}

hipError_t launch_muon(const MuonPlan& p, const MuonArgs& a, bool bf16, char* ws, hipStream_t s) {
  float* u = reinterpret_cast<float*>(ws + p.u);
  double* sums = reinterpret_cast<double*>(ws + p.sums);
  const dim3 g1((unsigned)p.parts, (unsigned)a.count);
  if (bf16) hipLaunchKernelGGL((muon_momentum<true>), g1, dim3(kThreads), 0, s, a, u, sums);
  else hipLaunchKernelGGL((muon_momentum<false>), g1, dim3(kThreads), 0, s, a, u, sums);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool wide = a.n <= a.k;
  const int64_t np = wide ? p.rp : p.lp, kp = wide ? p.lp : p.rp;
  f16* x = reinterpret_cast<f16*>(ws + p.x);
  f16* xt = reinterpret_cast<f16*>(ws + p.xt0);
  hipLaunchKernelGGL(muon_split, dim3((unsigned)(kp / 32), (unsigned)(np / 32), (unsigned)a.count), dim3(kThreads), 0,
                     s, u, sums, (int)p.parts, a.eps, a.n, a.k, np, kp, wide ? x : xt, wide ? xt : x);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return p.tile == 128 ? steps<128>(p, a, bf16, ws, s) : steps<64>(p, a, bf16, ws, s);
}

}  // namespace sherry
