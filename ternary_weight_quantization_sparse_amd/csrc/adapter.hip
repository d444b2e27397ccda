// Low-rank adapters of many requests beside one packed projection.
//
//   y[m] = (T alpha) x[m] + B_c (scale_c A_c x[m]),   c = ids[m]
//
// Two low-rank products around the packed one: v[m] = scale_c A_c x[m] (rank
// values a token), then B_c v[m] added to the packed product's fp32 result
// before y is rounded.
#include <algorithm>

#include "ops_internal.h"

namespace sherry {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ inline int adapter_of(const AdapterArgs& a, int64_t token) {
  const int c = a.ids[token];
  return c >= 0 && c < a.count ? c : -1;
}

// 8 products of bf16 pairs, added in fp32
__device__ inline float dot8(const u32x4 a, const u32x4 b, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += __uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16);
    s += __uint_as_float(a[i] & 0xFFFF0000u) * __uint_as_float(b[i] & 0xFFFF0000u);
  }
  return s;
}

// Decode: a wave per (token, row of a).
__global__ __launch_bounds__(256) void adapter_shrink(AdapterArgs ad, const uint16_t* __restrict__ x, int64_t k,
                                                      float* __restrict__ v) {
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t token = blockIdx.y;
  if (row >= ad.rank) return;
  const int c = adapter_of(ad, token);
  if (c < 0 || row >= adapter_rank(ad, c)) return;   // never read
  const u32x4* ar = reinterpret_cast<const u32x4*>(ad.a + ((int64_t)c * ad.rank + row) * k);
  const u32x4* xr = reinterpret_cast<const u32x4*>(x + token * k);
  float s = 0.f;
  for (int64_t i = lane; i < k / 8; i += 64) s = dot8(ar[i], xr[i], s);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) v[token * ad.rank + row] = s * ad.scale[c];
}

// Decode: y = base + B_c v.  G lanes read one output's row of b (16 bytes a
// lane, so an instruction reads consecutive memory: a thread per output, its
// row read alone, took 51 us for 16 x 16384 outputs of rank 64), G outputs of
// a group in turn, and lane j keeps the j-th.
template <int G, bool YBF16>
__global__ __launch_bounds__(256) void adapter_expand(AdapterArgs ad, const float* __restrict__ base,
                                                      const float* __restrict__ v, int64_t n, void* __restrict__ y) {
  const int lane = threadIdx.x & 63, j = lane % G;
  const int64_t col0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & ~63);   // of the wave's 64 outputs
  const int64_t token = blockIdx.y, col = col0 + lane;
  if (col0 >= n) return;
  float s = col < n ? base[token * n + col] : 0.f;
  const int c = adapter_of(ad, token);
  if (c >= 0) {
    const int rank = adapter_rank(ad, c), live = rank - 8 * j;   // of this lane's 8 columns
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < live ? v[token * ad.rank + 8 * j + e] : 0.f;
    const uint16_t* b = ad.b + ((int64_t)c * n + col0 + (lane - j)) * ad.rank + 8 * j;
    u32x4 rows[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
      rows[i] = live > 0 && col - j + i < n ? *reinterpret_cast<const u32x4*>(b + (int64_t)i * ad.rank) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = rows[i][e / 2];
        const float t = __uint_as_float(e % 2 ? u & 0xFFFF0000u : u << 16);
        d += e < live ? t * w[e] : 0.f;   // columns past the rank do not count, whatever they hold
      }
#pragma unroll
      for (int o = 1; o < G; o <<= 1) d += __shfl_xor(d, o);
      if (i == j) s += d;
    }
  }
  if (col >= n) return;
  if constexpr (YBF16) static_cast<uint16_t*>(y)[token * n + col] = __builtin_bit_cast(uint16_t, (__bf16)s);
  else static_cast<float*>(y)[token * n + col] = s;
}

// Prefill: v of 16 tokens and 16 kShrinkRows rows of a on MFMA (A operand: the
// rows, B operand: the tokens).  The workgroup's waves take every 8th step of
// 32 k, four steps' loads in flight each, and add their sums through LDS in wave
// order.  The tile's adapters, in rising order, go to kShrinkSlots workgroups in
// turn, so a tile in which one request ends and the next begins takes no
// longer.  v is kept as two bf16 terms, hi + lo (16 bits), as the product's
// epilogue multiplies it.
// Latency bounds it (look up the adapter, its rank, the rows): 2048 tokens x
// 64 rows x 2048 k in 13.9 us with four row tiles a workgroup, 17.6 with one; 517
// tokens x 16 rows in 7.1 with one, so ranks up to 16 take one.
constexpr int kShrinkWaves = 8, kShrinkAhead = 4, kShrinkSlots = 2;
template <int kShrinkRows>
__global__ __launch_bounds__(64 * kShrinkWaves) void adapter_shrink_mfma(AdapterArgs ad, const uint16_t* __restrict__ x,
                                                                         int64_t k, int64_t tokens,
                                                                         uint16_t* __restrict__ vh,
                                                                         uint16_t* __restrict__ vl) {
  __shared__ f32x4 part[kShrinkWaves][kShrinkRows][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int r0 = blockIdx.y * (16 * kShrinkRows);
  const int64_t token = (int64_t)blockIdx.x * 16 + r;
  const int id = token < tokens ? ad.ids[token] : -1;
  const uint16_t* xr = x + (token < tokens ? token : tokens - 1) * k + 8 * q;
  const int steps = (int)(k / 32);
  int slot = 0;
  for (int done = -1;; slot = (slot + 1) % kShrinkSlots) {
    int next = id > done && id < ad.count ? id : ad.count;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) next = min(next, __shfl_xor(next, o));
    const int c = __builtin_amdgcn_readfirstlane(next);
    if (c >= ad.count) break;
    done = c;
    if (slot != (int)blockIdx.z) continue;
    const int rank = adapter_rank(ad, c);
    if (r0 >= rank) continue;
    const float scale = ad.scale[c];
    // rows past the rank repeat its last: their sums are not used
    const uint16_t* ar[kShrinkRows];
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i)
      ar[i] = ad.a + ((int64_t)c * ad.rank + min(r0 + i * 16 + r, rank - 1)) * k + 8 * q;
    f32x4 acc[kShrinkRows];
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < steps; s += kShrinkAhead * kShrinkWaves) {
      u32x4 xv[kShrinkAhead], av[kShrinkAhead][kShrinkRows];
#pragma unroll
      for (int u = 0; u < kShrinkAhead; ++u) {
        // a step past the end repeats this turn's first one; it is not added
        const int64_t at = (int64_t)(s + u * kShrinkWaves < steps ? s + u * kShrinkWaves : s) * 32;
        xv[u] = *reinterpret_cast<const u32x4*>(xr + at);
#pragma unroll
        for (int i = 0; i < kShrinkRows; ++i) av[u][i] = *reinterpret_cast<const u32x4*>(ar[i] + at);
      }
#pragma unroll
      for (int u = 0; u < kShrinkAhead; ++u)
        if (s + u * kShrinkWaves < steps)
#pragma unroll
          for (int i = 0; i < kShrinkRows; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[u][i]),
                                                             __builtin_bit_cast(bf16x8, xv[u]), acc[i], 0, 0, 0);
    }
    __syncthreads();   // the last adapter's sums have been read
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    const int row = r0 + wave * 16 + 4 * q;   // D[row 4q + e][token r]
    if (wave < kShrinkRows && id == c && row < ad.rank) {
      f32x4 s = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) s += part[w][wave][lane];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = s[e] * scale;
        const __bf16 h = (__bf16)v;
        hi[e] = __builtin_bit_cast(uint16_t, h);
        lo[e] = __builtin_bit_cast(uint16_t, (__bf16)(v - (float)h));
      }
      *reinterpret_cast<uint2*>(vh + token * ad.rank + row) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2*>(vl + token * ad.rank + row) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
    }
  }
}

}  // namespace

AdapterPlan plan_adapter(int64_t n, int64_t k, int gran, int group_size, int64_t tokens, int rank, bool decode) {
  AdapterPlan p{};
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  p.base_offset = 0;
  if (decode) {
    const size_t base = plan_gemv(n, k, gran, group_size, (int)tokens, 1).workspace_bytes;
    p.y_offset = up(base);
    p.v_offset = p.y_offset + up((size_t)tokens * (size_t)n * 4);
  } else {
    p.v_offset = up(plan_gemm(n, k, gran, group_size, tokens, true).workspace_bytes);   // hi, then lo
  }
  p.workspace_bytes = p.v_offset + up((size_t)tokens * (size_t)rank * 4);
  return p;
}

hipError_t launch_adapter_gemv(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int batch, void* y,
                               bool y_bf16, const AdapterArgs& ad, char* ws, hipStream_t s) {
  float* v = reinterpret_cast<float*>(ws + p.v_offset);
  float* base = reinterpret_cast<float*>(ws + p.y_offset);
  hipLaunchKernelGGL(adapter_shrink, dim3((unsigned)((ad.rank + 3) / 4), (unsigned)batch), dim3(256), 0, s, ad, x, k, v);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GemvPlan g = plan_gemv(n, k, gran, group_size, batch, 1);
  e = launch_gemv(g, n, k, gran, group_size, packed, alpha, x, batch, base, false, 1, 0, 0, 0,
                  reinterpret_cast<float*>(ws + p.base_offset), s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((n + 255) / 256), (unsigned)batch);
#define SHERRY_EXPAND(G)                                                                                       \
  do {                                                                                                         \
    if (y_bf16) hipLaunchKernelGGL((adapter_expand<G, true>), grid, dim3(256), 0, s, ad, base, v, n, y);       \
    else hipLaunchKernelGGL((adapter_expand<G, false>), grid, dim3(256), 0, s, ad, base, v, n, y);             \
  } while (0)
  if (ad.rank <= 8) SHERRY_EXPAND(1);
  else if (ad.rank <= 16) SHERRY_EXPAND(2);
  else if (ad.rank <= 32) SHERRY_EXPAND(4);
  else if (ad.rank <= 64) SHERRY_EXPAND(8);
  else if (ad.rank <= 128) SHERRY_EXPAND(16);
  else SHERRY_EXPAND(32);
#undef SHERRY_EXPAND
  return hipGetLastError();
}

hipError_t launch_adapter_gemm(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m, uint16_t* y,
                               const AdapterArgs& ad, char* ws, hipStream_t s) {
  uint16_t* vh = reinterpret_cast<uint16_t*>(ws + p.v_offset);
  uint16_t* vl = vh + m * ad.rank;
  const unsigned tiles = (unsigned)((m + 15) / 16);
  if (ad.rank <= 16)
    hipLaunchKernelGGL(adapter_shrink_mfma<1>, dim3(tiles, 1, kShrinkSlots), dim3(64 * kShrinkWaves), 0, s, ad, x, k, m,
                       vh, vl);
  else
    hipLaunchKernelGGL(adapter_shrink_mfma<4>, dim3(tiles, (unsigned)((ad.rank + 63) / 64), kShrinkSlots),
                       dim3(64 * kShrinkWaves), 0, s, ad, x, k, m, vh, vl);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GemmPlan g = plan_gemm(n, k, gran, group_size, m, true);
  const AdapterTerm term{ad, vh, vl};
  return launch_gemm_adapted(g, n, k, gran, group_size, packed, alpha, x, m, y,
                             reinterpret_cast<float*>(ws + p.base_offset), term, s);
}

}  // namespace sherry
