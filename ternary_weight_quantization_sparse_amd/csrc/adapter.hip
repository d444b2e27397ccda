// Low-rank adapters of many requests beside one packed projection.
//
//   y[m] = (T alpha) x[m] + B_c (scale_c A_c x[m]),   c = ids[m]
//
// Two low-rank products around the packed one: v[m] = scale_c A_c x[m] (rank
// values a token), then B_c v[m] added to the packed product's fp32 result
// before y is rounded.
//
// Decode is two launches: the packed product's K ranges with v beside them (the
// same launch), and adapter_finish.  Latency and the call's host side bound it: 16 tokens x 16384 x
// 2048 with rank 64, 8.1 us and 8.6 us (34 MB of b), 18 us a call; by itself
// the packed product's call takes 17.  Prefill is v, then the packed product's GEMM
// with B_c v in its epilogue: 2048 tokens x 16384 x 2048, rank 64, 13 us and 149
// us (at the clocks of a long loop; 179 in the first calls); without adapters that GEMM takes 123.
#include <algorithm>

#include "ops_internal.h"

namespace sherry {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Decode: y = (sum of the packed product's K ranges, in order) * alpha + B_c v.
// G lanes read one output's row of b (16 bytes a lane, so an instruction reads
// consecutive memory: a thread per output, its row read alone, took 51 us for
// 16 x 16384 outputs of rank 64), G outputs of a group in turn, and lane j keeps the j-th.
template <int G, bool YBF16>
__global__ __launch_bounds__(256) void adapter_finish(AdapterArgs ad, const float* __restrict__ partial, int splits,
                                                      const float* __restrict__ alpha, int gran,
                                                      const float* __restrict__ v, int64_t n, void* __restrict__ y) {
  const int lane = threadIdx.x & 63, j = lane % G;
  const int64_t col0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & ~63);   // of the wave's 64 outputs
  const int64_t token = blockIdx.y, col = col0 + lane;
  if (col0 >= n) return;
  // b's rows are on their way while the partials are added
  const int c = adapter_of(ad, token);
  const int live = c < 0 ? 0 : adapter_rank(ad, c) - 8 * j;   // of this lane's 8 columns
  const uint16_t* b = ad.b + ((int64_t)(c < 0 ? 0 : c) * n + col0 + (lane - j)) * ad.rank + 8 * j;
  u32x4 rows[G];
#pragma unroll
  for (int i = 0; i < G; ++i)
    rows[i] = live > 0 && col - j + i < n ? *reinterpret_cast<const u32x4*>(b + (int64_t)i * ad.rank) : u32x4{0u, 0u, 0u, 0u};
  const int64_t per = gridDim.y * n;
  const float* p = partial + token * n + (col < n ? col : n - 1);
  float s = 0.f;
  for (int z = 0; z < splits; z += 16) {   // 16 loads ahead of their adds (one latency per 16 ranges)
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = z + i < splits ? p[(z + i) * per] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (z + i < splits) s += t[i];
  }
  if (gran == SHERRY_PER_CHANNEL) s *= alpha[col < n ? col : n - 1];
  if (gran == SHERRY_PER_TENSOR) s *= alpha[0];
  if (c >= 0) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < live ? v[token * ad.rank + 8 * j + e] : 0.f;
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
// rows, B operand: the tokens).  The workgroup's waves take every 8th 64 k (a
// memory line of each row: two steps, lane q with 16 consecutive values), two
// in flight each, and add their sums through LDS in wave order.  The tile's adapters, in rising order, go to kShrinkSlots workgroups in
// turn, so a tile in which one request ends and the next begins takes no
// longer.  v is kept as the bf16 terms that the product's epilogue multiplies.
// Latency bounds it (look up the adapter, its rank, the rows): 2048 tokens x
// 64 rows x 2048 k in 13.9 us with four row tiles a workgroup, 17.6 with one; 517
// tokens x 16 rows in 7.1 with one, so ranks up to 16 take one.
constexpr int kShrinkWaves = 8, kShrinkAhead = 4, kShrinkSlots = 2;
template <int kShrinkRows>
__global__ __launch_bounds__(64 * kShrinkWaves) void adapter_shrink_mfma(AdapterArgs ad, const uint16_t* __restrict__ x,
                                                                         int64_t k, int64_t tokens,
                                                                         uint16_t* __restrict__ v) {
  __shared__ f32x4 part[kShrinkWaves][kShrinkRows][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int r0 = blockIdx.y * (16 * kShrinkRows);
  const int64_t token = (int64_t)blockIdx.x * 16 + r;
  const int id = token < tokens ? ad.ids[token] : -1;
  const uint16_t* xr = x + (token < tokens ? token : tokens - 1) * k + 16 * q;
  const int chunks = (int)(k / 64);
  // the first turn's tokens are on their way while the adapters are looked up
  // (a step past the end repeats the turn's first one; it is not added)
  auto at = [&](int s, int u) {
    const int chunk = s + u / 2 * kShrinkWaves;
    return (int64_t)(chunk < chunks ? chunk : s) * 64 + u % 2 * 8;
  };
  u32x4 x0[kShrinkAhead];
#pragma unroll
  for (int u = 0; u < kShrinkAhead; ++u)
    x0[u] = wave < chunks ? *reinterpret_cast<const u32x4*>(xr + at(wave, u)) : u32x4{0u, 0u, 0u, 0u};
  int slot = 0;
  for (int done = -1;; slot = (slot + 1) % kShrinkSlots) {
    int next = id > done && id < ad.count ? id : ad.count;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) next = min(next, __shfl_xor(next, o));
    const int c = __builtin_amdgcn_readfirstlane(next);
    if (c >= ad.count) break;
    done = c;
    if (slot != (int)blockIdx.z) continue;
    // rows past the stored ones repeat the last; sums of rows past the rank are not used
    const uint16_t* ar[kShrinkRows];
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i)
      ar[i] = ad.a + ((int64_t)c * ad.rank + min(r0 + i * 16 + r, ad.rank - 1)) * k + 16 * q;
    const int rank = adapter_rank(ad, c);
    const float scale = ad.scale[c];
    f32x4 acc[kShrinkRows];
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < chunks; s += kShrinkAhead / 2 * kShrinkWaves) {
      u32x4 xv[kShrinkAhead], av[kShrinkAhead][kShrinkRows];
#pragma unroll
      for (int u = 0; u < kShrinkAhead; ++u) {
        xv[u] = s == wave ? x0[u] : *reinterpret_cast<const u32x4*>(xr + at(s, u));
#pragma unroll
        for (int i = 0; i < kShrinkRows; ++i) av[u][i] = *reinterpret_cast<const u32x4*>(ar[i] + at(s, u));
      }
#pragma unroll
      for (int u = 0; u < kShrinkAhead; ++u)
        if (s + u / 2 * kShrinkWaves < chunks)
#pragma unroll
          for (int i = 0; i < kShrinkRows; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[u][i]),
                                                             __builtin_bit_cast(bf16x8, xv[u]), acc[i], 0, 0, 0);
    }
    if (r0 >= rank) continue;
    __syncthreads();   // the last adapter's sums have been read
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    const int row = r0 + wave * 16 + 4 * q;   // D[row 4q + e][token r]
    if (wave < kShrinkRows && id == c && row < ad.rank) {
      f32x4 s = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) s += part[w][wave][lane];
      uint32_t term[kAdapterTerms][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float rest = s[e] * scale;
        const bool finite = __builtin_isfinite(rest);
#pragma unroll
        for (int t = 0; t < kAdapterTerms; ++t) {
          uint32_t h = __builtin_bit_cast(uint16_t, (__bf16)rest);
          // what lies beyond the largest bf16 stays finite; infinities and NaN have no further terms
          if ((h & 0x7FFFu) == 0x7F80u && finite) h -= 1;
          term[t][e] = t == 0 || finite ? h : 0u;
          rest -= __uint_as_float(h << 16);
        }
      }
#pragma unroll
      for (int t = 0; t < kAdapterTerms; ++t)
        *reinterpret_cast<uint2*>(v + (t * tokens + token) * ad.rank + row) =
            make_uint2(term[t][0] | (term[t][1] << 16), term[t][2] | (term[t][3] << 16));
    }
  }
}

}  // namespace

AdapterPlan plan_adapter(int64_t n, int64_t k, int gran, int group_size, int64_t tokens, int rank, bool decode) {
  AdapterPlan p{};
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  if (decode) {
    const int splits = plan_gemv(n, k, gran, group_size, (int)tokens, 1).ksplit;
    p.v_offset = up((size_t)splits * (size_t)tokens * (size_t)n * 4);
  } else {
    p.v_offset = up(plan_gemm(n, k, gran, group_size, tokens, true).workspace_bytes);
  }
  p.workspace_bytes = p.v_offset + up((size_t)tokens * (size_t)rank * (decode ? 4 : 2 * kAdapterTerms));
  return p;
}

hipError_t launch_adapter_gemv(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int batch, void* y,
                               bool y_bf16, const AdapterArgs& ad, char* ws, hipStream_t s) {
  float* v = reinterpret_cast<float*>(ws + p.v_offset);
  float* partial = reinterpret_cast<float*>(ws + p.partial_offset);
  const GemvPlan g = plan_gemv(n, k, gran, group_size, batch, 1);
  const hipError_t e = launch_gemv_partials(g, n, k, gran, group_size, packed, alpha, x, batch, partial,
                                            AdapterShrink{ad, v, batch, 0}, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((n + 255) / 256), (unsigned)batch);
#define SHERRY_FINISH(G)                                                                                             \
  do {                                                                                                               \
    if (y_bf16)                                                                                                      \
      hipLaunchKernelGGL((adapter_finish<G, true>), grid, dim3(256), 0, s, ad, partial, g.ksplit, alpha, gran, v, n, \
                         y);                                                                                         \
    else                                                                                                             \
      hipLaunchKernelGGL((adapter_finish<G, false>), grid, dim3(256), 0, s, ad, partial, g.ksplit, alpha, gran, v,   \
                         n, y);                                                                                      \
  } while (0)
  if (ad.rank <= 8) SHERRY_FINISH(1);
  else if (ad.rank <= 16) SHERRY_FINISH(2);
  else if (ad.rank <= 32) SHERRY_FINISH(4);
  else if (ad.rank <= 64) SHERRY_FINISH(8);
  else if (ad.rank <= 128) SHERRY_FINISH(16);
  else SHERRY_FINISH(32);
#undef SHERRY_FINISH
  return hipGetLastError();
}

hipError_t launch_adapter_gemm(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m, uint16_t* y,
                               const AdapterArgs& ad, char* ws, hipStream_t s) {
  uint16_t* v = reinterpret_cast<uint16_t*>(ws + p.v_offset);
  const unsigned tiles = (unsigned)((m + 15) / 16);
  if (ad.rank <= 16)
    hipLaunchKernelGGL(adapter_shrink_mfma<1>, dim3(tiles, 1, kShrinkSlots), dim3(64 * kShrinkWaves), 0, s, ad, x, k, m,
                       v);
  else
    hipLaunchKernelGGL(adapter_shrink_mfma<4>, dim3(tiles, (unsigned)((ad.rank + 63) / 64), kShrinkSlots),
                       dim3(64 * kShrinkWaves), 0, s, ad, x, k, m, v);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GemmPlan g = plan_gemm(n, k, gran, group_size, m, true);
  const AdapterTerm term{ad, v, m * ad.rank};
  return launch_gemm_adapted(g, n, k, gran, group_size, packed, alpha, x, m, y,
                             reinterpret_cast<float*>(ws + p.partial_offset), term, s);
}

}  // namespace sherry
