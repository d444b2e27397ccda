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

// Decode: y = base + B_c v, a thread per output.
template <bool YBF16>
__global__ __launch_bounds__(256) void adapter_expand(AdapterArgs ad, const float* __restrict__ base,
                                                      const float* __restrict__ v, int64_t n, void* __restrict__ y) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t token = blockIdx.y;
  if (col >= n) return;
  float s = base[token * n + col];
  const int c = adapter_of(ad, token);
  if (c >= 0) {
    const int rank = adapter_rank(ad, c);
    const uint16_t* b = ad.b + ((int64_t)c * n + col) * ad.rank;
    float d = 0.f;
    for (int r = 0; r < rank; ++r) d += bf16_to_f32(b[r]) * v[token * ad.rank + r];
    s += d;
  }
  if constexpr (YBF16) static_cast<uint16_t*>(y)[token * n + col] = __builtin_bit_cast(uint16_t, (__bf16)s);
  else static_cast<float*>(y)[token * n + col] = s;
}

// Prefill: v of 16 tokens on MFMA (A operand: 16 rows of a, B operand: the
// tokens), one pass over the workgroup's K range for each adapter in use among
// them and each 64 of its rows.  The workgroup's four waves take the 32-k
// steps in turn and add their sums through LDS, in wave order.
__global__ __launch_bounds__(256) void adapter_shrink_mfma(AdapterArgs ad, const uint16_t* __restrict__ x, int64_t k,
                                                           int64_t tokens, int64_t k_part, float* __restrict__ v) {
  __shared__ f32x4 part[3][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t token = (int64_t)blockIdx.x * 16 + r;
  const int64_t k0 = (int64_t)blockIdx.y * k_part;
  const int id = token < tokens ? ad.ids[token] : -1;
  const uint16_t* xr = x + (token < tokens ? token : tokens - 1) * k + k0 + 8 * q;
  v += (int64_t)blockIdx.y * tokens * ad.rank;
  for (int done = -1;;) {
    int next = id > done && id < ad.count ? id : ad.count;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) next = min(next, __shfl_xor(next, o));
    const int c = __builtin_amdgcn_readfirstlane(next);
    if (c >= ad.count) break;
    done = c;
    const int rank = adapter_rank(ad, c);
    const float scale = ad.scale[c];
    for (int r0 = 0; r0 < rank; r0 += 64) {
      const uint16_t* ar[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)   // rows past the stored ones repeat the last: never stored
        ar[i] = ad.a + ((int64_t)c * ad.rank + min(r0 + i * 16 + r, ad.rank - 1)) * k + k0 + 8 * q;
      f32x4 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int64_t kk = 32 * wave; kk < k_part; kk += 128) {
        const bf16x8 xv = *reinterpret_cast<const bf16x8*>(xr + kk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i * 16 < rank)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(ar[i] + kk), xv, acc[i],
                                                             0, 0, 0);
      }
      __syncthreads();
      if (wave > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave - 1][i][lane] = acc[i];
      __syncthreads();
      if (wave == 0 && id == c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = r0 + i * 16 + 4 * q;   // D[row 4q + e][token r]
          f32x4 s = acc[i];
          for (int w = 0; w < 3; ++w) s += part[w][i][lane];
          if (row < ad.rank) *reinterpret_cast<f32x4*>(v + token * ad.rank + row) = s * scale;
        }
      }
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
    p.ksplit = 1;
    p.y_offset = up(base);
    p.v_offset = p.y_offset + up((size_t)tokens * (size_t)n * 4);
  } else {
    const size_t base = plan_gemm(n, k, gran, group_size, tokens, true).workspace_bytes;
    p.ksplit = 1;
    const int64_t tiles = (tokens + 15) / 16;
    while (tiles * p.ksplit < 512 && p.ksplit < 8 && k % (128 * 2 * p.ksplit) == 0) p.ksplit *= 2;
    p.y_offset = 0;
    p.v_offset = up(base);
  }
  p.workspace_bytes = p.v_offset + up((size_t)p.ksplit * (size_t)tokens * (size_t)rank * 4);
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
  if (y_bf16) hipLaunchKernelGGL(adapter_expand<true>, grid, dim3(256), 0, s, ad, base, v, n, y);
  else hipLaunchKernelGGL(adapter_expand<false>, grid, dim3(256), 0, s, ad, base, v, n, y);
  return hipGetLastError();
}

hipError_t launch_adapter_gemm(const AdapterPlan& p, int64_t n, int64_t k, int gran, int group_size,
                               const uint8_t* packed, const float* alpha, const uint16_t* x, int64_t m, uint16_t* y,
                               const AdapterArgs& ad, char* ws, hipStream_t s) {
  float* v = reinterpret_cast<float*>(ws + p.v_offset);
  hipLaunchKernelGGL(adapter_shrink_mfma, dim3((unsigned)((m + 15) / 16), (unsigned)p.ksplit), dim3(256), 0, s, ad, x,
                     k, m, k / p.ksplit, v);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const GemmPlan g = plan_gemm(n, k, gran, group_size, m, true);
  const AdapterTerm term{ad, v, p.ksplit, m * ad.rank};
  return launch_gemm_adapted(g, n, k, gran, group_size, packed, alpha, x, m, y,
                             reinterpret_cast<float*>(ws + p.base_offset), term, s);
}

}  // namespace sherry
