// Distillation from a teacher's top logits, forward and backward.
//
// A row's student logits s [V], teacher logits u_j of ids i_j, temperature t,
// q = softmax(s / t), p = the teacher's probabilities of its slots (and rest =
// 1 - sum p, held against the student's mass outside the ids, where the
// teacher's own normaliser is given):
//
//   kd = t^2 (sum_j p_j log(p_j / q_ij) + rest log(rest / q_rest))
//   loss = w kd + (1 - w) (-log softmax(s)_label)
//   dloss/ds = w t ((P + rest) q - scatter(p) - [outside the ids] rest q / q_rest)
//              + (1 - w) (softmax(s) - onehot(label)),      P = sum_j p_j
//
// HBM bounds both directions: the forward pass reads the logits once (running maximum and sums), the backward pass
// reads them once more and writes the gradient: 2048 x 128000 bf16 with 64 slots 89 us (5.9 TB/s) + 12 us (the rows'
// losses) and 207 us (5.1 TB/s), 300 us together; three passes at a copy's 5.2 TB/s take 302.
// Everything that belongs to a row (sums past a 16-byte group, logarithms, the teacher's probabilities) is in 64 bits: the
// loss is a difference of terms of its own size or larger.
#include <algorithm>
#include <cfloat>

#include "ops_internal.h"

namespace sherry {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// log2(e) / t in two terms: rounded to one, every exponential of a far element would be off the same way.  The upper
// one is the next below, so that both are above zero and a distance of -infinity stays one.
constexpr float kLog2e = 1.44269502f, kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);
static_assert(kLog2eRest > 0.f, "the upper term lies below log2(e)");
__device__ inline float exp_below(float d, float c, float rest) { return __builtin_amdgcn_exp2f(fmaf(d, c, d * rest)); }
__device__ inline float exp_below(float d) { return exp_below(d, kLog2e, kLog2eRest); }   // t = 1
constexpr int kThreads = 256;
constexpr int kStatHead = kDistillHead;   // a row's statistics before its slots

template <bool BF16> constexpr int kLane = BF16 ? 8 : 4;   // elements of 16 bytes

__device__ inline int64_t load_index(const void* p, int64_t i, bool wide) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

template <bool BF16>
__device__ inline float load_one(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ inline void store_one(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
  else static_cast<float*>(p)[i] = v;
}

// A row as 16-byte groups: group g holds the elements kLane g - mis + (0 ..
// kLane - 1), mis the row's distance from the 16-byte boundary before it, so
// groups inside the row are aligned.
template <bool BF16>
struct RowGroups {
  const char* base;   // the boundary
  int mis;
  int64_t vocab, groups;
  __device__ RowGroups(const void* logits, int64_t first, int64_t vocab) : vocab(vocab) {
    const char* row = static_cast<const char*>(logits) + first * (BF16 ? 2 : 4);
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    base = row - off;
    mis = off / (BF16 ? 2 : 4);
    groups = (mis + vocab + kLane<BF16> - 1) / kLane<BF16>;
  }
  __device__ bool whole(int64_t g) const { return g * kLane<BF16> >= mis && (g + 1) * kLane<BF16> <= mis + vocab; }
  template <bool STREAM>
  __device__ u32x4 raw(int64_t g) const {
    const u32x4* p = reinterpret_cast<const u32x4*>(base + g * 16);
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
  }
  __device__ static void unpack(const u32x4 r, float (&x)[kLane<BF16>]) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
    }
  }
  // a group that reaches past the row: elements outside read -infinity
  __device__ void edge(int64_t g, float (&x)[kLane<BF16>]) const {
#pragma unroll
    for (int i = 0; i < kLane<BF16>; ++i) {
      const int64_t p = g * kLane<BF16> + i;
      x[i] = p >= mis && p < mis + vocab ? load_one<BF16>(base, p) : -INFINITY;
    }
  }
};

__device__ inline double shfl_xor_f64(double v, int o) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = __shfl_xor((uint32_t)u, o), hi = __shfl_xor((uint32_t)(u >> 32), o);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += shfl_xor_f64(v, o);
  return v;
}
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ inline double wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, shfl_xor_f64(v, o));
  return v;
}

// ------------------------------------------------------------------- forward
// One range of a row: its maximum m, sum of exp((s - m) / t) and with SOFT1 the
// sum of exp(s - m).  TAIL: of the elements outside the ids, which a bitmap of
// the range marks in LDS; so the tail is never a difference of sums, and it has a maximum of its own, however
// far below the ids it lies.  A thread adds up a group in fp32 and the groups in
// 64 bits: one fp32 sum over its whole share, 500 elements of 2048 x 128000, drops what lies 2^-24 below the
// largest and always to the same side (a loss of 5.3e-3 came out 0.4% low).  It rescales its sums when its
// maximum rises, once per four groups; threads and waves join in 64 bits.  The maximum starts at the lowest
// finite value, so that ranges of -infinity add zeros.
template <bool BF16, bool TAIL, bool SOFT1, bool STREAM>
__global__ __launch_bounds__(kThreads) void distill_range(DistillArgs a, int64_t row0) {
  constexpr int L = kLane<BF16>, kAhead = 4;
  extern __shared__ uint32_t marks[];
  __shared__ float wm[kThreads / 64];
  __shared__ double ws[kThreads / 64], ws1[kThreads / 64];
  __shared__ int twice;
  const int64_t row = row0 + blockIdx.x / a.ranges;
  const int range = (int)(blockIdx.x % a.ranges);
  const RowGroups<BF16> v(a.logits, row * a.stride, a.vocab);
  const int64_t g0 = (int64_t)range * a.range_groups;
  const int64_t g1 = min(v.groups, g0 + a.range_groups);
  const int tid = threadIdx.x;
  if constexpr (TAIL) {
    const int words = (int)((a.range_groups * L + 31) / 32);
    for (int i = tid; i < words; i += kThreads) marks[i] = 0u;
    if (tid == 0) twice = 0;
    __syncthreads();
    for (int j = tid; j < a.slots; j += kThreads) {
      const int64_t id = load_index(a.ids, row * a.slots + j, a.ids_wide);
      const int64_t p = id + v.mis - g0 * L;
      if (id < 0 || id >= a.vocab || p < 0 || p >= (g1 - g0) * L) continue;
      const uint32_t bit = 1u << (p & 31);
      if (atomicOr(&marks[p >> 5], bit) & bit) twice = 1;
    }
    __syncthreads();
  }
  float m = -FLT_MAX;
  double s = 0., s1 = 0.;
  auto drop_marked = [&](float (&x)[L], int64_t g) {
    if constexpr (TAIL) {
      const uint32_t p = (uint32_t)((g - g0) * L), mark = marks[p >> 5] >> (p & 31);
#pragma unroll
      for (int i = 0; i < L; ++i) x[i] = (mark >> i) & 1u ? -INFINITY : x[i];
    }
  };
  auto soft = [&](float d) { return exp_below(d, a.exp_hi, a.exp_lo); };
  auto add = [&](const float (&x)[L]) {
    float t = 0.f, t1 = 0.f;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float d = x[i] - m;
      t += soft(d);
      if constexpr (SOFT1) t1 += exp_below(d);
    }
    s += (double)t;
    if constexpr (SOFT1) s1 += (double)t1;
  };
  auto raise = [&](float top) {
    if (top > m) {
      s *= (double)soft(m - top);
      if constexpr (SOFT1) s1 *= (double)exp_below(m - top);
      m = top;
    }
  };
  auto peak = [](const float (&x)[L]) {
    float t = x[0];
#pragma unroll
    for (int i = 1; i < L; ++i) t = fmaxf(t, x[i]);
    return t;
  };
  // a row's first and last group may reach past it
  const int64_t w0 = g0 < g1 && !v.whole(g0) ? g0 + 1 : g0;
  const int64_t w1 = g1 > w0 && !v.whole(g1 - 1) ? g1 - 1 : g1;
  if (tid < 2) {
    const int64_t g = tid == 0 ? g0 : g1 - 1;
    if (tid == 0 ? w0 > g0 : w1 < g1) {
      float x[L];
      v.edge(g, x);
      drop_marked(x, g);
      raise(peak(x));
      add(x);
    }
  }
  for (int64_t g = w0 + tid; g < w1; g += kAhead * kThreads) {
    u32x4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (g + u * kThreads < w1) r[u] = v.template raw<STREAM>(g + u * kThreads);
    float x[kAhead][L], top = -FLT_MAX;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (g + u * kThreads < w1) {
        v.unpack(r[u], x[u]);
        drop_marked(x[u], g + u * kThreads);
        top = fmaxf(top, peak(x[u]));
      }
    raise(top);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (g + u * kThreads < w1) add(x[u]);
  }
  const float wmax = wave_max(m);
  const double sum = wave_sum(s * (double)soft(m - wmax));
  double sum1 = 0.;
  if constexpr (SOFT1) sum1 = wave_sum(s1 * (double)exp_below(m - wmax));
  if ((tid & 63) == 0) {
    wm[tid >> 6] = wmax;
    ws[tid >> 6] = sum;
    ws1[tid >> 6] = sum1;
  }
  __syncthreads();
  if (tid == 0) {
    DistillRange out{0., 0., wm[0], TAIL ? twice : 0};
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) out.m = fmaxf(out.m, wm[w]);
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      out.s += ws[w] * (double)soft(wm[w] - out.m);
      out.s1 += ws1[w] * (double)exp_below(wm[w] - out.m);
    }
    a.part[row * a.ranges + range] = out;
  }
}

// A row's loss and, for the backward pass, two references and the factors of
// the exponentials below them (m: off exp((s - m) / t) + c1 exp(s - m) for the
// elements outside the ids; top: at and c2 for those at the ids), then each
// slot's probability; all with the weights and the temperature in them.  One
// wave a row: ranges, then slots, 64 at a time.
template <bool BF16, bool T_BF16>
__global__ __launch_bounds__(64) void distill_finish(DistillArgs a, int64_t row0) {
  __shared__ int32_t ids[kDistillSlots];
  __shared__ double prob[kDistillSlots];
  const int64_t row = row0 + blockIdx.x;
  const int lane = threadIdx.x;
  const double inv_t = a.inv_t, inf = INFINITY;
  const bool tail = a.teacher_lse != nullptr;
  const int64_t label = a.labels ? load_index(a.labels, row, a.labels_wide) : -1;
  const bool has_label = label >= 0 && label < a.vocab;

  const DistillRange* part = a.part + row * a.ranges;
  float m = -FLT_MAX;
  int twice = 0;
  for (int r = lane; r < a.ranges; r += 64) {
    m = fmaxf(m, part[r].m);
    twice |= part[r].twice;
  }
  m = wave_max(m);
  twice = __any(twice);
  double s = 0., s1 = 0.;
  for (int r = lane; r < a.ranges; r += 64) {
    const double d = (double)part[r].m - (double)m;
    s += part[r].s * exp(d * inv_t);
    s1 += part[r].s1 * exp(d);
  }
  s = wave_sum(s);
  s1 = wave_sum(s1);

  // the teacher's probabilities
  const double lse = tail ? (double)a.teacher_lse[row] : 0.;
  double top = -inf;
  for (int j = lane; j < a.slots; j += 64) {
    const int64_t id = load_index(a.ids, row * a.slots + j, a.ids_wide);
    const bool used = id >= 0 && id < a.vocab;
    ids[j] = used ? (int32_t)id : -1;
    const double u = used ? (double)load_one<T_BF16>(a.teacher, row * a.slots + j) * inv_t : -inf;
    prob[j] = u;
    if (!(u <= top) && !(top != top)) top = u;   // (a NaN stays)
  }
  if (!tail) {
    const bool bad = __any(top != top);
    top = bad ? (double)NAN : wave_max(top);
  }
  const double ref = tail ? lse : top;
  const bool teach = tail || !(top == -inf);
  double mass = 0.;
  for (int j = lane; j < a.slots; j += 64) {
    const double u = prob[j];
    mass += u == -inf || !teach ? 0. : exp(u - ref);
  }
  mass = wave_sum(mass);
  const double norm = tail || !teach ? 1. : 1. / mass, lognorm = tail || !teach ? 0. : log(mass);
  double rest = 0.;
  if (tail) {
    rest = 1. - mass;
    if (rest <= 0.) rest = 0.;
  } else {
    mass = teach ? 1. : 0.;
    if (top != top) mass = top;
  }
  __syncthreads();

  // student: the ids' exponentials join the sums (TAIL left them out), an id
  // that stands in several slots once; the larger of both maxima is the reference
  auto logit = [&](int64_t id) { return (double)load_one<BF16>(a.logits, row * a.stride + id); };
  double top_s = (double)m, cross = 0.;
  int distinct = 0;
  if (tail) {
    for (int j = lane; j < a.slots; j += 64)
      if (ids[j] >= 0) top_s = fmax(top_s, logit(ids[j]));
    top_s = wave_max(top_s);
  }
  const double below = (double)m - top_s, left = s;
  s *= exp(below * inv_t);
  s1 *= exp(below);
  if (tail) {
    double in_t = 0., in_1 = 0.;
    for (int j = lane; j < a.slots; j += 64) {
      if (ids[j] < 0) continue;
      bool first = true;
      if (twice)
        for (int i = 0; i < j; ++i) first = first && ids[i] != ids[j];
      if (!first) continue;
      ++distinct;
      const double d = logit(ids[j]) - top_s;
      in_t += exp(d * inv_t);
      in_1 += exp(d);
    }
    s += wave_sum(in_t);
    s1 += wave_sum(in_1);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) distinct += __shfl_xor(distinct, o);
    if (distinct == a.vocab) rest = 0.;   // nothing is outside the ids
  }
  const double logs = log(s);
  for (int j = lane; j < a.slots; j += 64) {
    const double u = prob[j];
    const double p = u == -inf || !teach ? 0. : exp(u - ref) * norm;
    if (p != 0. && ids[j] >= 0) cross += p * (u - ref - lognorm - ((logit(ids[j]) - top_s) * inv_t - logs));
    prob[j] = p;
  }
  cross = wave_sum(cross);
  if (rest != 0.) cross += rest * (log(rest) - (log(left) + below * inv_t - logs));
  const double w = a.kd_weight, t = 1. / inv_t;
  double loss = w == 0. ? 0. : w * t * t * cross;
  const double one = a.inv_t == 1. ? s : s1;   // the sum of exp(s - top_s)
  const double hard = has_label ? 1. - w : 0.;
  if (hard != 0.) loss += hard * (log(one) - (logit(label) - top_s));
  if (lane == 0) a.loss[row] = (float)loss;
  if (!a.stats) return;
  float* st = a.stats + row * (kStatHead + a.slots);
  if (lane == 0) {
    const double soft = w * t, all = w == 0. || mass + rest == 0. ? 0. : soft * (mass + rest) / s;
    const double out = w == 0. || rest == 0. || left == 0. ? 0. : soft * rest / left;
    double at = all, off = all * exp(below * inv_t) - out, c2 = hard == 0. ? 0. : hard / one, c1 = c2 * exp(below);
    if (a.inv_t == 1.) {
      at += c2;
      off += c1;
      c1 = c2 = 0.;
    }
    st[0] = m;
    st[1] = (float)off;
    st[2] = (float)c1;
    st[3] = (float)top_s;
    st[4] = (float)at;
    st[5] = (float)c2;
  }
  for (int j = lane; j < a.slots; j += 64) st[kStatHead + j] = w == 0. ? 0.f : (float)(w * t * prob[j]);
}

// ------------------------------------------------------------------ backward
// One range of a row: gradient = g (off exp((s - m) / t) + c1 exp(s - m)) of the statistics,
// then the elements at the ids and the label over it.  Those values are made
// before the range is written, so that the gradient may take the logits'
// place.  An id in several slots takes the sum of its slots' probabilities in
// slot order, whichever slot writes it.
template <bool BF16, bool SOFT1, bool STREAM>
__global__ __launch_bounds__(kThreads) void distill_grad(DistillGrad a, int64_t row0) {
  constexpr int L = kLane<BF16>, kAhead = 4;
  __shared__ int32_t ids[kDistillSlots];
  __shared__ float prob[kDistillSlots];
  const int64_t row = row0 + blockIdx.x / a.ranges;
  const int range = (int)(blockIdx.x % a.ranges);
  const RowGroups<BF16> v(a.logits, row * a.stride, a.vocab);
  const int64_t g0 = (int64_t)range * a.range_groups, g1 = min(v.groups, g0 + a.range_groups);
  if (g0 >= g1) return;
  const int64_t e0 = max(g0 * L - v.mis, (int64_t)0), e1 = min(g1 * L - v.mis, a.vocab);   // its elements
  const int tid = threadIdx.x;
  const float gr = a.g[row];
  const int64_t first = row * a.out_stride;
  // where the output's rows stand at the same distance from a boundary, groups are stored whole
  char* ob = static_cast<char*>(a.out) + first * (BF16 ? 2 : 4) - v.mis * (BF16 ? 2 : 4);
  const bool same = (reinterpret_cast<uintptr_t>(ob) & 15) == 0;
  if (gr == 0.f) {   // nothing of the row counts, whatever it holds
    for (int64_t g = g0 + tid; g < g1; g += kThreads) {
      if (same && v.whole(g)) {
        *reinterpret_cast<u32x4*>(ob + g * 16) = u32x4{0u, 0u, 0u, 0u};
      } else {
        for (int i = 0; i < L; ++i) {
          const int64_t e = g * L + i - v.mis;
          if (e >= 0 && e < a.vocab) store_one<BF16>(a.out, first + e, 0.f);
        }
      }
    }
    return;
  }
  const float* st = a.stats + row * (kStatHead + a.slots);
  const float m = st[0], off = st[1] * gr, c1 = st[2] * gr, top = st[3], at = st[4] * gr, c2 = st[5] * gr;
  auto value = [&](float x, float reference, float f, float f1) {
    const float d = x - reference;
    float r = f == 0.f ? 0.f : f * exp_below(d, a.exp_hi, a.exp_lo);
    if constexpr (SOFT1) r += f1 == 0.f ? 0.f : f1 * exp_below(d);
    return r;
  };

  // the elements at the ids and the label in this range
  for (int j = tid; j < a.slots; j += kThreads) {
    const int64_t id = load_index(a.ids, row * a.slots + j, a.ids_wide);
    ids[j] = id >= e0 && id < e1 ? (int32_t)id : -1;
    prob[j] = st[kStatHead + j];
  }
  const int64_t lab = a.labels ? load_index(a.labels, row, a.labels_wide) : -1;
  const int32_t label = lab >= e0 && lab < e1 ? (int32_t)lab : -1;
  const float hard = (1.f - a.kd_weight) * gr;
  __syncthreads();
  float fix[kDistillSlots / kThreads];
#pragma unroll
  for (int u = 0; u < kDistillSlots / kThreads; ++u) {
    const int j = tid + u * kThreads;
    if (j >= a.slots || ids[j] < 0) continue;
    float p = 0.f;
    for (int i = 0; i < a.slots; ++i) p += ids[i] == ids[j] ? prob[i] : 0.f;
    fix[u] = value(load_one<BF16>(a.logits, row * a.stride + ids[j]), top, at, c2) - p * gr - (ids[j] == label ? hard : 0.f);
  }
  float label_fix = 0.f;
  bool label_here = false;
  if (tid == 0 && label >= 0) {
    label_here = true;
    for (int i = 0; i < a.slots; ++i) label_here = label_here && ids[i] != label;
    label_fix = value(load_one<BF16>(a.logits, row * a.stride + label), m, off, c1) - hard;
  }
  __syncthreads();

  auto store = [&](const float (&x)[L], int64_t g, bool whole) {
    float r[L];
#pragma unroll
    for (int i = 0; i < L; ++i) r[i] = value(x[i], m, off, c1);
    if (same && whole) {
      u32x4 o;
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)r[2 * i]) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)r[2 * i + 1]) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(r[i]);
      }
      if constexpr (STREAM) __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(ob + g * 16));
      else *reinterpret_cast<u32x4*>(ob + g * 16) = o;
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int64_t e = g * L + i - v.mis;
        if (e >= 0 && e < a.vocab) store_one<BF16>(a.out, first + e, r[i]);
      }
    }
  };
  const int64_t w0 = !v.whole(g0) ? g0 + 1 : g0;
  const int64_t w1 = g1 > w0 && !v.whole(g1 - 1) ? g1 - 1 : g1;
  if (tid < 2) {
    const int64_t g = tid == 0 ? g0 : g1 - 1;
    if (tid == 0 ? w0 > g0 : w1 < g1) {
      float x[L];
      v.edge(g, x);
      store(x, g, false);
    }
  }
  for (int64_t g = w0 + tid; g < w1; g += kAhead * kThreads) {
    u32x4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (g + u * kThreads < w1) r[u] = v.template raw<STREAM>(g + u * kThreads);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (g + u * kThreads < w1) {
        float x[L];
        v.unpack(r[u], x);
        store(x, g + u * kThreads, true);
      }
  }
  __syncthreads();   // the range is written: the ids' and the label's elements over it
#pragma unroll
  for (int u = 0; u < kDistillSlots / kThreads; ++u) {
    const int j = tid + u * kThreads;
    if (j < a.slots && ids[j] >= 0) store_one<BF16>(a.out, first + ids[j], fix[u]);
  }
  if (label_here) store_one<BF16>(a.out, first + label, label_fix);
}

// Logits that the last-level cache (256 MB) cannot keep from one pass to the next are streamed past it, and so are
// their gradients: 2048 x 128000 bf16, both directions, 332 -> 302 us.  Smaller ones find them there (333 x 50001
// fp32: 123 us a call by itself, streamed 138).
bool streams(int64_t rows, int64_t vocab, bool bf16) { return rows * vocab * (bf16 ? 2 : 4) > (int64_t)192 << 20; }

// Rows of a launch: at most 2^22 workgroups (2^30 threads).
int64_t rows_of_launch(int ranges) { return std::max<int64_t>(1, ((int64_t)1 << 22) / ranges); }

}  // namespace

// Ranges of a row: about 2048 workgroups, about 4096 elements each or more (16 a
// thread; 4096 and 8192 workgroups took as long), at most 2^18 (the bitmap's 32 KB); backward 16384 elements (8192
// as long, 32768 and 65536 5% longer).  A range is whole groups; one
// group more than the row's own covers a row that begins inside a group.
DistillSplit plan_distill(int64_t rows, int64_t vocab, bool bf16, bool backward) {
  const int64_t lane = bf16 ? 8 : 4, groups = (vocab + lane - 1) / lane + 1;
  DistillSplit p{};
  int64_t ranges;
  if (backward) {
    ranges = (vocab + 16384 - 1) / 16384;
  } else {
    ranges = std::min<int64_t>((2048 + rows - 1) / rows, (vocab + 4095) / 4096);
    ranges = std::max<int64_t>(ranges, (groups * lane + (1 << 18) - 1) >> 18);
  }
  ranges = std::max<int64_t>(ranges, 1);
  p.range_groups = (groups + ranges - 1) / ranges;
  p.ranges = (int)((groups + p.range_groups - 1) / p.range_groups);
  p.workspace_bytes = (size_t)rows * (size_t)p.ranges * sizeof(DistillRange);
  return p;
}

hipError_t launch_distill(const DistillArgs& a, int64_t rows, bool bf16, bool teacher_bf16, hipStream_t s) {
  const bool tail = a.teacher_lse != nullptr, soft1 = a.labels && a.inv_t != 1.;
  const size_t lds = tail ? (size_t)((a.range_groups * (bf16 ? 8 : 4) + 31) / 32) * 4 : 0;
  const int64_t step = rows_of_launch(a.ranges);
  const bool stream = streams(rows, a.vocab, bf16);
#define SHERRY_RANGE(B, T, S)                                                                                             \
  do {                                                                                                                    \
    const dim3 grid((unsigned)(n * a.ranges));                                                                            \
    if (stream) hipLaunchKernelGGL((distill_range<B, T, S, true>), grid, dim3(kThreads), lds, s, a, r0);                  \
    else hipLaunchKernelGGL((distill_range<B, T, S, false>), grid, dim3(kThreads), lds, s, a, r0);                        \
  } while (0)
#define SHERRY_RANGE_T(B)                 \
  do {                                    \
    if (tail && soft1) SHERRY_RANGE(B, true, true);  \
    else if (tail) SHERRY_RANGE(B, true, false);     \
    else if (soft1) SHERRY_RANGE(B, false, true);    \
    else SHERRY_RANGE(B, false, false);              \
  } while (0)
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = std::min(step, rows - r0);
    if (bf16) SHERRY_RANGE_T(true);
    else SHERRY_RANGE_T(false);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef SHERRY_RANGE_T
#undef SHERRY_RANGE
  const int64_t wide = rows_of_launch(1);
  for (int64_t r0 = 0; r0 < rows; r0 += wide) {
    const dim3 grid((unsigned)std::min(wide, rows - r0));
    if (bf16 && teacher_bf16) hipLaunchKernelGGL((distill_finish<true, true>), grid, dim3(64), 0, s, a, r0);
    else if (bf16) hipLaunchKernelGGL((distill_finish<true, false>), grid, dim3(64), 0, s, a, r0);
    else if (teacher_bf16) hipLaunchKernelGGL((distill_finish<false, true>), grid, dim3(64), 0, s, a, r0);
    else hipLaunchKernelGGL((distill_finish<false, false>), grid, dim3(64), 0, s, a, r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_distill_backward(const DistillGrad& a, int64_t rows, bool bf16, hipStream_t s) {
  const bool soft1 = a.labels && a.inv_t != 1., stream = streams(rows, a.vocab, bf16);
  const int64_t step = rows_of_launch(a.ranges);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const dim3 grid((unsigned)(std::min(step, rows - r0) * a.ranges));
#define SHERRY_GRAD(B, S)                                                                                    \
  do {                                                                                                       \
    if (stream) hipLaunchKernelGGL((distill_grad<B, S, true>), grid, dim3(kThreads), 0, s, a, r0);           \
    else hipLaunchKernelGGL((distill_grad<B, S, false>), grid, dim3(kThreads), 0, s, a, r0);                 \
  } while (0)
    if (bf16 && soft1) SHERRY_GRAD(true, true);
    else if (bf16) SHERRY_GRAD(true, false);
    else if (soft1) SHERRY_GRAD(false, true);
    else SHERRY_GRAD(false, false);
#undef SHERRY_GRAD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sherry
