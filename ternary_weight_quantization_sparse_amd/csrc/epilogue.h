// What follows a packed product before its one rounding: bias, activation (or
// an activated gate times the other half's values) and a scaled residual.
#pragma once

#include <cmath>

#include "ops_internal.h"

namespace sherry {

__device__ inline float activate(float z, int kind) {
  switch (kind) {
    case SHERRY_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case SHERRY_ACT_RELU2: return z > 0.f ? z * z : (z != z ? z : 0.f);
    case SHERRY_ACT_SILU: return z / (1.f + expf(-z));
    case SHERRY_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case SHERRY_ACT_GELU_TANH: {
      // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2 u))
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      return z / (1.f + expf(-2.f * u));
    }
    default: return z;
  }
}

__device__ inline float load_float(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

}  // namespace sherry
