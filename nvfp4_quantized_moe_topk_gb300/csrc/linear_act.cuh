// linear_act.cuh -- the activations of the matrix product's epilogue and their slopes.
#pragma once

#include "../../include/moe_nvfp4.h"
#include "common.cuh"

namespace moe {

// z / (1 + exp(-v)), by the exponential of -|v|, which neither overflows nor leaves the fast quotient's range (it is 0 for a
// divisor above 2^126).  The fast exponential and quotient are within (5 + 1.2 |v|) 2^-23 of the value, and within 2^-149
// |z| where that exponential is subnormal.
__device__ __forceinline__ float logistic(float v, float z = 1.f) {
  const float e = __expf(-fabsf(v));
  return __fdividef(v >= 0.f ? z : z * e, 1.f + e);
}

// gelu_tanh: z / 2 (1 + tanh(u)) = z logistic(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3).
constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float linear_act(float z, int32_t act) {
  switch (act) {
    case MOE_LINEAR_RELU2: {
      const float r = z > 0.f ? z : z == z ? 0.f : z;
      return r * r;
    }
    case MOE_LINEAR_SILU: return logistic(z, z);
    case MOE_LINEAR_GELU_TANH: return logistic(kGelu * z * fmaf(kGeluCube * z, z, 1.f), z);
    default: return z;
  }
}
__device__ __forceinline__ float linear_slope(float z, int32_t act) {
  switch (act) {
    case MOE_LINEAR_RELU2: return z > 0.f ? 2.f * z : z == z ? 0.f : z;
    case MOE_LINEAR_SILU: {
      const float p = logistic(z);
      return p * fmaf(z, 1.f - p, 1.f);
    }
    case MOE_LINEAR_GELU_TANH: {
      const float p = logistic(kGelu * z * fmaf(kGeluCube * z, z, 1.f));
      z = fminf(fmaxf(z, -1e4f), 1e4f);  // (1 - p or p is 0 long before; the square does not overflow)
      return fmaf(z * p * (1.f - p), kGelu * fmaf(3.f * kGeluCube * z, z, 1.f), p);
    }
    default: return 1.f;
  }
}

__device__ __forceinline__ float linear_read(const void* p, int64_t at, int32_t f32) {
  return f32 ? static_cast<const float*>(p)[at] : bf16lo(static_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void linear_write(void* p, int64_t at, int32_t f32, float v) {
  if (f32)
    static_cast<float*>(p)[at] = v;
  else
    static_cast<uint16_t*>(p)[at] = f2bf_rn(v);
}

}  // namespace moe
