// block.cuh -- loads and stores shared by the kernels around the layer
// (block_norm.cu, lora.cu): rows with a stride, 8 values at a time, bf16 or
// fp32 in memory and fp32 in registers.
#pragma once

#include "../../include/moe_nvfp4.h"
#include "common.cuh"

namespace moe {

// Row t of a moe_rows whose contiguous row holds `cols` elements of T.
template <typename T>
__device__ __forceinline__ T* row_ptr(const moe_rows& r, int64_t t, int64_t cols) {
  return static_cast<T*>(r.data) + t * (r.stride ? r.stride : cols);
}

// Two values rounded to bf16 by one instruction.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void unpack8(const uint4& d, float (&v)[8]) {
  v[0] = bf16lo(d.x);
  v[1] = bf16hi(d.x);
  v[2] = bf16lo(d.y);
  v[3] = bf16hi(d.y);
  v[4] = bf16lo(d.z);
  v[5] = bf16hi(d.z);
  v[6] = bf16lo(d.w);
  v[7] = bf16hi(d.w);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  uint4 d;
  d.x = pack2(v[0], v[1]);
  d.y = pack2(v[2], v[3]);
  d.z = pack2(v[4], v[5]);
  d.w = pack2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = d;
}

// An fp32 value as a sum of bf16 terms, each the upper half of what is left: three hold its 24 bits.  Takes the next term
// off s; the result's upper 16 bits are it.  (Cut off, not rounded: a value above the largest bf16 would round to
// infinity.  Of an infinity nothing is left, where a subtraction gives NaN; a NaN leaves one.)
__device__ __forceinline__ uint32_t take_term(float& s) {
  const uint32_t t = __float_as_uint(s) & 0xffff0000u;
  s = (__float_as_uint(s) & 0x7fffffffu) == 0x7f800000u ? 0.f : s - __uint_as_float(t);
  return t;
}
// Of two values, as a bf16 pair.
__device__ __forceinline__ uint32_t take_terms(float& lo, float& hi) {
  const uint32_t l = take_term(lo);
  return take_term(hi) | l >> 16;
}

// Two fp32 values that one instruction works on.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float v) { return {v, v}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A block's sum over rows [b0, b1] of 32 columns (col: this lane's is there) of
// a matrix of E: warp w adds rows b0 + w, + kJoinWarps, ... in order, kBatch
// loads at a time; then lane l of warp c holds column c's sum of warp l, and a
// butterfly adds those.  join_part is the warps' own part, join_parts (after
// s[warp][lane] = that and a barrier) gives every thread of warp c column c's sum.
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
template <int kBatch, typename T>
__device__ __forceinline__ T join_part(const T* __restrict__ m, int32_t b0, int32_t b1, int32_t E, int32_t e, bool col) {
  T v = 0;
  for (int32_t b = b0 + (int32_t)(threadIdx.x >> 5); b <= b1; b += kBatch * kJoinWarps) {
    T x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int32_t r = b + i * kJoinWarps;
      x[i] = col && r <= b1 ? m[(int64_t)r * E + e] : T(0);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v += x[i];
  }
  return v;
}
template <typename T>
__device__ __forceinline__ T join_parts(const T (*s)[33]) {
  T v = s[threadIdx.x & 31][threadIdx.x >> 5];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

}  // namespace moe
