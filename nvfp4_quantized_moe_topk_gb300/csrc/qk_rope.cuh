// qk_rope.cuh -- what the forward and the backward pass of the queries' and
// keys' norms with rotation share.
//
// A head vector of D elements is cut into units of 16, two vectors of 8: where
// it is rotated, unit u holds pairs 8u .. 8u + 7, (vectors u and u + rot / 16
// where a pair's members are half the rotated part apart, 2u and 2u + 1 where
// they are side by side), so that no pair is split over lanes; past the rotated
// part it holds vectors 2u and 2u + 1.  A lane takes one unit, GROUP lanes (a
// power of two) a head.
//
// Angles: pair i of a token at position p turns by p * inv_freq[i].  In fp32 that
// product is off by 2^-24 of itself, a whole turn's tenth for positions in the
// millions; instead each frequency becomes a 64-bit fixed-point part of a turn
// (rounded once from fp64), whose product with the position wraps at whole
// turns by itself.  That is within 2^-54 turns (times inv_freq where it is above
// 1) times the position of the exact one, 2^-34 turns a million tokens in, and is
// rounded to fp32's 24 bits once, as a part of half a turn: a small angle keeps
// them all.
#pragma once

#include "block.cuh"
#include "kernels.h"

namespace moe {

constexpr int kQkThreads = 128, kQkWarps = kQkThreads / 32;
constexpr int kQkMaxPairs = kQkMaxDim / 2;

struct QkSide {  // the queries or the keys
  moe_rows in, out;       // (backward: the forward's input; its gradient)
  moe_rows grad;          // backward: gradient of the forward's output
  const void* weight;     // [D] or NULL: no norm
  int32_t heads;
};
struct QkParams {
  int32_t n, D, rot, axes, pairs_interleaved, sections_interleaved, param_dtype;
  int32_t sections[MOE_MAX_AXES];
  float eps, offset, scale, inv_D;
  const int32_t* positions;  // [axes][n]
  const float* inv_freq;     // [rot / 2]
  QkSide side[2];
};

// Which axis turns pair i.
__device__ __forceinline__ int32_t axis_of_pair(const QkParams& a, int32_t i) {
  int32_t axis = 0;
  if (a.sections_interleaved) {
    const int32_t turn = i % a.axes;
    if (i / a.axes < a.sections[turn]) axis = turn;
  } else {
    for (int32_t end = a.sections[0]; axis + 1 < a.axes && i >= end; end += a.sections[axis]) ++axis;
  }
  return axis;
}

// A pair's step in turns, as 64-bit fixed point, and its axis.
struct QkTable {
  uint64_t step[kQkMaxPairs];
  int32_t axis[kQkMaxPairs];
};
__device__ __forceinline__ void fill_table(const QkParams& a, QkTable& t) {
  for (int32_t i = threadIdx.x; i < a.rot / 2; i += blockDim.x) {
    double turns = (double)a.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
    turns -= floor(turns);
    t.step[i] = __double2ull_rn(turns * 18446744073709551616.0);
    t.axis[i] = axis_of_pair(a, i);
  }
}
// offset + weight of both sides (1 without a norm), by the CTA's threads.
__device__ __forceinline__ void fill_weights(const QkParams& a, float (&w)[2][kQkMaxDim]) {
  for (int32_t i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
    const int32_t which = i >= a.D, e = i - which * a.D;
    const void* from = a.side[which].weight;
    w[which][e] = !from ? 1.f
                        : a.offset + (a.param_dtype == MOE_DTYPE_BF16 ? bf16lo(static_cast<const uint16_t*>(from)[e])
                                                                      : static_cast<const float*>(from)[e]);
  }
}
// cos and sin of a token's pairs, times the rotation's scale, by one warp for itself: [pairs] cosines, [pairs] sines.
struct QkTurns {
  float c[kQkMaxPairs], s[kQkMaxPairs];
};
__device__ __forceinline__ void fill_turns(const QkParams& a, const QkTable& t, int32_t token, int lane, QkTurns& o) {
  __syncwarp();
  for (int32_t i = lane; i < a.rot / 2; i += 32) {
    const int64_t p = __ldg(a.positions + (int64_t)t.axis[i] * a.n + token);
    // the part of a turn, signed: half turns in [-1, 1]
    const float half_turns = __ll2float_rn((int64_t)((uint64_t)p * t.step[i])) * 0x1p-63f;
    float c, s;
    sincospif(half_turns, &s, &c);
    o.c[i] = c * a.scale;
    o.s[i] = s * a.scale;
  }
  __syncwarp();
}
// A lane's 16 elements: two vectors of 8 at element offsets at[0], at[1] (< 0: not there).
struct QkUnit {
  int32_t at[2];
  bool rotated;
};
template <bool INTERLEAVED>
__device__ __forceinline__ QkUnit unit_of(int32_t u, int32_t D, int32_t rot) {
  QkUnit r;
  r.rotated = 16 * u < rot;
  const bool apart = !INTERLEAVED && r.rotated;
  r.at[0] = apart ? 8 * u : 16 * u;
  r.at[1] = apart ? rot / 2 + 8 * u : 16 * u + 8;
  if (r.at[0] >= D) r.at[0] = -1;
  if (r.at[1] >= D) r.at[1] = -1;
  return r;
}

// A lane's unit as it lies in memory, and its way through a ring in shared memory by asynchronous copies: every lane reads
// what it has copied itself, so the ring needs no barrier.
template <typename T>
struct QkRaw {
  uint4 v[2][sizeof(T) / 2];
};
template <typename T>
constexpr uint32_t kQkSlot = 32 * sizeof(QkRaw<T>);  // bytes of a warp's slot
template <typename T>
__device__ __forceinline__ void qk_fetch(uint32_t slot, int lane, const T* head, const QkUnit& u, bool live) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < (int)sizeof(T) / 2; ++q)
      if (live && u.at[h] >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + ((h * (uint32_t)sizeof(T) / 2 + q) * 32 + lane) * 16),
                     "l"(reinterpret_cast<const uint4*>(head + u.at[h]) + q)
                     : "memory");
}
template <typename T>
__device__ __forceinline__ QkRaw<T> qk_slot(uint32_t slot, int lane, const QkUnit& u, bool live) {
  QkRaw<T> r;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
      uint4& v = r.v[h][q];
      v = make_uint4(0, 0, 0, 0);
      if (live && u.at[h] >= 0)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(slot + ((h * (uint32_t)sizeof(T) / 2 + q) * 32 + lane) * 16)
                     : "memory");
    }
  return r;
}
// The lane's 16 values as pairs of neighbours: vector m's are [4 m] to [4 m + 3].
struct QkVals {
  F2 v[8];
};
__device__ __forceinline__ QkVals qk_values(const QkRaw<uint16_t>& r) {
  QkVals o;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint4& d = r.v[m][0];
    o.v[4 * m] = {bf16lo(d.x), bf16hi(d.x)};
    o.v[4 * m + 1] = {bf16lo(d.y), bf16hi(d.y)};
    o.v[4 * m + 2] = {bf16lo(d.z), bf16hi(d.z)};
    o.v[4 * m + 3] = {bf16lo(d.w), bf16hi(d.w)};
  }
  return o;
}
__device__ __forceinline__ QkVals qk_values(const QkRaw<float>& r) {
  QkVals o;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4& d = r.v[m][q];
      o.v[4 * m + 2 * q] = {__uint_as_float(d.x), __uint_as_float(d.y)};
      o.v[4 * m + 2 * q + 1] = {__uint_as_float(d.z), __uint_as_float(d.w)};
    }
  return o;
}
// The unit's values of an array of floats by element (0 where it has none).
__device__ __forceinline__ QkVals qk_floats(const float* p, const QkUnit& u) {
  QkVals o;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
      if (u.at[m] >= 0) d = *reinterpret_cast<const float4*>(p + u.at[m] + 4 * q);
      o.v[4 * m + 2 * q] = {d.x, d.y};
      o.v[4 * m + 2 * q + 1] = {d.z, d.w};
    }
  return o;
}
__device__ __forceinline__ void qk_store(uint16_t* head, const QkUnit& u, const QkVals& o) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
    if (u.at[m] >= 0) {
      uint4 d;
      d.x = pack2(o.v[4 * m].x, o.v[4 * m].y);
      d.y = pack2(o.v[4 * m + 1].x, o.v[4 * m + 1].y);
      d.z = pack2(o.v[4 * m + 2].x, o.v[4 * m + 2].y);
      d.w = pack2(o.v[4 * m + 3].x, o.v[4 * m + 3].y);
      *reinterpret_cast<uint4*>(head + u.at[m]) = d;
    }
}
__device__ __forceinline__ void qk_store(float* head, const QkUnit& u, const QkVals& o) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
    if (u.at[m] >= 0)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4*>(head + u.at[m] + 4 * q) =
            make_float4(o.v[4 * m + 2 * q].x, o.v[4 * m + 2 * q].y, o.v[4 * m + 2 * q + 1].x, o.v[4 * m + 2 * q + 1].y);
}
// A turn of the lane's pairs as out = v * own + partner * other: the partner of a value is the other member of its pair.
struct QkTurn {
  QkVals own, other;
};
// The other members: of the other vector, or of the same pair of neighbours.
template <bool INTERLEAVED>
__device__ __forceinline__ F2 partner(const QkVals& v, int i) {
  return INTERLEAVED ? F2{v.v[i].y, v.v[i].x} : v.v[(i + 4) % 8];
}
// cos and -sin (first members), cos and sin (second) of the unit's pairs; 1 and 0 past the rotated part.
template <bool INTERLEAVED>
__device__ __forceinline__ QkTurn turn_of(const QkTurns& t, const QkUnit& u, int unit) {
  QkTurn r;
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // pairs 8 unit + 4 q ..
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (u.rotated) {
      c = *reinterpret_cast<const float4*>(t.c + 8 * unit + 4 * q);
      s = *reinterpret_cast<const float4*>(t.s + 8 * unit + 4 * q);
    }
    if (INTERLEAVED) {
      r.own.v[4 * q] = f2(c.x);
      r.own.v[4 * q + 1] = f2(c.y);
      r.own.v[4 * q + 2] = f2(c.z);
      r.own.v[4 * q + 3] = f2(c.w);
      r.other.v[4 * q] = {-s.x, s.x};
      r.other.v[4 * q + 1] = {-s.y, s.y};
      r.other.v[4 * q + 2] = {-s.z, s.z};
      r.other.v[4 * q + 3] = {-s.w, s.w};
    } else {
      r.own.v[2 * q] = r.own.v[4 + 2 * q] = {c.x, c.y};
      r.own.v[2 * q + 1] = r.own.v[4 + 2 * q + 1] = {c.z, c.w};
      r.other.v[2 * q] = {-s.x, -s.y};
      r.other.v[2 * q + 1] = {-s.z, -s.w};
      r.other.v[4 + 2 * q] = {s.x, s.y};
      r.other.v[4 + 2 * q + 1] = {s.z, s.w};
    }
  }
  return r;
}
template <int GROUP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = GROUP / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

}  // namespace moe
