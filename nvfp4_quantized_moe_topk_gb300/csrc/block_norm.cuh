// block_norm.cuh -- what the forward and the backward pass of the norms around
// a block share (block_norm.cu, block_norm_bwd.cu): row addressing, the
// threads' own rings in shared memory, sums over a row's group of threads, and
// the shape of a persistent launch.
#pragma once

#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kNormMaxThreads = 512;
constexpr int kNormSmem = 220 * 1024;

// What a kernel knows at compile time.  kNormAny: nothing.  The others: branch,
// post_weight and pre_weight (and, backward, d_x) are there, as between two
// blocks, and the gate is none or per token, per channel, or full.
enum NormMode { kNormAny, kNormScalar, kNormChannel, kNormFull };

// Rows of a matrix, addressed in 16-byte vectors (a product of two 32-bit
// numbers instead of a 64-bit multiplication per access).
struct NormRows {
  char* p;
  int32_t stride;
  __device__ __forceinline__ char* at(int32_t t, int32_t vec) const {
    return p + (((uint64_t)(uint32_t)t * (uint32_t)stride + (uint32_t)vec) << 4);
  }
};
inline NormRows norm_rows(const moe_rows& r, int64_t cols, int64_t bytes) {
  return {static_cast<char*>(r.data), (int32_t)((r.stride ? r.stride : cols) * bytes / 16)};
}

struct NormParams {
  int32_t n, H, gate_kind, gate_sigmoid, param_dtype;
  float inv_h, eps, alpha, beta, offset;
  NormRows residual, branch, gate, residual_out, x_out;
  const void *post, *pre;
  float *rstd_post, *rstd_pre;
};
inline NormParams norm_params(const moe_block_norm_args& a) {
  const int64_t rb = a.residual_dtype == MOE_DTYPE_BF16 ? 2 : 4, yb = a.branch_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  NormParams p;
  p.n = a.n;
  p.H = a.hidden;
  p.gate_kind = a.gate_kind;
  p.gate_sigmoid = a.gate_sigmoid;
  p.param_dtype = a.param_dtype;
  p.inv_h = 1.f / (float)a.hidden;
  p.eps = a.eps;
  p.alpha = a.residual_scale;
  p.beta = a.branch_scale;
  p.offset = a.weight_offset;
  p.residual = norm_rows(a.residual, a.hidden, rb);
  p.branch = norm_rows(a.branch, a.hidden, yb);
  p.gate = norm_rows(a.gate, a.hidden, yb);
  p.residual_out = norm_rows(a.residual_out, a.hidden, rb);
  p.x_out = norm_rows(a.x_out, a.hidden, 2);
  p.post = a.post_weight;
  p.pre = a.pre_weight;
  p.rstd_post = a.rstd_post;
  p.rstd_pre = a.rstd_pre;
  return p;
}

// Threads of a row: every thread owns ITERS times 8 channels.
inline int norm_iters(int32_t hidden) { return hidden / 8 > kNormMaxThreads ? 2 : 1; }
inline int norm_threads(int32_t hidden) {
  const int it = norm_iters(hidden), vecs = hidden / 8;
  return ((vecs + it - 1) / it + 31) / 32 * 32;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

// 16-byte vectors that hold 8 values of T.
template <typename T>
struct Vec8 {
  static constexpr int kVecs = sizeof(T) / 2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `depth` (0, 1 or 3) of this thread's newest groups are unfinished.
__device__ __forceinline__ void cp_async_wait(int depth) {
  if (depth == 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (depth == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Which 8 channels of a warp's 256 a lane owns.  QUADS false (all matrices
// bf16): 8 neighbouring ones, 16 bytes.  QUADS true (some matrix is fp32): 4
// at 4 lane and 4 at 128 + 4 lane, so that an fp32 access of the warp is two
// runs of 512 contiguous bytes (8 neighbouring fp32 channels a lane would
// touch every memory sector twice) and a bf16 one two runs of 256.
template <bool QUADS>
struct Lane {
  int32_t c0;  // first channel; the second four are at c0 + kNext
  bool ok0, ok1;
  static constexpr int32_t kNext = QUADS ? 128 : 4;
  __device__ __forceinline__ Lane(int32_t i, int32_t hidden) {
    const int32_t lane = threadIdx.x & 31;
    c0 = (int32_t)(threadIdx.x - lane + i * blockDim.x) * 8 + lane * (QUADS ? 4 : 8);
    ok0 = c0 < hidden;
    ok1 = c0 + kNext < hidden;
  }
};

// The ring: for every matrix of a row, each warp's 256 channels lie contiguous
// in shared memory (fp32: in two parts, `pitch` apart); `at` is the lane's 16
// bytes there.  A lane copies 16 contiguous bytes an instruction, in order; in
// QUADS form it reads bytes that its warp copied (__syncwarp in between).
template <typename T, bool QUADS>
__device__ __forceinline__ void ring_copy(uint32_t at, uint32_t pitch, const char* row, int32_t i, int32_t hidden) {
  const int32_t lane = threadIdx.x & 31, base = (int32_t)(threadIdx.x - lane + i * blockDim.x) * 8;
  if constexpr (Vec8<T>::kVecs == 1) {
    const int32_t c = base + lane * 8;
    if (c < hidden) cp_async16(at, row + (uint32_t)c * 2u);
  } else {
    static_assert(QUADS, "fp32 rows are dealt in quads");
    const int32_t c = base + lane * 4;
    if (c < hidden) cp_async16(at, row + (uint32_t)c * 4u);
    if (c + 128 < hidden) cp_async16(at + pitch, row + (uint32_t)c * 4u + 512);
  }
}
// The lane's values from the ring (`at`: offset of its 16 bytes in the CTA's
// dynamic shared memory), 0 where it has no channel.
template <typename T, bool QUADS>
__device__ __forceinline__ void ring_read(const char* ring, uint32_t at, uint32_t pitch, const Lane<QUADS>& l,
                                          F2 (&v)[4]) {
  if constexpr (Vec8<T>::kVecs == 1 && !QUADS) {
    const uint4 d = *reinterpret_cast<const uint4*>(ring + at);
    v[0] = {bf16lo(d.x), bf16hi(d.x)};
    v[1] = {bf16lo(d.y), bf16hi(d.y)};
    v[2] = {bf16lo(d.z), bf16hi(d.z)};
    v[3] = {bf16lo(d.w), bf16hi(d.w)};
  } else if constexpr (Vec8<T>::kVecs == 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 d = *reinterpret_cast<const uint2*>(ring + at - (threadIdx.x & 31) * 8 + h * 256);
      v[2 * h] = {bf16lo(d.x), bf16hi(d.x)};
      v[2 * h + 1] = {bf16lo(d.y), bf16hi(d.y)};
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 d = *reinterpret_cast<const float4*>(ring + at + h * pitch);
      v[2 * h] = {d.x, d.y};
      v[2 * h + 1] = {d.z, d.w};
    }
  }
  if (QUADS && !l.ok1) v[2] = v[3] = f2(0.f);
}
template <typename T, bool QUADS>
__device__ __forceinline__ void row_store(const NormRows& r, int32_t t, const Lane<QUADS>& l, const F2 (&v)[4]) {
  char* row = r.at(t, 0);
  if constexpr (Vec8<T>::kVecs == 1 && !QUADS) {
    *reinterpret_cast<uint4*>(row + (uint32_t)l.c0 * 2u) =
        make_uint4(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y), pack2(v[2].x, v[2].y),
                   pack2(v[3].x, v[3].y));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && !l.ok1) break;
      const uint32_t c = (uint32_t)(l.c0 + h * Lane<QUADS>::kNext);
      if constexpr (Vec8<T>::kVecs == 1)
        *reinterpret_cast<uint2*>(row + c * 2u) =
            make_uint2(pack2(v[2 * h].x, v[2 * h].y), pack2(v[2 * h + 1].x, v[2 * h + 1].y));
      else
        *reinterpret_cast<float4*>(row + c * 4u) = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
    }
  }
}
template <bool QUADS>
__device__ __forceinline__ void load_param(const void* p, int32_t dtype, const Lane<QUADS>& l, F2 (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[2 * h] = v[2 * h + 1] = f2(0.f);
    if (h && !l.ok1) continue;
    const int32_t c = l.c0 + h * Lane<QUADS>::kNext;
    if (dtype == MOE_DTYPE_BF16) {
      const uint2 d = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c);
      v[2 * h] = {bf16lo(d.x), bf16hi(d.x)};
      v[2 * h + 1] = {bf16lo(d.y), bf16hi(d.y)};
    } else {
      const float4 d = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
      v[2 * h] = {d.x, d.y};
      v[2 * h + 1] = {d.z, d.w};
    }
  }
}
__device__ __forceinline__ void sigmoid2(F2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = {sigmoid(v[j].x), sigmoid(v[j].y)};
}

__device__ __forceinline__ float shfl_xor(float v, int lanes) { return __shfl_xor_sync(0xffffffffu, v, lanes); }

// Sum of a value over the CTA, in a fixed order, by one barrier; red is this
// reduction's own 16 floats of shared memory.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += shfl_xor(v, off);
  if (warps == 1) return v;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (lane & 15) < warps ? red[lane & 15] : 0.f;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += shfl_xor(v, off);
  return v;
}
// Of three values at once: the first two steps halve what a lane carries (the
// quarters of the warp end up with one value each), red has 64 floats.
__device__ __forceinline__ void cta_sums3(float& a, float& b, float& c, float* red) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool upper = lane & 16, odd = lane & 8;
  float x = upper ? b : a, y = upper ? 0.f : c;  // kept: (a, c) below, (b, -) above
  x += shfl_xor(upper ? a : b, 16);
  y += shfl_xor(upper ? c : 0.f, 16);
  float v = odd ? y : x;  // quarters: a, c, b, -
  v += shfl_xor(odd ? x : y, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) v += shfl_xor(v, off);
  if (warps > 1) {
    if ((lane & 7) == 0) red[(lane >> 3) * 16 + (threadIdx.x >> 5)] = v;
    __syncthreads();
    const int w = lane & 7;
    const float* mine = red + (lane >> 3) * 16;
    v = (w < warps ? mine[w] : 0.f) + (w + 8 < warps ? mine[w + 8] : 0.f);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) v += shfl_xor(v, off);
  }
  a = __shfl_sync(0xffffffffu, v, 0);
  c = __shfl_sync(0xffffffffu, v, 8);
  b = __shfl_sync(0xffffffffu, v, 16);
}

inline int norm_sms() {  // (asked for once a device)
  static std::atomic<int> held[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 1;
  sms = held[dev].load(std::memory_order_relaxed);
  if (sms) return sms;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  sms = std::max(sms, 1);
  held[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Shape of a persistent launch: CTAs of about `sm_threads` threads an SM, and
// ring stages: two where the SM's CTAs have 40 KB of rows in flight with one
// stage ahead, else four (4314 x 2688 backward, 22 KB a row: 32.4 us with two,
// 34.3 with four); one where two do not fit.
struct NormPlan {
  int threads, stages, smem, ctas;
};
constexpr int kNormMaxPerSm = 24;
inline NormPlan norm_plan(int32_t n, int32_t hidden, int stage_vecs, int sm_threads) {
  NormPlan p;
  p.threads = norm_threads(hidden);
  const int stage = stage_vecs * p.threads * 16;
  int per_sm = std::max(1, std::min(sm_threads / p.threads, kNormMaxPerSm));
  p.stages = 2 * stage > kNormSmem ? 1 : per_sm * stage >= 40 * 1024 ? 2 : 4;
  p.smem = p.stages * stage;
  per_sm = std::max(1, std::min(per_sm, kNormSmem / (p.smem + 1024)));
  p.ctas = (int)std::min<int64_t>(n, (int64_t)norm_sms() * per_sm);
  return p;
}

}  // namespace moe
