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
constexpr int kNormMaxGroups = 8;  // rows side by side in a CTA
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

// Threads of a row: every thread owns ITERS groups of 8 channels.
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

// A thread's 8 values of type T in its ring: vectors `pitch` bytes apart.
template <typename T>
__device__ __forceinline__ void ring_copy(uint32_t dst, uint32_t pitch, const char* src) {
#pragma unroll
  for (int i = 0; i < Vec8<T>::kVecs; ++i) cp_async16(dst + i * pitch, src + 16 * i);
}
template <typename T>
__device__ __forceinline__ void ring_read(uint32_t at, uint32_t pitch, float (&v)[8]) {
  uint4 d[Vec8<T>::kVecs];
#pragma unroll
  for (int i = 0; i < Vec8<T>::kVecs; ++i)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[i].x), "=r"(d[i].y), "=r"(d[i].z), "=r"(d[i].w)
                 : "r"(at + i * pitch)
                 : "memory");
  if constexpr (Vec8<T>::kVecs == 1) {
    unpack8(d[0], v);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(d[i].x);
      v[4 * i + 1] = __uint_as_float(d[i].y);
      v[4 * i + 2] = __uint_as_float(d[i].z);
      v[4 * i + 3] = __uint_as_float(d[i].w);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sums of N values over a group of blockDim.x threads (threadIdx.y: which), in
// a fixed order, by one barrier; red is this reduction's own [N][warps] floats
// of shared memory.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * warps + warp] = v[i];
  }
  if (blockDim.y == 1)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? red[i * warps + lane] : 0.f);
}

inline int norm_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

// Shape of a persistent launch: threads x groups a CTA, ring stages (4, or 2
// where two CTAs of 4 stages do not fit an SM, or 1 where two do not), CTAs of
// about `sm_threads` threads an SM.
struct NormPlan {
  dim3 block;
  int stages, smem, ctas;
};
inline NormPlan norm_plan(int32_t n, int32_t hidden, int stage_vecs, int sm_threads) {
  NormPlan p;
  const int threads = norm_threads(hidden);
  const int groups = std::max(1, std::min(kNormMaxGroups, 256 / threads));
  p.block = dim3(threads, groups);
  const int stage = stage_vecs * threads * groups * 16;
  p.stages = 2 * 4 * stage <= kNormSmem ? 4 : 2 * stage <= kNormSmem ? 2 : 1;
  p.smem = p.stages * stage;
  const int per_sm = std::max(1, std::min({sm_threads / (threads * groups), kNormSmem / p.smem, 8}));
  p.ctas = (int)std::min<int64_t>(((int64_t)n + groups - 1) / groups, (int64_t)norm_sms() * per_sm);
  return p;
}

}  // namespace moe
