// lora.cu -- low-rank adapters of many requests at once, added to a shared
// projection's result (moe_lora_apply).
//
//   v = A[l] x (over the adapter's rank),  out = y + scale[l] B[l] v
//
// One CTA per token: its warps form the rank's dot products over x, then its
// threads the outputs from v in shared memory.
#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kLoraThreads = 256;

template <typename YT, typename OT>
__global__ void __launch_bounds__(kLoraThreads) lora_token_kernel(const moe_lora_args a) {
  __shared__ float v[128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int32_t l = a.adapter_ids[t];
  int32_t rank = 0;
  float scale = 0.f;
  if (l >= 0 && l < a.n_adapters) {
    rank = a.ranks ? min(max(a.ranks[l], 0), a.max_rank) : a.max_rank;
    scale = a.scale ? a.scale[l] : 1.f;
  }
  const uint16_t* x = row_ptr<const uint16_t>(a.x, t, a.in_features);
  for (int32_t i = warp; i < rank; i += kLoraThreads / 32) {
    const uint16_t* w = a.a + ((int64_t)l * a.max_rank + i) * a.in_features;
    float sum = 0.f;
    for (int32_t c = lane * 8; c < a.in_features; c += 256) {
      float p[8], q[8];
      load8(x + c, p);
      load8(w + c, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(p[j], q[j], sum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) v[i] = sum;
  }
  __syncthreads();
  for (int32_t o = threadIdx.x * 8; o < a.out_features; o += kLoraThreads * 8) {
    float r[8] = {};
    if (a.y.data) load8(row_ptr<const YT>(a.y, t, a.out_features) + o, r);
    if (rank > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t* w = a.b + ((int64_t)l * a.out_features + o + j) * a.max_rank;
        float sum = 0.f;
        for (int32_t i = 0; i < rank; ++i) sum = fmaf(v[i], bf16lo(w[i]), sum);
        r[j] = fmaf(scale, sum, r[j]);
      }
    }
    store8(row_ptr<OT>(a.out, t, a.out_features) + o, r);
  }
}

}  // namespace

size_t lora_workspace(int32_t n, int32_t n_adapters) {
  (void)n;
  (void)n_adapters;
  return 0;
}

cudaError_t launch_lora(const moe_lora_args& a, void* workspace, cudaStream_t s) {
  (void)workspace;
  const bool yb = a.y_dtype == MOE_DTYPE_BF16, ob = a.out_dtype == MOE_DTYPE_BF16;
  const unsigned n = (unsigned)a.n;
  if (yb && ob)
    lora_token_kernel<uint16_t, uint16_t><<<n, kLoraThreads, 0, s>>>(a);
  else if (yb)
    lora_token_kernel<uint16_t, float><<<n, kLoraThreads, 0, s>>>(a);
  else if (ob)
    lora_token_kernel<float, uint16_t><<<n, kLoraThreads, 0, s>>>(a);
  else
    lora_token_kernel<float, float><<<n, kLoraThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
