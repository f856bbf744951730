// layer.cu -- the router of the whole-layer call: logits and picks in one launch.
//
// For a few tokens the router is all latency: its weights (0.7 MB for 128
// experts of 2688) take 0.1 us to read.  A block takes 16 experts, each of its 32
// warps two or three steps of 32 columns, whose loads are all in flight at once;
// warp-level matrix instructions take 16 experts by 8 tokens, and the warps' sums
// meet in shared memory, in order.  An fp32 weight goes in as three bf16 terms,
// which keep its 24 bits, as products with bf16 x are exact.  Of up to 8 tokens the
// kernel that follows picks the experts itself (layer_few.cu).  Otherwise the block that
// finishes last routes the tokens, a warp a token, from the logits that the others
// left in L2, adds the shared experts to the picks, and cuts experts of more than 8
// tokens into parts, as one such expert
// would keep the streaming kernel (decode.cu) from staging and have its warps pass
// over their tiles again and again (a decode batch of 32, gated, two shared
// experts, an expert of 10 tokens: 461 us with the shared ones cut alone, 200 so).
#include <algorithm>

#include "block.cuh"
#include "kernels.h"
#include "layer_pick.cuh"
#include "tile.cuh"

namespace moe {

namespace {

constexpr int kLayerThreads = 1024, kLayerWarps = kLayerThreads / 32, kLayerExperts = 16;

// After the picks, by one block: an expert's tokens beyond each 8 move to a further part of it.  Parts are dealt in the
// order of shared experts, then experts, and tokens in their order, so that the layer's bits do not depend on timing.
struct PartSpace {
  int32_t id[kDecMaxPairs], count[1024], base[1024];
};
__device__ void deal_parts(const LayerRouterArgs& a, PartSpace& sp) {
  const int32_t pairs = a.n * a.k, slots = a.k + a.shared, more = (a.n + kDecPassTok - 1) / kDecPassTok - 1;
  for (int32_t e = threadIdx.x; e < a.E; e += kLayerThreads) sp.count[e] = 0;
  for (int32_t i = threadIdx.x; i < a.shared * more; i += kLayerThreads) a.part_of[i] = a.E + i / more;
  __syncthreads();
  bool any = false;
  for (int32_t p = threadIdx.x; p < pairs; p += kLayerThreads) {
    const int32_t e = a.ids[p / a.k * slots + p % a.k];
    sp.id[p] = e;
    any |= atomicAdd(&sp.count[e], 1) >= kDecPassTok;
  }
  if (!__syncthreads_or(any)) return;
  if (threadIdx.x < 32) {
    int32_t run = a.shared * more;
    for (int32_t e0 = 0; e0 < a.E; e0 += 32) {
      const int32_t e = e0 + (int32_t)threadIdx.x, own = e < a.E && sp.count[e] > 0 ? (sp.count[e] - 1) / kDecPassTok : 0;
      int32_t sum = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, sum, d);
        if ((int)threadIdx.x >= d) sum += v;
      }
      if (e < a.E) sp.base[e] = run + sum - own;
      for (int32_t i = 0; i < own; ++i) a.part_of[run + sum - own + i] = e;
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  for (int32_t p = threadIdx.x; p < pairs; p += kLayerThreads) {
    const int32_t e = sp.id[p];
    if (sp.count[e] <= kDecPassTok) continue;
    int32_t rank = 0;
    for (int32_t q = 0; q < p; ++q) rank += sp.id[q] == e;
    if (rank >= kDecPassTok)
      a.ids[p / a.k * slots + p % a.k] = a.E + a.shared + sp.base[e] + rank / kDecPassTok - 1;
  }
}

// Eight consecutive values of a weight row as bf16 terms whose sum they are.
template <typename T>
struct RouterTerms {
  static constexpr int kTerms = sizeof(T) == 2 ? 1 : 3;
  uint4 v[kTerms];
};
__device__ __forceinline__ RouterTerms<uint16_t> router_terms(const uint16_t* p) {
  return {{__ldg(reinterpret_cast<const uint4*>(p))}};
}
__device__ __forceinline__ RouterTerms<float> router_terms(const float* p) {
  const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
  float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  RouterTerms<float> r;
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
  // None of them rounds to infinity: by rounding, which takes fewer instructions than cutting off (32 tokens: 20.7 us, 22.4).
  if (most < 0x1.ffp127f) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] = pack2(v[2 * i], v[2 * i + 1]);
        v[2 * i] -= bf16lo(d[i]);
        v[2 * i + 1] -= bf16hi(d[i]);
      }
      r.v[k] = make_uint4(d[0], d[1], d[2], d[3]);
    }
    return r;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = take_terms(v[2 * i], v[2 * i + 1]);
    r.v[k] = make_uint4(d[0], d[1], d[2], d[3]);
  }
  return r;
}

// TILES: tiles of 8 tokens that a pass over the weights serves.  Up to 64 tokens a block takes 8 of them, and a bf16
// weight's steps are all in flight at once (32 tokens, 128 experts in fp32: 20.7 us by events, most of it the last block's
// work; a block for all of them 29).  More read the weights once for 64.
constexpr int32_t block_tokens(int tiles) { return tiles == 1 ? 8 : 64; }
template <typename T, int TILES>
__global__ void __launch_bounds__(kLayerThreads) layer_router_kernel(const __grid_constant__ LayerRouterArgs a, int32_t pick) {
  extern __shared__ __align__(16) float dyn[];  // [warps][8 TILES][17], then the last block's work
  __shared__ int32_t last;
  constexpr int kGroup = 8 * TILES, kAhead = TILES == 1 && sizeof(T) == 2 ? 3 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int32_t e0 = blockIdx.x * kLayerExperts, steps = (a.H + 31) / 32;
  const int32_t s0 = steps * warp / kLayerWarps, s1 = steps * (warp + 1) / kLayerWarps;
  const T* ra = static_cast<const T*>(a.weight) + (int64_t)min(e0 + g, a.E - 1) * a.H + 8 * t;
  const T* rb = static_cast<const T*>(a.weight) + (int64_t)min(e0 + g + 8, a.E - 1) * a.H + 8 * t;
  pdl_wait();
  pdl_launch_dependents();
  if (a.few && blockIdx.x == 0) {  // (one group of tokens)
    if (threadIdx.x == 0) a.few->ticket = 0;
    if (threadIdx.x < kFewPairs) a.few->done[threadIdx.x] = 0;
  }
  constexpr int32_t kTokens = block_tokens(TILES);
  const int32_t end = min(a.n, ((int32_t)blockIdx.y + 1) * kTokens);
  for (int32_t t0 = blockIdx.y * kTokens; t0 < end; t0 += kGroup) {
    const int32_t tokens = min(kGroup, end - t0);
    float acc[TILES][4] = {};
    for (int32_t s = s0; s < s1; s += kAhead) {  // (a step is whole: H is a multiple of 64)
      RouterTerms<T> wa[kAhead], wb[kAhead];
      uint4 x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s + i >= s1) break;
        wa[i] = router_terms(ra + 32 * (s + i));
        wb[i] = router_terms(rb + 32 * (s + i));
        if (TILES == 1) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (g < tokens) x[i] = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + g) * a.H + 32 * (s + i) + 8 * t));
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (s + i >= s1) break;
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          if (8 * j >= tokens) break;
          if (TILES > 1) {
            x[i] = make_uint4(0, 0, 0, 0);
            if (8 * j + g < tokens)
              x[i] = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + 8 * j + g) * a.H + 32 * (s + i) + 8 * t));
          }
#pragma unroll
          for (int k = 0; k < RouterTerms<T>::kTerms; ++k) {
            mma_bf16_16816(acc[j], wa[i].v[k].x, wb[i].v[k].x, wa[i].v[k].y, wb[i].v[k].y, x[i].x, x[i].y);
            mma_bf16_16816(acc[j], wa[i].v[k].z, wb[i].v[k].z, wa[i].v[k].w, wb[i].v[k].w, x[i].z, x[i].w);
          }
        }
      }
    }
    float(*sums)[kGroup][17] = reinterpret_cast<float(*)[kGroup][17]>(dyn);
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      if (8 * j >= tokens) break;
      sums[warp][8 * j + 2 * t][g] = acc[j][0];
      sums[warp][8 * j + 2 * t + 1][g] = acc[j][1];
      sums[warp][8 * j + 2 * t][g + 8] = acc[j][2];
      sums[warp][8 * j + 2 * t + 1][g + 8] = acc[j][3];
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < tokens * kLayerExperts; i += kLayerThreads) {
      const int32_t e = e0 + i % kLayerExperts;
      if (e >= a.E) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kLayerWarps; ++w) v += sums[w][i / kLayerExperts][i % kLayerExperts];
      a.logits_out[(int64_t)(t0 + i / kLayerExperts) * a.E + e] = v;
    }
    __syncthreads();
  }
  if (!pick) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(a.count, 1) == (int32_t)(gridDim.x * gridDim.y) - 1;
    if (last) *a.count = 0;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  const int32_t slots = a.k + a.shared;
  for (int32_t k = warp; k < a.n; k += kLayerWarps)
    pick_any(a, k, lane, a.ids + (int64_t)k * slots, a.w + (int64_t)k * slots, true);
  __syncthreads();
  if (a.part_of && a.n > kDecPassTok) deal_parts(a, *reinterpret_cast<PartSpace*>(dyn));
}

__global__ void __launch_bounds__(256) layer_pick_kernel(const LayerRouterArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < a.n) pick_any(a, (int32_t)t, threadIdx.x & 31, a.ids + t * (a.k + a.shared), a.w + t * (a.k + a.shared), true);
}

}  // namespace

namespace {

template <typename T, int TILES>
cudaError_t router_launch(const LayerRouterArgs& a, bool pick, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  constexpr size_t smem = std::max({(size_t)kLayerWarps * 8 * TILES * 17 * sizeof(float), sizeof(PartSpace)});
  const cudaError_t e = raise_smem_limit(layer_router_kernel<T, TILES>, (int)smem, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.E + kLayerExperts - 1) / kLayerExperts),
                  (unsigned)((a.n + block_tokens(TILES) - 1) / block_tokens(TILES)));
  return launch_ex(layer_router_kernel<T, TILES>, grid, dim3(kLayerThreads), smem, s, true, a, (int32_t)pick);
}

}  // namespace

cudaError_t launch_layer_router(const LayerRouterArgs& a, bool have_logits, cudaStream_t s) {
  if (!have_logits) {
    const bool pick = a.n <= kLayerFusedTokens && !a.few;
    const bool few = a.n <= kLayerFusedTokens;
    const cudaError_t e =
        a.weight_f32 ? (few ? router_launch<float, 1>(a, pick, s) : router_launch<float, 4>(a, pick, s))
                     : (few ? router_launch<uint16_t, 1>(a, pick, s) : router_launch<uint16_t, 4>(a, pick, s));
    if (e != cudaSuccess || pick || a.few) return e;
  }
  layer_pick_kernel<<<(unsigned)((a.n + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
