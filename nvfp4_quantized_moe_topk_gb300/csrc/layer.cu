// layer.cu -- the router of the whole-layer call: logits and picks in one launch.
//
// For a few tokens the router is all latency: its weights (0.7 MB for 128
// experts of 2688) take 0.1 us to read.  A block takes four experts, four warps
// each; a warp holds its part of an expert's row in registers and goes over the
// tokens.  The block that finishes last routes the tokens, a warp a token, from
// the logits the others left in L2, and adds the shared experts to the picks, so
// that the streaming kernel that follows serves them beside the routed ones; an
// expert of more than 8 tokens it cuts into parts (a decode batch of 32, gated,
// two shared experts, an expert of 10 tokens: 461 us with the shared ones cut alone, 200 so).
#include <algorithm>

#include "block.cuh"
#include "kernels.h"
#include "router.cuh"

namespace moe {

namespace {

constexpr int kLayerThreads = 512, kLayerWarps = kLayerThreads / 32;
constexpr int kSplit = 4, kLayerExperts = kLayerWarps / kSplit;  // warps an expert, experts a block
constexpr int kMaxVecs = 4;  // 16-byte vectors of a row a lane holds at once: 32 lanes x 4 warps x 4 x 8 values = 4096

// One token's picks: k of the logits, then the shared experts.
template <int SLOTS>
__device__ __forceinline__ void pick_token(const LayerRouterArgs& a, int32_t t, int lane) {
  float z[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int32_t e = lane + 32 * i;
    z[i] = 0.f;
    if (e < a.E) z[i] = __ldcg(a.logits + (int64_t)t * a.E + e) + (a.bias ? __ldg(a.bias + e) : 0.f);
  }
  const int32_t slots = a.k + a.shared;
  int32_t* ids = a.ids + (int64_t)t * slots;
  float* w = a.w + (int64_t)t * slots;
  route_token<SLOTS>(z, a.E, a.k, lane, ids, w, nullptr);
  __syncwarp();
  if (lane < a.k) {
    if (a.ids_out) a.ids_out[(int64_t)t * a.k + lane] = ids[lane];
    if (a.w_out) a.w_out[(int64_t)t * a.k + lane] = w[lane];
  }
  if (lane < a.shared) {
    const int32_t part = a.part_of ? t / kDecPassTok : 0, more = (a.n + kDecPassTok - 1) / kDecPassTok - 1;
    ids[a.k + lane] = part == 0 ? a.E + lane : a.E + a.shared + lane * more + part - 1;
    w[a.k + lane] = 1.f;
  }
}
__device__ __forceinline__ void pick_any(const LayerRouterArgs& a, int32_t t, int lane) {
  if (a.E <= 64)
    pick_token<2>(a, t, lane);
  else if (a.E <= 128)
    pick_token<4>(a, t, lane);
  else if (a.E <= 256)
    pick_token<8>(a, t, lane);
  else if (a.E <= 512)
    pick_token<16>(a, t, lane);
  else
    pick_token<32>(a, t, lane);
}

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

template <typename T>
__global__ void __launch_bounds__(kLayerThreads) layer_router_kernel(const LayerRouterArgs a, int32_t pick) {
  __shared__ union {
    float sums[kLayerWarps][kLayerFusedTokens];
    PartSpace parts;
  } sm;
  __shared__ int32_t last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp % kSplit;
  const int32_t e = blockIdx.x * kLayerExperts + warp / kSplit, vecs = a.H / 8;
  const int32_t t0 = blockIdx.y * kLayerFusedTokens, tokens = min(kLayerFusedTokens, a.n - t0);
  const T* row = static_cast<const T*>(a.weight) + (int64_t)min(e, a.E - 1) * a.H;
  float w[kMaxVecs][8];
#pragma unroll
  for (int i = 0; i < kMaxVecs; ++i) {
    const int32_t v = (i * kSplit + slice) * 32 + lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 0.f;
    if (v < vecs) {
      if (sizeof(T) == 2) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(row) + v), w[i]);
      } else {
        const float4 lo = __ldg(reinterpret_cast<const float4*>(row) + 2 * v), hi = __ldg(reinterpret_cast<const float4*>(row) + 2 * v + 1);
        w[i][0] = lo.x;
        w[i][1] = lo.y;
        w[i][2] = lo.z;
        w[i][3] = lo.w;
        w[i][4] = hi.x;
        w[i][5] = hi.y;
        w[i][6] = hi.z;
        w[i][7] = hi.w;
      }
    }
  }
  for (int32_t t = 0; t < tokens; ++t) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * a.H);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxVecs; ++i) {
      const int32_t v = (i * kSplit + slice) * 32 + lane;
      if (v < vecs) {
        float xv[8];
        unpack8(__ldg(x + v), xv);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(xv[j], w[i][j], sum);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) sm.sums[warp][t] = sum;
  }
  __syncthreads();
  for (int32_t i = threadIdx.x; i < tokens * kLayerExperts; i += kLayerThreads) {
    const int32_t t = i / kLayerExperts, q = i % kLayerExperts, to = blockIdx.x * kLayerExperts + q;
    if (to >= a.E) continue;
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kSplit; ++s) v += sm.sums[q * kSplit + s][t];
    a.logits[(int64_t)(t0 + t) * a.E + to] = v;
  }
  if (!pick) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(a.count, 1) == (int32_t)gridDim.x - 1;
    if (last) *a.count = 0;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  for (int32_t t = warp; t < a.n; t += kLayerWarps) pick_any(a, t, lane);
  if (!a.part_of || a.n <= kDecPassTok) return;
  __syncthreads();
  deal_parts(a, sm.parts);
}

__global__ void __launch_bounds__(256) layer_pick_kernel(const LayerRouterArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < a.n) pick_any(a, (int32_t)t, threadIdx.x & 31);
}

}  // namespace

cudaError_t launch_layer_router(const LayerRouterArgs& a, bool have_logits, cudaStream_t s) {
  if (!have_logits) {
    const int32_t pick = a.n <= kLayerFusedTokens;
    const dim3 grid((unsigned)((a.E + kLayerExperts - 1) / kLayerExperts), (unsigned)((a.n + kLayerFusedTokens - 1) / kLayerFusedTokens));
    if (a.weight_f32)
      layer_router_kernel<float><<<grid, kLayerThreads, 0, s>>>(a, pick);
    else
      layer_router_kernel<uint16_t><<<grid, kLayerThreads, 0, s>>>(a, pick);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || pick) return e;
  }
  layer_pick_kernel<<<(unsigned)((a.n + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
