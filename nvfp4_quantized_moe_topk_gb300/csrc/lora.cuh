// lora.cuh -- what the adapter kernels share (lora.cu: few tokens, lora_rows.cu:
// many): the plan that groups tokens by adapter, matrix instructions, the
// clusters' shared memory and asynchronous copies.
#pragma once

#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kFusedTokens = 256;         // at most one token a thread
constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 16;              // tokens a thread of the sorting kernel
constexpr int kPlanSlice = kPlanThreads * kPlanPer;

// Sorted tokens and group starts; bucket n_adapters holds the tokens without
// an adapter.
struct LoraPlan {
  int32_t* order;      // [n] tokens by bucket
  int32_t* starts;     // [n_adapters + 2] first entry of each bucket in order
  int32_t* tile_base;  // [n_adapters + 2] first tile of each bucket
  int32_t* hist;       // [slices][n_adapters + 1], several slices only
};

inline int64_t up4(int64_t v) { return (v + 3) & ~int64_t(3); }
inline int32_t plan_slices(int32_t n) { return (int32_t)(((int64_t)n + kPlanSlice - 1) / kPlanSlice); }

inline LoraPlan lora_plan(void* ws, int32_t n, int32_t L) {
  LoraPlan p;
  p.order = static_cast<int32_t*>(ws);
  p.starts = p.order + up4(n);
  p.tile_base = p.starts + up4(L + 2);
  p.hist = p.tile_base + up4(L + 2);
  return p;
}

__device__ __forceinline__ int32_t bucket_of(int32_t id, int32_t L) { return id >= 0 && id < L ? id : L; }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at this CTA's shared address `p`, in CTA `rank` of the cluster.
__device__ __forceinline__ float peer_float(const float* p, uint32_t rank) {
  uint32_t addr;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// What a CTA works on.
struct Tile {
  int32_t adapter, count;
};

// Finds this CTA's tile and its tokens (row[i], -1 past the count).  Returns
// false, for the whole cluster alike, where there is none left.
template <int MT>
__device__ __forceinline__ bool find_tile(const moe_lora_args& a, const LoraPlan& p, bool fused, int32_t tile,
                                          int32_t* row, int32_t* scratch, Tile& t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, L = a.n_adapters;
  __shared__ int32_t found[3];
  if (tid == 0) found[0] = -1;
  if (tid < MT) row[tid] = -1;
  if (!fused) {
    pdl_wait();
    __syncthreads();
    for (int32_t l = tid; l <= L; l += kLoraThreads) {
      const int32_t b0 = p.tile_base[l], b1 = p.tile_base[l + 1];
      if (tile >= b0 && tile < b1) {
        const int32_t first = p.starts[l] + (tile - b0) * MT;
        found[0] = l;
        found[1] = first;
        found[2] = min(MT, p.starts[l + 1] - first);
      }
    }
    __syncthreads();
    t.adapter = found[0];
    if (t.adapter < 0) return false;
    t.count = found[2];
    if (tid < t.count) row[tid] = p.order[found[1] + tid];
    __syncthreads();
    return true;
  }
  // ids in shared memory; a token whose rank among its adapter's is a multiple
  // of MT leads a tile, tiles in the order of their leaders
  const int32_t n = a.n;
  int32_t* leaders = scratch + kFusedTokens;  // per warp
  const int32_t mine = tid < n ? bucket_of(a.adapter_ids[tid], L) : -1;
  scratch[tid] = mine;
  __syncthreads();
  int32_t rank = 0;
  const int4* ids4 = reinterpret_cast<const int4*>(scratch);
  for (int32_t i = 0; i < (tid & ~31); i += 4) {  // the warps before this one
    const int4 v = ids4[i >> 2];
    rank += (v.x == mine) + (v.y == mine) + (v.z == mine) + (v.w == mine);
  }
  rank += __popc(__match_any_sync(0xffffffffu, mine) & ((1u << lane) - 1u));
  const bool leads = mine >= 0 && rank % MT == 0;
  const uint32_t lead = __ballot_sync(0xffffffffu, leads);
  if (lane == 0) leaders[warp] = __popc(lead);
  __syncthreads();
  int32_t at = __popc(lead & ((1u << lane) - 1u));
  for (int w = 0; w < warp; ++w) at += leaders[w];
  if (leads && at == tile) {
    found[0] = mine;
    found[1] = rank / MT;
  }
  __syncthreads();
  t.adapter = found[0];
  if (t.adapter < 0) return false;
  const bool in = mine == t.adapter && rank / MT == found[1];
  if (in) row[rank % MT] = tid;
  t.count = __syncthreads_count(in);
  return true;
}

// 16 (or 8) bytes into a ring slot.
__device__ __forceinline__ void ring16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ring8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 slot16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `ahead` (0..3) of the thread's newest groups are unfinished.
__device__ __forceinline__ void ring_wait(int ahead) {
  switch (ahead) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory");
  }
}

constexpr uint32_t kSlotVec = kLoraThreads * 16;  // one 16-byte vector of every thread

// lora_rows.cu: at most `tiles` tiles of kRowsTile tokens.
constexpr int kRowsTile = 64;
cudaError_t launch_lora_rows(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, cudaStream_t s);

}  // namespace moe
