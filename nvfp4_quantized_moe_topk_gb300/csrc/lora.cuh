// lora.cuh -- what the adapter kernels share (lora.cu: few tokens; lora_mma.cu
// and lora_rows.cu: many): the ways to group tokens by adapter, matrix
// instructions, the clusters' shared memory and asynchronous copies.
#pragma once

#include <algorithm>

#include "block.cuh"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 16;              // tokens a thread of the sorting kernel
constexpr int kPlanSlice = kPlanThreads * kPlanPer;

// v goes into the second product as a sum of this many bf16 terms, each the upper half of what is left: all 24 bits of
// its fp32 value, for a bf16 out too (where y cancels most of B v, the 16 bits of two terms show there as well).  Two
// against three, us on a GB300: 16384 tokens, 4096 to 2048, ranks to 64 74.5 / 76.1; 4096 to 4096, rank 128 121 / 130;
// 32 tokens no difference.
constexpr int kLoraTerms = 3;
// Takes the next term off s; the result's upper 16 bits are it.  (Cut off, not rounded: a v above the largest bf16
// would round to infinity.  Of an infinity nothing is left, where a subtraction gives NaN; a NaN has bits in its upper
// half, as every result of arithmetic has.)
__device__ __forceinline__ uint32_t take_term(float& s) {
  const uint32_t t = __float_as_uint(s) & 0xffff0000u;
  s = (t & 0x7fffffffu) == 0x7f800000u ? 0.f : s - __uint_as_float(t);
  return t;
}
// Of two values, as a bf16 pair.
__device__ __forceinline__ uint32_t take_terms(float& lo, float& hi) {
  const uint32_t l = take_term(lo);
  return take_term(hi) | l >> 16;
}

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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores M (1, 2 or 4) floats at this CTA's shared address `p`, in CTA `rank` of
// the cluster, and counts their bytes on that CTA's mbarrier `bar`.
template <int M>
__device__ __forceinline__ void push_floats(const float* p, uint32_t rank, const float (&v)[M], uint64_t* bar) {
  uint32_t to, on;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(p)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(on) : "r"(smem_u32(bar)), "r"(rank));
  if constexpr (M == 1)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
                 "r"(__float_as_uint(v[0])), "r"(on)
                 : "memory");
  else if constexpr (M == 2)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(on)
                 : "memory");
  else
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(on)
                 : "memory");
}
// Two floats at this CTA's shared address `p`, in CTA `rank` of the cluster.
__device__ __forceinline__ float2 peer_float2(const float* p, uint32_t rank) {
  uint32_t addr;
  float2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
// Four.
__device__ __forceinline__ float4 peer_float4(const float* p, uint32_t rank) {
  uint32_t addr;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// What a CTA works on: up to MT tokens of an adapter (n_adapters: tokens
// without one, rank 0).
struct Tile {
  int32_t adapter, count, rank;
  float scale;
};
__device__ __forceinline__ int32_t adapter_rank(const moe_lora_args& a, int32_t l) {
  if (l >= a.n_adapters) return 0;
  return a.ranks ? min(max(a.ranks[l], 0), a.max_rank) : a.max_rank;
}
__device__ __forceinline__ float adapter_scale(const moe_lora_args& a, int32_t l) {
  return l < a.n_adapters && a.scale ? a.scale[l] : 1.f;
}

// Finds this CTA's tile in the plan and its tokens (row[i], -1 past the
// count).  Returns false, for the whole cluster alike, where there is none left.
template <int MT>
__device__ __forceinline__ bool planned_tile(const moe_lora_args& a, const LoraPlan& p, int32_t tile, int32_t* row,
                                             Tile& t) {
  const int tid = threadIdx.x, L = a.n_adapters;
  __shared__ int32_t found[3];
  if (tid == 0) found[0] = -1;
  if (tid < MT) row[tid] = -1;
  pdl_wait();
  __syncthreads();
  for (int32_t l = tid; l <= L; l += blockDim.x) {
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
  t.rank = adapter_rank(a, t.adapter);
  t.scale = adapter_scale(a, t.adapter);
  if (tid < t.count) row[tid] = p.order[found[1] + tid];
  __syncthreads();
  return true;
}

// The same without a plan, for at most one token a thread: every CTA ranks the
// ids itself.  A token whose rank among its adapter's is a multiple of MT leads
// a tile, tiles in the order of their leaders.
template <int MT>
__device__ __forceinline__ bool ranked_tile(const moe_lora_args& a, int32_t tile, int32_t* row, int32_t* scratch,
                                            Tile& t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, L = a.n_adapters, n = a.n;
  __shared__ int32_t found[2];
  int32_t* leaders = scratch + kLoraThreads;  // per warp
  const int32_t mine = tid < n ? bucket_of(a.adapter_ids[tid], L) : -1;
  if (tid == 0) found[0] = -1;
  if (tid < MT) row[tid] = -1;
  scratch[tid] = mine;
  int32_t rank = __popc(__match_any_sync(0xffffffffu, mine) & ((1u << lane) - 1u));
  if (n > 32) {
    __syncthreads();
    const int4* ids4 = reinterpret_cast<const int4*>(scratch);
    const int32_t before = warp * 32 < n ? warp * 32 : 0;  // the warps before this one
#pragma unroll 8
    for (int32_t i = 0; i < before; i += 4) {
      const int4 v = ids4[i >> 2];
      rank += (v.x == mine) + (v.y == mine) + (v.z == mine) + (v.w == mine);
    }
  }
  const bool leads = mine >= 0 && rank % MT == 0;
  const uint32_t lead = __ballot_sync(0xffffffffu, leads);
  if (lane == 0) leaders[warp] = __popc(lead);
  __syncthreads();
  int32_t at = __popc(lead & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kLoraWarps; ++w) at += w < warp ? leaders[w] : 0;
  if (leads && at == tile) {
    found[0] = mine;
    found[1] = rank / MT;
  }
  __syncthreads();
  t.adapter = found[0];
  if (t.adapter < 0) return false;
  t.rank = adapter_rank(a, t.adapter);
  t.scale = adapter_scale(a, t.adapter);
  const bool in = mine == t.adapter && rank / MT == found[1];
  if (in) row[rank % MT] = tid;
  t.count = __syncthreads_count(in);
  return true;
}

// The block's inclusive scan of v; sums: 32 entries of shared memory.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  const int32_t before = lane < warp ? sums[lane] : 0;
  return v + __reduce_add_sync(0xffffffffu, before);
}

// The same without a plan for up to PER tokens a thread: every CTA counts the
// adapters' tokens and picks its tile's, an adapter's in the batch's order (which
// all CTAs agree on).  scratch: n_adapters + 1 and PER x warps entries.
template <int MT, int PER>
__device__ __forceinline__ bool counted_tile(const moe_lora_args& a, int32_t tile, int32_t* row, int32_t* scratch,
                                             Tile& t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, W = T / 32;
  const int32_t L = a.n_adapters, n = a.n;
  __shared__ int32_t found[2], tile_sums[32], token_sums[32];
  int32_t* count = scratch + PER * W;
  const int steps = (n + T - 1) / T;
  int32_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = tid + j * T < n ? a.adapter_ids[tid + j * T] : 0;
  for (int32_t l = tid; l <= L; l += T) count[l] = 0;
  if (tid == 0) found[0] = -1;
  if (tid < MT) row[tid] = -1;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {  // (one addition for a warp whose tokens share their adapter)
    if (j >= steps) break;
    key[j] = tid + j * T < n ? bucket_of(key[j], L) : -1;
    const bool one = __all_sync(0xffffffffu, key[j] == __shfl_sync(0xffffffffu, key[j], 0));
    if (key[j] >= 0 && (!one || lane == 0)) atomicAdd(&count[key[j]], one ? 32 : 1);
  }
  __syncthreads();
  // the adapter of this tile, adapters in order: each thread looks at a few
  const int32_t each = (L + T) / T, l0 = tid * each, l1 = min(l0 + each, L + 1);
  int32_t tiles = 0;
  for (int32_t l = l0; l < l1; ++l) tiles += (count[l] + MT - 1) / MT;
  int32_t at = block_scan(tiles, tile_sums) - tiles;
  if (tile >= at && tile < at + tiles)
    for (int32_t l = l0; l < l1; ++l) {
      const int32_t mine = (count[l] + MT - 1) / MT;
      if (tile < at + mine) {
        found[0] = l;
        found[1] = (tile - at) * MT;
        break;
      }
      at += mine;
    }
  __syncthreads();
  t.adapter = found[0];
  if (t.adapter < 0) return false;
  t.rank = adapter_rank(a, t.adapter);
  t.scale = adapter_scale(a, t.adapter);
  const int32_t first = found[1];
  t.count = min(MT, count[t.adapter] - first);
  // each of its tokens' place among them: tokens before it in its warp, and in the warps of lower tokens
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (j >= steps) break;
    const uint32_t same = __ballot_sync(0xffffffffu, key[j] == t.adapter);
    if (lane == 0) scratch[j * W + warp] = __popc(same);
  }
  __syncthreads();
  const int32_t mine = tid < steps * W ? scratch[tid] : 0;
  const int32_t before = block_scan(mine, token_sums) - mine;
  if (tid < steps * W) scratch[tid] = before;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (j >= steps) break;
    const uint32_t same = __ballot_sync(0xffffffffu, key[j] == t.adapter);
    const int32_t place = scratch[j * W + warp] + __popc(same & ((1u << lane) - 1u)) - first;
    if (key[j] == t.adapter && place >= 0 && place < MT) row[place] = tid + j * T;
  }
  __syncthreads();
  return true;
}

// 16 (or 8) bytes into a ring slot.
__device__ __forceinline__ void ring16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ring8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes of shared memory at offset `at` of the CTA's dynamic part.  (A plain
// load: what orders it after the copies is ring_wait, and in between the
// compiler may move it ahead of matrix instructions.)
__device__ __forceinline__ uint4 slot16(const char* sm, uint32_t at) { return *reinterpret_cast<const uint4*>(sm + at); }
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `ahead` (0..6) of the thread's newest groups are unfinished.
__device__ __forceinline__ void ring_wait(int ahead) {
  switch (ahead) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 6;" ::: "memory");
  }
}

// Ring stages of `step` bytes that fit, at most four.
__device__ __forceinline__ int ring_stages(uint32_t bytes, uint32_t step) {
  return 1 + (bytes >= 2 * step) + (bytes >= 3 * step) + (bytes >= 4 * step);
}

constexpr uint32_t kSlotVec = kLoraThreads * 16;  // one 16-byte vector of every thread

// Launches tiles x cluster CTAs in clusters of `cluster`; pdl: the kernel begins
// with a wait for the kernel before it.
template <typename... KArgs, typename... Args>
cudaError_t lora_launch_cluster(void (*kernel)(KArgs...), int32_t tiles, int32_t cluster, int threads, size_t smem,
                                bool pdl, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs that share a tile where one occupies an SM: as many (up to
// kLoraMaxCluster) as leave all tiles on the GPU at once.  How many clusters of
// a size that is depends on the SMs of its clusters of SMs and is asked for
// once a device and size.  `tiles`: the tiles to expect (where there are a few
// more, they wait for the first to finish).
constexpr int32_t kLoraMaxCluster = 8;
template <typename... KArgs>
cudaError_t lora_cluster(void (*kernel)(KArgs...), int threads, size_t smem, int32_t tiles,
                         std::atomic<int32_t> (&held)[kMaxDevices][kLoraMaxCluster + 1], int32_t* cluster) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (*cluster = kLoraMaxCluster; *cluster > 1; --*cluster) {
    int32_t most = dev < kMaxDevices ? held[dev][*cluster].load(std::memory_order_relaxed) : 0;
    if (!most) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)*cluster);
      cfg.blockDim = dim3((unsigned)threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = (unsigned)*cluster;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (dev < kMaxDevices) held[dev][*cluster].store(std::max(most, 1), std::memory_order_relaxed);
    }
    if (tiles <= most) break;
  }
  return cudaSuccess;
}

// lora_mma.cu: at most `tiles` tiles of kMmaTokens tokens; whether it takes a call's larger batches (lora_rows.cu the
// others, with both sides measured there).
constexpr int kMmaTokens = 128;
bool lora_mma_takes(const moe_lora_args& a);
cudaError_t launch_lora_mma(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, int32_t expected, cudaStream_t s);

// Reads and clears the flags of lora.cu's bounded waits.
cudaError_t lora_small_flags(int32_t* flags);

// lora_rows.cu: at most `tiles` tiles of kRowsTile tokens.
constexpr int kRowsTile = 64;
cudaError_t launch_lora_rows(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, int32_t expected, cudaStream_t s);

}  // namespace moe
