// linear_mma.cu -- matrix products of bf16 with an epilogue, on the tensor cores'
// asynchronous path (tcgen05, operands by TMA, accumulators in tensor memory).
//
// The features (a weight's rows) are the instruction's M and the rows of x its
// N, so that one kernel serves a single token (N = 16: the weights stream
// through) and thousands (N = 256), and a warp of the epilogue, whose lanes hold
// consecutive features of one row, turns its blocks of 32 by 32 in a padded slot of
// shared memory, so that memory sees 16 bytes a lane and whole sectors.
//
// Large products: a pair of CTAs (cta_group::2) shares an instruction of 256
// features, each holding its own features and half of the rows; a persistent
// grid takes the tiles in an order that keeps a few rows' and all weights' tiles
// in L2, and two accumulators let a tile's epilogue run beside the next tile's
// products.  Small ones: a CTA a tile of 128 features; where there are fewer
// tiles than SMs, the CTAs of a cluster split the columns and add their sums
// through each other's shared memory, in order.
//
// The products bound large ones: 16384 tokens of 4096 to 8192 with bias and relu2,
// its argument kept, 655 us back to back in a graph (1.68 PFLOP/s), 690 as called
// with inputs that change; 4314 tokens of 4096 to 2688 with a residual 64 us (1.48)
// and 71.  Small ones are bound by their start, 4 us until the first result, and a
// cluster's meeting: 24 tokens of 4096 to 4096 11.6 us.  A backward pass of 4314
// tokens of 2688 to 4608, d_weight in fp32, takes 164 us (1.30 PFLOP/s for 214
// GFLOP) and 170.
#include <algorithm>

#include "block.cuh"
#include "linear_act.cuh"
#include "linear_mma.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384, kEpilogueWarps = 8;  // warp 0: copies, 1: products, 2: tensor memory, 4..11: epilogue
constexpr int kMaxStages = 12;
constexpr uint32_t kSmem = 227 * 1024, kBarBytes = 1024;
constexpr uint32_t kPBytes = 128 * 128;  // a stage's features: 128 of 64 columns
constexpr uint32_t kSlotBytes = 16 * 36 * 4;  // of an epilogue warp
constexpr int kMaxCluster = 8;
// The tensor core cuts what it adds to a sum where it would round, always towards zero, which costs a sum of C products
// about 1e-9 C of its size, 5e-9 C where all have one sign.  A result in fp32 is therefore summed in tensor memory for 8
// blocks of 64 columns at a time, and from there on in registers (4314 columns: 4.7e-6 off without, 4.7e-7 so).  So is a
// result in bf16 of more than 512 blocks: 32768 columns of one sign lose a twentieth of half a step (131072: a fifth), for
// which reading the sums back is too dear (2048 x 32768 to 2048: 150 us, 183 so).
constexpr int32_t kChain = 8, kLongSum = 512;
constexpr int kChainBlocks = 4;  // of 32 sums a thread

// Set where a bounded wait ran out of a product that has no flags of its own; read by moe_linear_get_device_error.
__device__ int32_t g_linear_flags;

struct Plan {
  int32_t R, F, KB, terms;    // KB: blocks of 64 columns; terms: of q
  int32_t rows;               // of a tile: the instruction's N
  int32_t tiles_r, tiles, group;
  int32_t split, stages;
  int32_t beside;             // 1: runs beside the kernel before it, whose results it does not take
  int32_t chain;              // blocks of 64 columns that tensor memory sums before their sum moves to registers
  uint32_t stage_bytes;
  int32_t* flags;             // or nullptr: g_linear_flags
  LinearFinish e;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 peer_float4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Relaxed: what it announces are reads of tensor memory, which have returned (tmem_ld_wait); a release would wait for the
// epilogue's stores to global memory as well (a tile of one block of 64 columns: a sixth of its time).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_for(const Plan& p, uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait_sleep(bar, parity, 1000u)) return true;
    if (*gave_up) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *gave_up = 1;
      atomicOr(p.flags ? p.flags : &g_linear_flags, kFlagTimeout);
      return false;
    }
  }
}

template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if (CG == 2)  // the barrier is the pair's first CTA's
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc_mma_bf16(d, a, b, idesc, accumulate);
}
// Arrives on the barrier of each CTA of the pair once the products issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t first_cta) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)(3u << first_cta))
        : "memory");
  else
    tc_commit(bar);
}
template <int CG>
__device__ __forceinline__ void tmem_allocate(uint32_t* slot, uint32_t cols) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    tmem_dealloc(addr, cols);
}
// Descriptor of an operand with its M or N side contiguous: blocks of 64 (128 bytes) by 64 columns, 8 KB each, 128-byte
// swizzle; the leading offset goes from block to block, the stride offset from one group of 8 columns to the next.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(8192u >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// 32 lanes x 32 bit, 32 consecutive columns: fewer and wider reads, since each waits behind the products under way.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Warps 1 and 2 meet; whether warp 2 gave up.
__device__ __forceinline__ bool hand_over(bool gave_up) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, 64, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)gave_up)
      : "memory");
  return r != 0;
}

struct Maps {
  CUtensorMap p, q[kLinearTerms];
};

struct Tile {
  int32_t f0, r0;
};
// Tiles in bands of `group` row tiles, within a band all row tiles of one feature tile side by side.
__device__ __forceinline__ Tile tile_at(const Plan& p, int32_t t, int32_t feats) {
  const int32_t tiles_f = p.tiles / p.tiles_r, band = t / (p.group * tiles_f), in = t - band * p.group * tiles_f;
  const int32_t high = min(p.group, p.tiles_r - band * p.group);
  return {in / high * feats, (band * p.group + in % high) * p.rows};
}

// A block of 32 rows by 32 features between memory, where a lane moves 16 bytes of a row, and the sums, where a lane has a
// feature.  It turns in the warp's slot of shared memory: bf16 as words of two rows, so that a lane writes 16 words and
// reads 16; fp32 in two rounds.  Rows of the slot are 36 words apart, which keeps both sides off each other's banks.
constexpr int kSlotRow = 36;
struct BlockRows {  // the warp's 32 features of the rows from the tile's first on
  char* at;
  int64_t row;
};
__device__ __forceinline__ BlockRows block_rows(void* base, int64_t stride, int32_t f32, int32_t r0, int32_t f0) {
  const int64_t size = f32 ? 4 : 2;
  return {static_cast<char*>(base) + ((int64_t)r0 * stride + f0) * size, stride * size};
}
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, uint32_t which) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(which));
  return d;
}
constexpr uint32_t kLowHalves = 0x5410, kHighHalves = 0x7632;
// rows: how many there are from row c0 on; feats: from the warp's first feature on.
__device__ __forceinline__ void store32(const BlockRows& to, int32_t f32, const float (&v)[32], int32_t c0, int32_t rows,
                                        int32_t feats, int lane, uint32_t* slot) {
  char* at = to.at + c0 * to.row;
  if (f32) {
    at += (lane >> 3) * to.row + 16 * (lane & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 16; ++i) slot[i * kSlotRow + lane] = __float_as_uint(v[16 * h + i]);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k, at += 4 * to.row)
        if (16 * h + 4 * k + (lane >> 3) < rows && 4 * (lane & 7) < feats)
          *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(slot + (4 * k + (lane >> 3)) * kSlotRow + 4 * (lane & 7));
      __syncwarp();
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) slot[i * kSlotRow + lane] = pack2(v[2 * i], v[2 * i + 1]);
  __syncwarp();
  at += 2 * (lane >> 2) * to.row + 16 * (lane & 3);
#pragma unroll
  for (int k = 0; k < 2; ++k, at += 16 * to.row) {
    const uint32_t* from = slot + (8 * k + (lane >> 2)) * kSlotRow + 8 * (lane & 3);
    const uint4 a = *reinterpret_cast<const uint4*>(from), b = *reinterpret_cast<const uint4*>(from + 4);
    const int32_t r = 16 * k + 2 * (lane >> 2);
    if (8 * (lane & 3) < feats) {
      if (r < rows)
        *reinterpret_cast<uint4*>(at) = make_uint4(halves(a.x, a.y, kLowHalves), halves(a.z, a.w, kLowHalves),
                                                   halves(b.x, b.y, kLowHalves), halves(b.z, b.w, kLowHalves));
      if (r + 1 < rows)
        *reinterpret_cast<uint4*>(at + to.row) = make_uint4(halves(a.x, a.y, kHighHalves), halves(a.z, a.w, kHighHalves),
                                                            halves(b.x, b.y, kHighHalves), halves(b.z, b.w, kHighHalves));
    }
  }
  __syncwarp();
}
// The bf16 residual of a block as it lies in memory, on its way to the lanes that will put it into the slot.
__device__ __forceinline__ void load_residual(const BlockRows& from, int32_t c0, int32_t rows, int32_t feats, int lane,
                                              uint4 (&raw)[4]) {
  const char* at = from.at + (c0 + 2 * (lane >> 2)) * from.row + 16 * (lane & 3);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int32_t r = 16 * (k / 2) + 2 * (lane >> 2) + k % 2;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (8 * (lane & 3) < feats && r < rows)
      raw[k] = *reinterpret_cast<const uint4*>(at + (16 * (k / 2) + k % 2) * from.row);
  }
}
// v += scale times the residual; a bf16 one from raw.
__device__ __forceinline__ void add_residual(const BlockRows& from, int32_t f32, float scale, const uint4 (&raw)[4],
                                             int32_t c0, int32_t rows, int32_t feats, int lane, uint32_t* slot,
                                             float (&v)[32]) {
  if (f32) {
    const char* at = from.at + (c0 + (lane >> 3)) * from.row + 16 * (lane & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 d[4];
#pragma unroll
      for (int k = 0; k < 4; ++k, at += 4 * from.row) {
        d[k] = make_uint4(0, 0, 0, 0);
        if (16 * h + 4 * k + (lane >> 3) < rows && 4 * (lane & 7) < feats) d[k] = *reinterpret_cast<const uint4*>(at);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(slot + (4 * k + (lane >> 3)) * kSlotRow + 4 * (lane & 7)) = d[k];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * h + i] = fmaf(scale, __uint_as_float(slot[i * kSlotRow + lane]), v[16 * h + i]);
      __syncwarp();
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t* to = slot + (8 * k + (lane >> 2)) * kSlotRow + 8 * (lane & 3);
    const uint4 &a = raw[2 * k], &b = raw[2 * k + 1];  // the first and the second of two rows
    *reinterpret_cast<uint4*>(to) = make_uint4(halves(a.x, b.x, kLowHalves), halves(a.x, b.x, kHighHalves),
                                               halves(a.y, b.y, kLowHalves), halves(a.y, b.y, kHighHalves));
    *reinterpret_cast<uint4*>(to + 4) = make_uint4(halves(a.z, b.z, kLowHalves), halves(a.z, b.z, kHighHalves),
                                                   halves(a.w, b.w, kLowHalves), halves(a.w, b.w, kHighHalves));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t d = slot[i * kSlotRow + lane];
    v[2 * i] = fmaf(scale, bf16lo(d), v[2 * i]);
    v[2 * i + 1] = fmaf(scale, bf16hi(d), v[2 * i + 1]);
  }
  __syncwarp();
}
template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = linear_act(v[i], ACT);
}

template <int CG, bool P_MN, bool Q_MN, bool CHAIN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Plan p) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], t_full[2], t_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), cta = rank % CG, part = rank / CG, first_cta = rank - cta;  // of the pair
  const int32_t units = gridDim.x / (CG * p.split), unit = blockIdx.x / (CG * p.split);
  const uint32_t cols = p.rows <= 32 ? 64 : p.rows <= 64 ? 128 : p.rows <= 128 ? 256 : 512;
  const int32_t kb0 = (int32_t)((int64_t)p.KB * p.terms * part / p.split);
  const int32_t kb1 = (int32_t)((int64_t)p.KB * p.terms * (part + 1) / p.split);
  const int32_t my_rows = p.rows / CG;  // rows that this CTA holds

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&t_full[s], 1);
      mbar_init(&t_empty[s], CG * kEpilogueWarps);
    }
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.p);
    prefetch_tensormap(&maps.q[0]);
  }
  if (warp == 2) tmem_allocate<CG>(&tmem_slot, cols);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (!p.beside) pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int32_t t = unit; t < p.tiles && ok; t += units) {
        const Tile ti = tile_at(p, t, 128 * CG);
        const int32_t f = ti.f0 + 128 * cta, r = ti.r0 + my_rows * cta;
        int32_t term = kb0 / p.KB, c = (kb0 - term * p.KB) * 64;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
          if (!wait_for(p, &empty[s], ph ^ 1u, &gave_up)) {
            ok = false;
            break;
          }
          const uint32_t bar = CG == 2 ? peer_addr(&full[s], first_cta) : smem_u32(&full[s]);
          if (cta == 0) mbar_arrive_expect_tx(&full[s], CG * p.stage_bytes);
          const uint32_t at = smem_u32(sm) + s * p.stage_bytes;
          const CUtensorMap* mq = &maps.q[term];
          if (P_MN) {
            load_2d<CG>(at, &maps.p, f, c, bar);
            load_2d<CG>(at + 8192, &maps.p, f + 64, c, bar);
          } else {
            load_2d<CG>(at, &maps.p, c, f, bar);
          }
          if (Q_MN) {  // (whole boxes of 64 rows)
            for (int32_t j = 0; j < my_rows; j += 64) load_2d<CG>(at + kPBytes + j * 128, mq, r + j, c, bar);
          } else {
            load_2d<CG>(at + kPBytes, mq, c, r, bar);
          }
          if ((c += 64) >= 64 * p.KB) {
            c = 0;
            ++term;
          }
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {  // copies in flight land before the CTA goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && cta == 0) {
    // A shared-memory access by the thread that issues the products waits until those before it have read their operands;
    // so this warp makes none: warp 2 waits on the barriers and hands each block of 64 columns over.
    const uint32_t idesc = idesc_bf16(128 * CG, (uint32_t)p.rows) | (P_MN ? 1u << 15 : 0u) | (Q_MN ? 1u << 16 : 0u);
    const uint64_t desc_p = P_MN ? smem_desc_mn128(smem_u32(sm)) : smem_desc_k128(smem_u32(sm));
    const uint64_t desc_q = Q_MN ? smem_desc_mn128(smem_u32(sm) + kPBytes) : smem_desc_k128(smem_u32(sm) + kPBytes);
    int s = 0, it = 0;
    bool ok = true;
    for (int32_t t = unit; t < p.tiles && ok; t += units, ++it) {
      for (int32_t kb = kb0, chained = 0; kb < kb1; ++kb, ++chained) {
        if (CHAIN && chained == p.chain) chained = 0;
        const bool first = CHAIN ? chained == 0 : kb == kb0;
        if (first && kb != kb0) {
          if (lane == 0) commit<CG>(&t_full[it & 1], first_cta);
          ++it;
        }
        ok = !hand_over(false);
        if (!ok) break;
        if (lane == 0) {
          tc_fence_after();
          const uint64_t at = (uint64_t)((uint32_t)(s * p.stage_bytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma<CG>(tmem + (it & 1) * p.rows, desc_p + at + (P_MN ? 128 : 2) * k, desc_q + at + (Q_MN ? 128 : 2) * k,
                    idesc, !first || k != 0);
          commit<CG>(&empty[s], first_cta);
        }
        if (++s == p.stages) s = 0;
      }
      if (ok && lane == 0) commit<CG>(&t_full[it & 1], first_cta);
    }
    __syncwarp();
  } else if (warp == 2 && cta == 0) {
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int32_t t = unit; t < p.tiles && ok; t += units, ++it) {
      for (int32_t kb = kb0, chained = 0; kb < kb1 && ok; ++kb, ++chained) {
        if (CHAIN && chained == p.chain) chained = 0;
        const bool first = CHAIN ? chained == 0 : kb == kb0;
        if (first && kb != kb0) ++it;
        if (lane == 0) {
          if (first) ok = wait_for(p, &t_empty[it & 1], ((it >> 1) & 1) ^ 1u, &gave_up);
          ok = ok && wait_for(p, &full[s], ph, &gave_up);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (hand_over(!ok)) break;
        if (++s == p.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    uint32_t* slot = reinterpret_cast<uint32_t*>(sm + p.stages * p.stage_bytes + (warp - 4) * kSlotBytes);
    int it = 0;
    bool ok = true;
    for (int32_t t = unit; t < p.tiles && ok; t += units) {
      const Tile ti = tile_at(p, t, 128 * CG);
      const int32_t f0 = ti.f0 + 128 * cta + 32 * q, f = f0 + lane, rows = min(p.rows, p.R - ti.r0);
      const bool direct = p.split == 1;
      const float bias = direct && p.e.bias && f < p.F ? linear_read(p.e.bias, f, p.e.bias_f32) : 0.f;
      const BlockRows to_out = block_rows(p.e.out, p.e.out_stride, p.e.out_f32, ti.r0, f0),
                      to_z = block_rows(p.e.z, p.e.z_stride, p.e.z_f32, ti.r0, f0),
                      from_res = block_rows(const_cast<void*>(p.e.residual), p.e.residual_stride, p.e.residual_f32, ti.r0, f0);
      const int32_t feats = p.F - f0;
      const bool ahead = !CHAIN && direct && p.e.residual && !p.e.residual_f32;  // the next block's residual
      uint4 raw[4];
      if (ahead && 32 * half < rows) load_residual(from_res, 32 * half, rows - 32 * half, feats, lane, raw);
      // a block's sums: finished, or to shared memory where a cluster's meet (every copy has been read by then: they take
      // the stages' place)
      auto out = [&](float (&v)[32], int32_t c0) {
        const int32_t left = rows - c0;
        if (!direct) {
          float* to = reinterpret_cast<float*>(sm) + c0 * 128 + 32 * q + lane;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < p.rows) to[i * 128] = v[i];
          return;
        }
        if (p.e.bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += bias;
        }
        if (p.e.z) store32(to_z, p.e.z_f32, v, c0, left, feats, lane, slot);
        if (p.e.act == MOE_LINEAR_RELU2)
          act32<MOE_LINEAR_RELU2>(v);
        else if (p.e.act == MOE_LINEAR_SILU)
          act32<MOE_LINEAR_SILU>(v);
        else if (p.e.act == MOE_LINEAR_GELU_TANH)
          act32<MOE_LINEAR_GELU_TANH>(v);
        if (p.e.residual) {
          if (!ahead && !p.e.residual_f32) load_residual(from_res, c0, left, feats, lane, raw);
          add_residual(from_res, p.e.residual_f32, p.e.scale, raw, c0, left, feats, lane, slot, v);
          if (ahead && left > 64) load_residual(from_res, c0 + 64, left - 64, feats, lane, raw);
        }
        store32(to_out, p.e.out_f32, v, c0, left, feats, lane, slot);
      };
      auto arrive = [&](uint32_t acc) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            peer_arrive(peer_addr(&t_empty[acc], first_cta));
          else
            mbar_arrive(&t_empty[acc]);
        }
      };
      if (CHAIN) {
        float sum[kChainBlocks][32];
        for (int32_t kb = kb0; kb < kb1; kb += p.chain, ++it) {
          const uint32_t acc = it & 1;
          ok = wait_for(p, &t_full[acc], (it >> 1) & 1, &gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < kChainBlocks; ++b) {
            const int32_t c0 = 32 * half + 64 * b;
            if (c0 >= rows) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // (wider reads would not leave the sums their registers)
              uint32_t d[16];
              tmem_ld16(tmem + lanes + acc * p.rows + c0 + 16 * h, d);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                sum[b][16 * h + i] = (kb == kb0 ? 0.f : sum[b][16 * h + i]) + __uint_as_float(d[i]);
            }
          }
          arrive(acc);
        }
        if (!ok) break;
#pragma unroll
        for (int b = 0; b < kChainBlocks; ++b) {
          const int32_t c0 = 32 * half + 64 * b;
          if (c0 < rows) out(sum[b], c0);
        }
      } else {
        const uint32_t acc = it & 1;
        ok = wait_for(p, &t_full[acc], (it >> 1) & 1, &gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        for (int32_t c0 = 32 * half; c0 < rows; c0 += 64) {
          uint32_t d[32];
          tmem_ld32(tmem + lanes + acc * p.rows + c0, d);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(d[i]);
          out(v, c0);
        }
        arrive(acc);
        ++it;
      }
    }
  }
  __syncwarp();
  if (p.split > 1) {
    cluster_sync();
    Tile ti = tile_at(p, unit, 128 * CG);
    ti.f0 += 128 * cta;
    const int32_t rows = min(p.rows, p.R - ti.r0);
    // four features of a row a thread; the CTAs' sums are added in order
    for (int32_t i = (int32_t)part * kThreads + threadIdx.x; i < rows * 32 && !gave_up; i += p.split * kThreads) {
      const int32_t r = ti.r0 + i / 32, f = ti.f0 + 4 * (i & 31);
      if (f >= p.F) continue;
      float v[4] = {};
      for (int c = 0; c < p.split; ++c) {
        const float4 x = peer_float4(peer_addr(sm + i * 16, c * CG + cta));
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      }
      const LinearFinish& e = p.e;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float z = v[j] + (e.bias ? linear_read(e.bias, f + j, e.bias_f32) : 0.f);
        if (e.z) linear_write(e.z, (int64_t)r * e.z_stride + f + j, e.z_f32, z);
        v[j] = linear_act(z, e.act);
        if (e.residual)
          v[j] = fmaf(e.scale, linear_read(e.residual, (int64_t)r * e.residual_stride + f + j, e.residual_f32), v[j]);
      }
      if (e.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(e.out) + (int64_t)r * e.out_stride + f) =
            make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.out) + (int64_t)r * e.out_stride + f) =
            make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2 || p.split > 1) cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<CG>(tmem, cols);
  }
  if (p.beside) pdl_wait();  // (what follows this kernel follows the one before it too)
}

template <int CG, bool P_MN, bool Q_MN, bool CHAIN>
cudaError_t launch(const Plan& p, const Maps& m, int32_t units, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(linear_kernel<CG, P_MN, Q_MN, CHAIN>, kSmem - kBarBytes, configured);
  if (e != cudaSuccess) return e;
  const uint32_t cluster = (uint32_t)(CG * p.split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + p.stages * p.stage_bytes + kEpilogueWarps * kSlotBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_kernel<CG, P_MN, Q_MN, CHAIN>, m, p);
}
template <int CG, bool CHAIN>
cudaError_t launch_as(bool p_mn, bool q_mn, const Plan& p, const Maps& m, int32_t units, cudaStream_t s) {
  if (p_mn) return q_mn ? launch<CG, true, true, CHAIN>(p, m, units, s) : launch<CG, true, false, CHAIN>(p, m, units, s);
  return q_mn ? cudaErrorInvalidValue : launch<CG, false, false, CHAIN>(p, m, units, s);
}

// An operand of `outer` features or rows and C columns, in boxes of `box` of them by 64 columns.
cudaError_t operand_map(CUtensorMap* map, const LinearOperand& o, int32_t outer, int32_t C, int32_t box) {
  return o.c_inner ? make_tmap_bf16(map, o.data, C, outer, o.stride, 64, box)
                   : make_tmap_bf16(map, o.data, outer, C, o.stride, 64, 64);
}

// How many clusters of each size the device holds at once, asked for once a device.
cudaError_t held_clusters(int32_t (&held)[kMaxCluster + 1]) {
  static std::atomic<int32_t> known[kMaxDevices][kMaxCluster + 1];
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!known[dev][kMaxCluster].load(std::memory_order_acquire)) {
    e = raise_smem_limit(linear_kernel<1, false, false, false>, kSmem - kBarBytes, configured);
    for (int n = 1; n <= kMaxCluster && e == cudaSuccess; ++n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)n);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmem - kBarBytes;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = (unsigned)n;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int most = 0;
      e = cudaOccupancyMaxActiveClusters(&most, linear_kernel<1, false, false, false>, &cfg);
      if (e == cudaSuccess) known[dev][n].store(std::max(most, 1), std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
  }
  for (int n = 1; n <= kMaxCluster; ++n) held[n] = known[dev][n].load(std::memory_order_acquire);
  return cudaSuccess;
}

struct Shape {
  int32_t cg, rows, split;
  double cost;
};
// The tiles that should take least, in clocks: a block of 64 columns costs an SM 2 clocks a row of its tile for the
// products or its bytes from L2 (64 a clock), and never less than 500 (128 rows of 4096 columns to 4096: 22.5 us in tiles of
// 32 rows, 22.2 in one of 128); a tile its start or, where its blocks are few, its epilogue; a pair its meetings; a split
// that of its sums.  Over 96 products of 30 to 16384 tokens the tiles that this takes are 1.6 % slower than the best that
// there are.  share: of the SMs, a split takes one part of so many.
Shape choose(int32_t R, int32_t F, int32_t blocks, bool q_mn, int32_t share, const int32_t (&clusters)[kMaxCluster + 1]) {
  static const int32_t kRows[] = {16, 32, 64, 96, 128, 160, 192, 224, 256};
  Shape best = {};
  double least = 0;
  for (int cg = 1; cg <= 2; ++cg)
    for (const int32_t rows : kRows) {
      if (rows % (16 * cg) || (q_mn && rows < 64 * cg)) continue;
      if (rows >= 2 * (int64_t)R && rows > 64 * cg) continue;
      const int64_t tiles = (int64_t)((R + rows - 1) / rows) * ((F + 128 * cg - 1) / (128 * cg));
      const int32_t held = rows / cg, units = clusters[cg];
      const double block = std::max({2.0 * rows, (16384.0 + 128.0 * (q_mn ? (held + 63) / 64 * 64 : held)) / 64, 500.0});
      for (int split = 1; split <= kMaxCluster / cg && split <= blocks; ++split) {
        if (split > 1 && tiles > clusters[cg * split] / share) break;
        const double waves = split > 1 ? 1 : (double)((tiles + units - 1) / units);
        const double own = (blocks + split - 1) / split * block;
        const double cost = waves * std::max(own + 1000, 14.0 * rows + 500) + 2000 + 16.0 * rows + (cg == 2 ? 800 : 0) +
                            (split > 1 ? 3000 + 16.0 * rows : 0);
        if (!best.cg || cost < least) {
          least = cost;
          best = {cg, rows, split, cost};
        }
      }
    }
  return best;
}

}  // namespace

cudaError_t launch_linear_mma(const LinearProduct& a, cudaStream_t s) {
  int32_t clusters[kMaxCluster + 1];
  cudaError_t e = held_clusters(clusters);
  if (e != cudaSuccess) return e;
  Plan p = {};
  p.R = a.R;
  p.F = a.F;
  p.KB = (a.C + 63) / 64;
  p.terms = a.terms;
  p.e = a.finish;
  p.beside = a.beside;
  p.flags = a.flags;
  p.split = 1;
  const LinearFinish& f = a.finish;
  const bool q_mn = !a.q[0].c_inner, p_mn = !a.p.c_inner;
  const bool f32 = f.out_f32 || (f.z && f.z_f32);
  Shape shape = choose(a.R, a.F, p.KB * p.terms, q_mn, 1, clusters);
  if (a.share > 1) {  // half of the SMs where that costs less than the other product would lose
    const Shape half = choose(a.R, a.F, p.KB * p.terms, q_mn, a.share, clusters);
    if (half.cost < 1.25 * shape.cost) shape = half;
  }
  const int cg = shape.cg;
  p.rows = shape.rows;
  p.split = shape.split;
  const int32_t feats = 128 * cg, q_rows = q_mn ? (p.rows / cg + 63) / 64 * 64 : p.rows / cg;
  p.tiles_r = (a.R + p.rows - 1) / p.rows;
  const int64_t tiles = (int64_t)p.tiles_r * ((a.F + feats - 1) / feats);
  if (tiles > INT32_MAX / kMaxCluster) return cudaErrorInvalidValue;
  p.tiles = (int32_t)tiles;
  p.group = std::min(8, p.tiles_r);
  p.stage_bytes = kPBytes + (uint32_t)q_rows * 128;
  const int32_t units = p.split > 1 ? p.tiles : std::min(clusters[cg], p.tiles);
  p.stages = std::min<int32_t>(kMaxStages, (kSmem - kBarBytes - 1024 - kEpilogueWarps * kSlotBytes) / p.stage_bytes);
  // (the sums of a cluster meet where the stages were)
  if (p.split > 1 && (uint32_t)p.rows * 512 > p.stages * p.stage_bytes) return cudaErrorInvalidConfiguration;
  const int32_t own = (p.KB * p.terms + p.split - 1) / p.split;
  const bool chain = own > (f32 ? kChain : kLongSum);
  p.chain = chain ? kChain : own;
  Maps m;
  e = operand_map(&m.p, a.p, a.F, a.C, 128);
  for (int i = 0; i < kLinearTerms && e == cudaSuccess; ++i) {
    if (i < p.terms)
      e = operand_map(&m.q[i], a.q[i], a.R, a.C, p.rows / cg);
    else
      m.q[i] = m.q[0];
  }
  if (e != cudaSuccess) return e;
  if (cg == 2) return chain ? launch_as<2, true>(p_mn, q_mn, p, m, units, s) : launch_as<2, false>(p_mn, q_mn, p, m, units, s);
  return chain ? launch_as<1, true>(p_mn, q_mn, p, m, units, s) : launch_as<1, false>(p_mn, q_mn, p, m, units, s);
}

cudaError_t linear_mma_flags(int32_t* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_linear_flags, sizeof(int32_t));
  const int32_t zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_linear_flags, &zero, sizeof(int32_t));
  return e;
}

}  // namespace moe
