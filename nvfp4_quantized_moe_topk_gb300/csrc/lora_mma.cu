// lora_mma.cu -- the adapters for many tokens: a CTA, or a cluster of CTAs,
// takes 128 tokens of one adapter through both products on the tensor cores'
// asynchronous path (tcgen05, accumulators in tensor memory).
//
// Moving x, y and out bounds it.  Warp-level matrix instructions reread the
// adapter's matrices from shared memory for every 16 tokens; here one
// instruction takes 128 tokens, the operands go from shared memory to the
// tensor core without passing the warps, and the warps only copy and finish.
// What a step then costs is issuing its copies, one barrier and a few waits,
// one after the other; so two halves of the CTA (8 warps each) take alternate
// steps with barriers, rings and accumulators of their own, and one half's
// copies run beside the other's waits (16384 tokens, 4096 to 2048, rank 64,
// bf16: 92 us with one half of 512 threads, 75 with two, and 76 since v has three
// terms, of which the bytes are 40; 3.6 TB/s).  Where there are fewer tiles than SMs, the CTAs of a cluster
// take turns with the steps of both products and add their D1 through each
// other's shared memory (4096 tokens, 4096 to 4096, rank 64: 94 us with a CTA a
// tile, 43 with three, 38 with four).
//
//   first product:  D1[128 tokens][ranks] += x chunk . A chunk^T, 64 columns of
//     in_features a step (the tokens' rows are gathered: 8 lanes copy 128 bytes
//     of one); each half has a D1, and they are added at the end.
//   v = scale D1 as a sum of three bf16 terms, each a K-major operand in shared
//     memory.
//   second product: D2[128][a block of 64 columns, 32 where y or out is fp32] =
//     sum over terms of v . B rows^T.  y comes in and out leaves through shared
//     memory, so that both move in whole 128-byte lines.  Above 64 ranks, where v
//     takes 96 KB, a bf16 out takes a bf16 y's place there.
#include "lora.cuh"

namespace moe {

namespace {

constexpr int kMmaTile = kMmaTokens;
constexpr int kMmaThreads = 512, kMmaHalf = kMmaThreads / 2;
constexpr uint32_t kOperandTile = 128 * 128;  // 128 rows of 64 bf16
constexpr uint32_t kMmaMaxStages = 8;
constexpr uint32_t kMmaSmem = 226 * 1024;
constexpr uint32_t kD2 = 256, kTmemCols = 512;  // tensor memory: the halves' D1 in 128 columns each, then their D2

// Set where a bounded wait ran out; read by moe_lora_get_device_error.
__device__ int32_t g_lora_flags;

// Offset of 16-byte piece p of row r in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t p) { return r * 128 + ((p ^ (r & 7)) << 4); }

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// The barrier of a half; true for all where `any` is for one.
__device__ __forceinline__ bool half_or(int half, bool any) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)any), "r"(half + 1), "n"(kMmaHalf)
      : "memory");
  return r != 0;
}

__host__ __device__ inline int32_t block_columns(bool y_f32, bool out_f32) { return y_f32 || out_f32 ? 32 : 64; }
// Bytes of a half's ring steps: x and A; y and B.
__host__ __device__ inline uint32_t mma_step1(int32_t ranks16) { return kOperandTile + (uint32_t)ranks16 * 16 * 128; }
__host__ __device__ constexpr uint32_t mma_step2(bool has_y, int32_t rank_blocks, int32_t columns) {
  return (has_y ? kOperandTile : 0) + (uint32_t)rank_blocks * columns * 128;
}

// Whether out takes y's place in its ring step (the same types; each thread writes what it has read), which leaves room
// for a second step beside v; else the halves have an out block each.
__host__ __device__ inline bool out_over_y(const moe_lora_args& a, int rank_blocks) {
  return rank_blocks > 1 && a.y.data && a.y_dtype == MOE_DTYPE_BF16 && a.out_dtype == MOE_DTYPE_BF16;
}
// Bytes of the out blocks and v.
__host__ __device__ constexpr uint32_t mma_fixed(bool over_y, int rank_blocks) {
  return ((over_y ? 0u : 2u) + kLoraTerms * rank_blocks) * kOperandTile;
}
// Bytes of a half's ring in the second product.
constexpr uint32_t mma_ring(bool over_y, int rank_blocks) {
  return (kMmaSmem - 1024 - mma_fixed(over_y, rank_blocks)) / 2 / 1024 * 1024;
}
// (the waits are for all but the newest step; the sums of a cluster meet in the 64 KB before v)
static_assert(mma_ring(false, 1) >= 2 * mma_step2(true, 1, 64) && mma_ring(true, 2) >= 2 * mma_step2(true, 2, 64) &&
                  mma_ring(false, 2) >= 2 * mma_step2(true, 2, 32) && mma_ring(false, 2) >= 2 * mma_step2(false, 2, 64),
              "two steps of the second product have to fit");
static_assert(mma_ring(true, 2) >= 128 * kMmaTile * 4 && mma_ring(false, 2) + 2 * kOperandTile >= 128 * kMmaTile * 4,
              "the sums of 128 ranks have to end before v");

// RB: blocks of 64 ranks (1 or 2).
template <int RB>
__global__ void __launch_bounds__(kMmaThreads, 1)
    lora_mma_kernel(const moe_lora_args a, const LoraPlan plan, uint32_t ring_bytes) {
  extern __shared__ __align__(16) char sm_raw[];
  __shared__ int32_t row[kMmaTile];
  __shared__ __align__(8) uint64_t done1[2][kMmaMaxStages], done2[2];
  __shared__ uint32_t tmem_slot;
  char* sm = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = tid / kMmaHalf, htid = tid % kMmaHalf, hwarp = htid >> 5;
  const uint32_t C = cluster_size(), cr = cluster_rank();
  const int32_t mine = (int32_t)cr * 2 + half, jump = (int32_t)C * 2;  // this half's first step, and from one to the next
  if (tid == 0) {
    for (int h = 0; h < 2; ++h) {
      for (uint32_t s = 0; s < kMmaMaxStages; ++s) mbar_init(&done1[h][s], 1);
      mbar_init(&done2[h], 1);
    }
    fence_mbar_init();
  }
  // While the plan is made: x to L2 (up to 48 MB, so that it is still there when it is read), the rows dealt to the
  // grid's threads.  3 to 4 % of a call of 2000 to 6000 tokens; y as well, or a larger x, gains nothing or loses.
  if ((int64_t)a.n * a.in_features <= (24 << 20)) {
    const int64_t xs = (a.x.stride ? a.x.stride : a.in_features) * 2;
    for (int64_t r = blockIdx.x + (int64_t)tid * gridDim.x; r < a.n; r += (int64_t)kMmaThreads * gridDim.x)
      prefetch_l2(static_cast<const char*>(a.x.data) + r * xs, (uint32_t)a.in_features * 2);
  }
  Tile t;
  if (!planned_tile<kMmaTile>(a, plan, (int32_t)(blockIdx.x / C), row, t)) return;
  if (warp == 0) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int32_t rank = t.rank, ranks16 = (rank + 15) / 16;
  // First product: each half's ring is half of the space.  Then: the first half's ring, the halves' out blocks, v
  // [kLoraTerms][RB] operand tiles, the second half's ring (which each half may fill when its own part of the first
  // product is done).
  const bool over_y = out_over_y(a, RB);
  const uint32_t sm_u32 = smem_u32(sm), space = 2 * ring_bytes + mma_fixed(over_y, RB);
  const uint32_t ring1_bytes = space / 2 / 1024 * 1024, ring1 = half * ring1_bytes;
  const uint32_t ring = half * (space - ring_bytes), out_at = ring_bytes;
  const uint32_t v_at = ring_bytes + (over_y ? 0 : 2 * kOperandTile);
  const uint32_t quadrant = (uint32_t)(32 * (warp & 3)) << 16;  // this warp's lanes of tensor memory
  const int m = 32 * (warp & 3) + lane;                         // its thread's token
  const int p8 = htid & 7, r8 = htid >> 3;  // copies of 128-byte rows: piece, first row (the others 32, 64, 96 further)
  const uint32_t to8 = swizzled(r8, p8);    // (32 rows further: the same swizzle)
  bool dead = false;                        // a wait ran out

  // out = y + B v (its first steps are fetched before v is made)
  const bool yf = a.y_dtype == MOE_DTYPE_F32, of = a.out_dtype == MOE_DTYPE_F32, has_y = a.y.data != nullptr;
  const int32_t columns = block_columns(yf, of), blocks = (a.out_features + columns - 1) / columns;
  const uint32_t y_size = yf ? 4 : 2, o_size = of ? 4 : 2, out_idesc = idesc_bf16(128, (uint32_t)columns);
  const uint32_t b_at = has_y ? kOperandTile : 0, b_tile = columns * 128;
  const uint32_t out_step = max(mma_step2(has_y, rank > 0 ? RB : 0, columns), 1024u);
  const int out_stages = (int)min(kMmaMaxStages, ring_bytes / out_step);
  // rows of y and out in vectors of 16 bytes: a product of two 32-bit numbers a row
  const uint32_t y_stride = (uint32_t)((a.y.stride ? a.y.stride : a.out_features) * y_size / 16);
  const uint32_t o_stride = (uint32_t)((a.out.stride ? a.out.stride : a.out_features) * o_size / 16);
  const char* y_base = static_cast<const char*>(a.y.data);
  char* o_base = static_cast<char*>(a.out.data);
  const uint32_t y_pieces = columns * y_size / 16, o_pieces = columns * o_size / 16;  // of a block's row: 8 or 4
  const uint32_t y_row = (uint32_t)a.out_features * y_size / 16, o_row = (uint32_t)a.out_features * o_size / 16;
  const uint32_t b_bytes = (uint32_t)a.max_rank * 2;
  const char* B = reinterpret_cast<const char*>(a.b) +
                  (rank > 0 ? ((int64_t)t.adapter * a.out_features + r8) * (int64_t)b_bytes + 16 * p8 : 0);
  auto fetch_out = [&](int32_t ob, int stage) {
    if (ob < blocks) {
      const uint32_t at = ring + stage * out_step + to8, vec = (uint32_t)ob * y_pieces + p8;
      if (has_y && (uint32_t)p8 < y_pieces && vec < y_row) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t tok = row[r8 + 32 * i];
          if (tok >= 0) ring16(sm_u32 + at + i * 32 * 128, y_base + (((uint64_t)(uint32_t)tok * y_stride + vec) << 4));
        }
      }
      const int32_t left = min(a.out_features - ob * columns, columns);
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        const int32_t rest = rank - 64 * k - 8 * p8;  // ranks in this thread's piece and after it
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (p8 + 8 * k >= 2 * ranks16 || r8 + 32 * i >= left) break;
          const uint32_t to = at + b_at + k * b_tile + i * 32 * 128;
          const char* from = B + ((uint64_t)(uint32_t)(ob * columns + 32 * i) * b_bytes + 128 * k);
          if (rest >= 8) {
            ring16(sm_u32 + to, from);
          } else {  // what lies beyond the rank may hold anything
            uint4 b = make_uint4(0, 0, 0, 0);
            if (rest > 0) {
              b = __ldg(reinterpret_cast<const uint4*>(from));
              b.x &= rest >= 2 ? 0xffffffffu : 0xffffu;
              b.y &= rest >= 4 ? 0xffffffffu : rest == 3 ? 0xffffu : 0u;
              b.z &= rest >= 6 ? 0xffffffffu : rest == 5 ? 0xffffu : 0u;
              b.w &= rest == 7 ? 0xffffu : 0u;
            }
            *reinterpret_cast<uint4*>(sm + to) = b;
          }
        }
      }
    }
    ring_commit();
  };
  if (rank > 0) {
    const uint32_t row_bytes = (uint32_t)a.in_features * 2, idesc = idesc_bf16(128, (uint32_t)ranks16 * 16);
    const int32_t chunks = (a.in_features + 63) / 64;
    const int64_t xs = (a.x.stride ? a.x.stride : a.in_features) * 2;
    const char* xr[4];  // (places past the tile's count: its first token, and their rows are not looked at)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t tok = row[r8 + 32 * i];
      xr[i] = static_cast<const char*>(a.x.data) + (int64_t)(tok >= 0 ? tok : row[0]) * xs + 16 * p8;
    }
    // rows of A past the rank reach only columns of D1 that are not looked at
    const int32_t a_rows = min(16 * ranks16, a.max_rank);
    const char* Ar = reinterpret_cast<const char*>(a.a) +
                     ((int64_t)t.adapter * a.max_rank + r8) * (int64_t)row_bytes + 16 * p8;
    const uint32_t step = mma_step1(ranks16);
    const int stages = (int)min(kMmaMaxStages, ring1_bytes / step);
    auto fetch = [&](int32_t c, int stage) {
      if (c < chunks) {
        const uint32_t off = (uint32_t)c * 128, at = ring1 + stage * step + to8;
        if (off + 16 * p8 < row_bytes) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ring16(sm_u32 + at + i * 32 * 128, xr[i] + off);
#pragma unroll
          for (int i = 0; i < 2 * RB; ++i)
            if (r8 + 32 * i < a_rows)
              ring16(sm_u32 + at + kOperandTile + i * 32 * 128, Ar + ((uint64_t)(32 * i) * row_bytes + off));
        } else {  // past the row's end
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint4*>(sm + at + i * 32 * 128) = make_uint4(0, 0, 0, 0);
            if (i < 2 * RB && r8 + 32 * i < a_rows)
              *reinterpret_cast<uint4*>(sm + at + kOperandTile + i * 32 * 128) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      ring_commit();
    };
    for (int s = 0; s + 1 < stages; ++s) fetch(mine + jump * s, s);
    int stage = 0, last = 0;
    uint32_t parity = 0, last_parity = 0;
    for (int32_t c = mine; c < chunks; c += jump) {
      ring_wait(stages - 2);
      fence_proxy_async_smem();
      dead = half_or(half, dead);
      if (dead) break;
      if (hwarp == 0) {
        if (elect_one()) {
          const uint32_t x_at = sm_u32 + ring1 + stage * step, a_at = x_at + kOperandTile;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16(tmem + half * 128, smem_desc_k128(x_at + 32 * k), smem_desc_k128(a_at + 32 * k), idesc,
                        c != mine || k != 0);
          tc_commit(&done1[half][stage]);
        }
        __syncwarp();
      }
      // the step before this one has been read: its slot takes the chunk `stages - 1` steps ahead
      if (c != mine && !mbar_wait(&done1[half][last], last_parity, &g_lora_flags)) dead = true;
      fetch(c + jump * (stages - 1), stage == 0 ? stages - 1 : stage - 1);
      last = stage;
      last_parity = parity;
      if (++stage == stages) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (mine < chunks && !dead && !mbar_wait(&done1[half][last], last_parity, &g_lora_flags)) dead = true;
    ring_wait(0);
    // the CTAs' sums of a cluster meet in the (still unused) out blocks, those of two blocks of ranks in the 64 KB
    // before v: the first ring, and out blocks where there are any
    const bool ring_meets = RB > 1 && C > 1;
    if (!dead && !ring_meets)
      for (int s = 0; s + 1 < out_stages; ++s) fetch_out(mine + jump * s, s);
    dead = __syncthreads_or(dead);
    tc_fence_after();
    // D1 -> v: a thread its token's 16 ranks from 16 j on, j = j0, j0 + 4
    const int32_t j0 = warp >> 2;
    float s[RB][16];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int32_t j = j0 + 4 * b;
      if (j >= ranks16 || dead) continue;
      uint32_t d0[16] = {}, d1[16] = {};
      if ((int32_t)cr * 2 < chunks) tmem_ld16(tmem + quadrant + 16 * j, d0);  // (a half without a step has no sum)
      if ((int32_t)cr * 2 + 1 < chunks) tmem_ld16(tmem + quadrant + 128 + 16 * j, d1);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = __uint_as_float(d0[i]) + __uint_as_float(d1[i]);
    }
    if (C > 1) {  // [4 ranks][128 tokens], added in the order of the CTAs, the same in each of them
      float* meet = reinterpret_cast<float*>(sm + (ring_meets ? 0 : out_at)) + m * 4;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + 4 * b < ranks16 && !dead)
            *reinterpret_cast<float4*>(meet + (4 * (j0 + 4 * b) + i) * kMmaTile * 4) =
                make_float4(s[b][4 * i], s[b][4 * i + 1], s[b][4 * i + 2], s[b][4 * i + 3]);
      cluster_sync();
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        if (j0 + 4 * b >= ranks16 || dead) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
        for (uint32_t r = 0; r < C; ++r) {
          float4 p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = peer_float4(meet + (4 * (j0 + 4 * b) + i) * kMmaTile * 4, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[b][4 * i] += p[i].x;
            s[b][4 * i + 1] += p[i].y;
            s[b][4 * i + 2] += p[i].z;
            s[b][4 * i + 3] += p[i].w;
          }
        }
      }
      cluster_arrive();  // (waited for before the first write to where they met)
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int32_t j = j0 + 4 * b;
      if (j >= ranks16 || dead) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 16 * j + i < rank ? s[b][i] * t.scale : 0.f;
      for (int k = 0; k < kLoraTerms; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = take_terms(s[b][8 * h + 2 * i], s[b][8 * h + 2 * i + 1]);
          *reinterpret_cast<uint4*>(sm + v_at + (uint32_t)(k * RB + b) * kOperandTile + swizzled(m, j0 * 2 + h)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    if (C > 1) cluster_wait();
    if (ring_meets && !dead)
      for (int s = 0; s + 1 < out_stages; ++s) fetch_out(mine + jump * s, s);
    __syncthreads();
    tc_fence_after();
  } else {
    for (int s = 0; s + 1 < out_stages; ++s) fetch_out(mine + jump * s, s);
  }

  // adds y (in ring step `stage`) to the half's D2, 16 of a thread's columns from `first` on, into the out block
  auto finish = [&](uint32_t first, int stage, char* obuf) {
    uint32_t d[16];
    if (rank > 0) {
      tmem_ld16(tmem + quadrant + kD2 + half * 64 + first, d);
      tmem_ld_wait();
    }
    float r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = rank > 0 ? __uint_as_float(d[i]) : 0.f;
    if (has_y && yf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 y = slot16(sm, ring + stage * out_step + swizzled(m, first / 4 + i));
        r[4 * i] += __uint_as_float(y.x);
        r[4 * i + 1] += __uint_as_float(y.y);
        r[4 * i + 2] += __uint_as_float(y.z);
        r[4 * i + 3] += __uint_as_float(y.w);
      }
    } else if (has_y) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float y[8];
        unpack8(slot16(sm, ring + stage * out_step + swizzled(m, first / 8 + i)), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[8 * i + j] += y[j];
      }
    }
    if (of) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(obuf + swizzled(m, first / 4 + i)) =
            make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(obuf + swizzled(m, first / 8 + i)) =
            make_uint4(pack2(r[8 * i], r[8 * i + 1]), pack2(r[8 * i + 2], r[8 * i + 3]),
                       pack2(r[8 * i + 4], r[8 * i + 5]), pack2(r[8 * i + 6], r[8 * i + 7]));
    }
  };
  int stage = 0;
  uint32_t parity = 0;
  for (int32_t ob = mine; ob < blocks && !dead; ob += jump) {
    ring_wait(out_stages - 2);
    fence_proxy_async_smem();
    dead = half_or(half, dead);  // block ob has landed, and the out block before it has been written out
    if (dead) break;
    char* obuf = sm + (over_y ? ring + stage * out_step : out_at + half * kOperandTile);
    if (rank > 0) {
      if (hwarp == 0) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t b = sm_u32 + ring + stage * out_step + b_at;
          for (int k = 0; k < kLoraTerms; ++k)
            for (int32_t j = 0; j < ranks16; ++j)
              tc_mma_bf16(tmem + kD2 + half * 64, smem_desc_k128(sm_u32 + v_at + (uint32_t)(k * RB + j / 4) * kOperandTile + (j % 4) * 32),
                          smem_desc_k128(b + (uint32_t)(j / 4) * b_tile + (j % 4) * 32), out_idesc, (k | j) != 0);
          tc_commit(&done2[half]);
        }
        __syncwarp();
      }
    }
    // the step before this one has been read: its slot takes the block `out_stages - 1` steps ahead
    fetch_out(ob + jump * (out_stages - 1), stage == 0 ? out_stages - 1 : stage - 1);
    if (rank > 0) {
      if (!mbar_wait(&done2[half], parity, &g_lora_flags)) dead = true;
      parity ^= 1;
      __syncwarp();
      tc_fence_after();
    }
    for (int32_t u = (hwarp >> 2) * 16; u < columns; u += 32) finish(u, stage, obuf);
    tc_fence_before();
    if (half_or(half, dead)) {
      dead = true;
      break;
    }
    // the out block to memory, whole lines at a time
    const uint32_t vec = (uint32_t)ob * o_pieces + p8;
    if ((uint32_t)p8 < o_pieces && vec < o_row) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t tok = row[r8 + 32 * i];
        if (tok >= 0)
          *reinterpret_cast<uint4*>(o_base + (((uint64_t)(uint32_t)tok * o_stride + vec) << 4)) =
              *reinterpret_cast<const uint4*>(obuf + to8 + i * 32 * 128);
      }
    }
    stage = stage + 1 == out_stages ? 0 : stage + 1;
  }
  ring_wait(0);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int RB>
cudaError_t lora_mma_launch(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, int32_t expected, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = raise_smem_limit(lora_mma_kernel<RB>, kMmaSmem, configured);
  if (e != cudaSuccess) return e;
  static std::atomic<int32_t> held[kMaxDevices][kLoraMaxCluster + 1];
  int32_t cluster = 1;
  e = lora_cluster(lora_mma_kernel<RB>, kMmaThreads, kMmaSmem, expected, held, &cluster);
  if (e != cudaSuccess) return e;
  const uint32_t step = std::max(mma_step1((a.max_rank + 15) / 16),
                                 mma_step2(a.y.data != nullptr, RB, block_columns(a.y_dtype == MOE_DTYPE_F32,
                                                                                  a.out_dtype == MOE_DTYPE_F32)));
  const bool over_y = out_over_y(a, RB);
  const uint32_t rest = 1024 + mma_fixed(over_y, RB), ring = std::min(mma_ring(over_y, RB), kMmaMaxStages * step);
  return lora_launch_cluster(lora_mma_kernel<RB>, tiles, cluster, kMmaThreads, 2 * ring + rest, true, s, a, p, ring);
}

}  // namespace

bool lora_mma_takes(const moe_lora_args& a) { return a.max_rank <= 64 || a.out_dtype == MOE_DTYPE_BF16; }

cudaError_t launch_lora_mma(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, int32_t expected, cudaStream_t s) {
  return a.max_rank <= 64 ? lora_mma_launch<1>(a, p, tiles, expected, s) : lora_mma_launch<2>(a, p, tiles, expected, s);
}

cudaError_t lora_device_flags(int32_t* flags) {
  cudaError_t e = cudaDeviceSynchronize();
  int32_t mine = 0;
  if (e == cudaSuccess) e = lora_small_flags(flags);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&mine, g_lora_flags, sizeof(int32_t));
  const int32_t zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_lora_flags, &zero, sizeof(int32_t));
  if (e == cudaSuccess) *flags |= mine;
  return e;
}

}  // namespace moe
