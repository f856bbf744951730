// lora_mma.cu -- the adapters for batches that fill the GPU with tiles of 128
// tokens: one CTA takes a tile through both products on the tensor cores'
// asynchronous path (tcgen05, accumulators in tensor memory).
//
// Moving x, y and out bounds it.  Warp-level matrix instructions reread the
// adapter's matrices from shared memory for every 16 tokens, and at rank 64
// that and the instructions themselves took twice the time of the memory
// traffic; here one instruction takes 128 tokens, the operands go from shared
// memory to the tensor core without passing the warps, and the warps only copy
// and finish.
//
//   first product:  D1[128 tokens][ranks] += x chunk . A chunk^T, 64 columns of
//     in_features a step; a ring of steps filled by asynchronous copies (the
//     tokens' rows are gathered: 8 lanes copy 128 bytes of one).
//   v = scale D1 as a sum of two bf16 terms (three for an fp32 out), each
//     term a K-major operand in shared memory.
//   second product: D2[128][64 columns] = sum over terms of v . B rows^T, D2
//     twice, so that the warps add y to one block and write it out while the
//     tensor core works on the next.  y comes in and out leaves through shared
//     memory, so that both move in whole 128-byte lines.
#include "lora.cuh"

namespace moe {

namespace {

constexpr int kMmaTile = kMmaTokens;
constexpr uint32_t kOperandTile = 128 * 128;  // 128 rows of 64 bf16
constexpr int kMmaMaxStages = 6;
constexpr uint32_t kD2 = 128, kTmemCols = 256;  // tensor memory: D1 in columns 0..127, D2 in two halves of 64 after it

// Set where a bounded wait ran out; read by moe_lora_get_device_error.
__device__ int32_t g_lora_flags;

// Offset of 16-byte piece p of row r in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t p) { return r * 128 + ((p ^ (r & 7)) << 4); }

__host__ __device__ inline uint32_t mma_step1(int32_t ranks16) { return kOperandTile + (uint32_t)ranks16 * 16 * 128; }
// y (128 rows of 64 columns), then B (64 rows of up to 128 ranks)
__host__ __device__ inline uint32_t mma_step2(uint32_t y_size, int32_t rank_blocks) {
  return 128 * 64 * y_size + (uint32_t)rank_blocks * 64 * 128;
}

__global__ void __launch_bounds__(kLoraThreads, 1)
    lora_mma_kernel(const moe_lora_args a, const LoraPlan plan, int32_t terms, uint32_t ring_bytes) {
  extern __shared__ __align__(16) char sm_raw[];
  __shared__ int32_t row[kMmaTile];
  __shared__ __align__(8) uint64_t done1[kMmaMaxStages], done2[2];
  __shared__ uint32_t tmem_slot;
  char* sm = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kMmaMaxStages; ++s) mbar_init(&done1[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&done2[s], 1);
    fence_mbar_init();
  }
  Tile t;
  if (!planned_tile<kMmaTile>(a, plan, (int32_t)blockIdx.x, row, t)) return;
  if (warp == 0) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int32_t rank = t.rank, ranks16 = (rank + 15) / 16, rank_blocks = (a.max_rank + 63) / 64;
  const bool yf = a.y_dtype == MOE_DTYPE_F32, of = a.out_dtype == MOE_DTYPE_F32, has_y = a.y.data != nullptr;
  // ring; out block; v [terms][rank_blocks] operand tiles
  const uint32_t sm_u32 = smem_u32(sm);
  char* obuf = sm + ring_bytes;
  const uint32_t v_at = ring_bytes + 128 * 64 * (of ? 4 : 2);
  const uint32_t quadrant = (uint32_t)(32 * (warp & 3)) << 16;  // this warp's lanes of tensor memory
  const int m = 32 * (warp & 3) + lane;                         // its thread's token
  bool dead = false;  // a wait ran out
  const int p8 = tid & 7, r8 = tid >> 3;  // copies of 128-byte rows: piece, first row (+ 32, ...)

  if (rank > 0) {
    const char* A = reinterpret_cast<const char*>(a.a + (int64_t)t.adapter * a.max_rank * a.in_features);
    const uint32_t row_bytes = (uint32_t)a.in_features * 2, idesc = idesc_bf16(128, (uint32_t)ranks16 * 16);
    const int32_t chunks = (a.in_features + 63) / 64;
    const int64_t xs = (a.x.stride ? a.x.stride : a.in_features) * 2;
    const char* xr[4];  // (places past the tile's count: its first token, and their rows are not looked at)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t tok = row[r8 + 32 * i];
      xr[i] = static_cast<const char*>(a.x.data) + (int64_t)(tok >= 0 ? tok : row[0]) * xs;
    }
    const uint32_t step = mma_step1(ranks16);
    const int stages = (int)min((uint32_t)kMmaMaxStages, ring_bytes / step);
    // rows of A past the rank reach only columns of D1 that are not looked at
    const int32_t a_rows = min(16 * ranks16, a.max_rank);
    auto fetch = [&](int32_t c, int stage) {
      if (c < chunks) {
        const uint32_t off = (uint32_t)c * 128 + 16 * p8, at = stage * step;
        if (off < row_bytes) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ring16(sm_u32 + at + swizzled(r8 + 32 * i, p8), xr[i] + off);
          for (int32_t r = r8; r < a_rows; r += 32)
            ring16(sm_u32 + at + kOperandTile + swizzled(r, p8), A + (uint64_t)r * row_bytes + off);
        } else {  // past the row's end
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(sm + at + swizzled(r8 + 32 * i, p8)) = make_uint4(0, 0, 0, 0);
          for (int32_t r = r8; r < a_rows; r += 32)
            *reinterpret_cast<uint4*>(sm + at + kOperandTile + swizzled(r, p8)) = make_uint4(0, 0, 0, 0);
        }
      }
      ring_commit();
    };
    for (int s = 0; s + 1 < stages; ++s) fetch(s, s);
    int stage = 0, last = 0;
    uint32_t last_parity = 0, parity = 0;
    for (int32_t c = 0; c < chunks; ++c) {
      ring_wait(stages - 2);
      fence_proxy_async_smem();
      if (__syncthreads_or(dead)) {
        dead = true;
        break;
      }
      if (warp == 0) {
        if (elect_one()) {
          const uint32_t x_at = sm_u32 + stage * step, a_at = x_at + kOperandTile;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16(tmem, smem_desc_k128(x_at + 32 * k), smem_desc_k128(a_at + 32 * k), idesc, (c | k) != 0);
          tc_commit(&done1[stage]);
        }
        __syncwarp();
      }
      // the step before this one has been read: its slot takes the chunk `stages - 1` ahead
      if (c > 0 && !mbar_wait(&done1[last], last_parity, &g_lora_flags)) dead = true;
      fetch(c + stages - 1, stage == 0 ? stages - 1 : stage - 1);
      last = stage;
      last_parity = parity;
      if (++stage == stages) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (!dead && !mbar_wait(&done1[last], last_parity, &g_lora_flags)) dead = true;
    ring_wait(0);
    dead = __syncthreads_or(dead);
    tc_fence_after();
    // D1 -> v: a thread its token's 16 ranks at a time
    if (!dead)
      for (int32_t j = warp >> 2; j < ranks16; j += 2) {
        uint32_t d[16];
        tmem_ld16(tmem + quadrant + 16 * j, d);
        tmem_ld_wait();
        float s[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 16 * j + i < rank ? __uint_as_float(d[i]) * t.scale : 0.f;
        for (int k = 0; k < terms; ++k) {  // s = a sum of bf16 terms, each the rounding of what is left
          const uint32_t tile = v_at + (uint32_t)(k * rank_blocks + j / 4) * kOperandTile;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float &lo = s[8 * h + 2 * i], &hi = s[8 * h + 2 * i + 1];
              o[i] = pack2(lo, hi);
              lo -= bf16lo(o[i]);
              hi -= bf16hi(o[i]);
            }
            *reinterpret_cast<uint4*>(sm + tile + swizzled(m, (j % 4) * 2 + h)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    tc_fence_before();
    fence_proxy_async_smem();
  }
  dead = __syncthreads_or(dead);
  tc_fence_after();

  // out = y + B v over blocks of 64 columns
  const uint32_t y_size = has_y ? (yf ? 4 : 2) : 0, y_bytes = 128 * 64 * y_size, idesc2 = idesc_bf16(128, 64);
  const uint32_t step = max(mma_step2(y_size, rank > 0 ? rank_blocks : 0), 1024u);
  const int stages = (int)min(4u, ring_bytes / step);
  const char* B = reinterpret_cast<const char*>(a.b) + (rank > 0 ? (int64_t)t.adapter * a.out_features * a.max_rank * 2 : 0);
  const uint32_t b_bytes = (uint32_t)a.max_rank * 2;
  const int64_t ys = (a.y.stride ? a.y.stride : a.out_features) * y_size;
  const int32_t blocks = (a.out_features + 63) / 64;
  auto fetch = [&](int32_t ob, int stage) {
    if (ob < blocks) {
      const uint32_t at = stage * step;
      const int32_t left = a.out_features - ob * 64;
      if (has_y && !yf) {
        if (8 * p8 < left)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t r = r8 + 32 * i, tok = row[r];
            if (tok >= 0)
              ring16(sm_u32 + at + swizzled(r, p8),
                     static_cast<const char*>(a.y.data) + (int64_t)tok * ys + (uint32_t)(ob * 64 + 8 * p8) * 2);
          }
      } else if (has_y) {
        const int p = tid & 15;
        if (4 * p < left)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int32_t r = (tid >> 4) + 16 * i, tok = row[r];
            if (tok >= 0)
              ring16(sm_u32 + at + r * 256 + ((p ^ (r & 7)) << 4),
                     static_cast<const char*>(a.y.data) + (int64_t)tok * ys + (uint32_t)(ob * 64 + 4 * p) * 4);
          }
      }
      const char* src = B + (uint64_t)((uint32_t)ob * 64) * b_bytes;
      for (int32_t k = 0; 64 * k < 16 * ranks16; ++k) {
        const int32_t rest = rank - (64 * k + 8 * p8);  // ranks in this thread's piece and after it
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int32_t o = r8 + 32 * i;
          const uint32_t to = at + y_bytes + k * 64 * 128 + swizzled(o, p8);
          const char* from = src + (uint32_t)o * b_bytes + 128 * k + 16 * p8;
          if (rest <= 0) {
            *reinterpret_cast<uint4*>(sm + to) = make_uint4(0, 0, 0, 0);
          } else if (o < left) {
            if (rest >= 8) {
              ring16(sm_u32 + to, from);
            } else {  // what lies beyond the rank may hold anything
              uint4 b = __ldg(reinterpret_cast<const uint4*>(from));
              b.x &= rest >= 2 ? 0xffffffffu : 0xffffu;
              b.y &= rest >= 4 ? 0xffffffffu : rest == 3 ? 0xffffu : 0u;
              b.z &= rest >= 6 ? 0xffffffffu : rest == 5 ? 0xffffu : 0u;
              b.w &= rest == 7 ? 0xffffu : 0u;
              *reinterpret_cast<uint4*>(sm + to) = b;
            }
          }
        }
      }
    }
    ring_commit();
  };
  // adds y to block ob (in ring step `stage`, D2 half ob & 1) into the out block
  auto finish = [&](int32_t ob, int stage) {
    const uint32_t half = (uint32_t)(warp >> 2);  // this warp's 32 of the 64 columns
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t d[16];
      if (rank > 0) {
        tmem_ld16(tmem + quadrant + kD2 + (ob & 1) * 64 + half * 32 + g * 16, d);
        tmem_ld_wait();
      }
      float r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = rank > 0 ? __uint_as_float(d[i]) : 0.f;
      const uint32_t first = half * 32 + g * 16;  // column in the block
      if (has_y && yf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 y = slot16(sm, stage * step + m * 256 + (((first / 4 + i) ^ (m & 7)) << 4));
          r[4 * i] += __uint_as_float(y.x);
          r[4 * i + 1] += __uint_as_float(y.y);
          r[4 * i + 2] += __uint_as_float(y.z);
          r[4 * i + 3] += __uint_as_float(y.w);
        }
      } else if (has_y) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float y[8];
          unpack8(slot16(sm, stage * step + swizzled(m, first / 8 + i)), y);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[8 * i + j] += y[j];
        }
      }
      if (of) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(obuf + m * 256 + (((first / 4 + i) ^ (m & 7)) << 4)) =
              make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<uint4*>(obuf + swizzled(m, first / 8 + i)) =
              make_uint4(pack2(r[8 * i], r[8 * i + 1]), pack2(r[8 * i + 2], r[8 * i + 3]),
                         pack2(r[8 * i + 4], r[8 * i + 5]), pack2(r[8 * i + 6], r[8 * i + 7]));
      }
    }
    tc_fence_before();
  };
  // the out block to memory, whole lines at a time
  auto write_out = [&](int32_t ob) {
    const int32_t left = a.out_features - ob * 64;
    const int64_t os = a.out.stride ? a.out.stride : a.out_features;
    if (!of) {
      if (8 * p8 < left)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t r = r8 + 32 * i, tok = row[r];
          if (tok >= 0)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out.data) + (int64_t)tok * os + ob * 64 + 8 * p8) =
                *reinterpret_cast<const uint4*>(obuf + swizzled(r, p8));
        }
    } else {
      const int p = tid & 15;
      if (4 * p < left)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t r = (tid >> 4) + 16 * i, tok = row[r];
          if (tok >= 0)
            *reinterpret_cast<uint4*>(static_cast<float*>(a.out.data) + (int64_t)tok * os + ob * 64 + 4 * p) =
                *reinterpret_cast<const uint4*>(obuf + r * 256 + ((p ^ (r & 7)) << 4));
        }
    }
  };
  if (!dead)
    for (int s = 0; s + 2 < stages; ++s) fetch(s, s);
  int stage = 0, before = 0;
  // pass ob starts block ob on the tensor core and finishes block ob - 1
  for (int32_t ob = 0; !dead && ob <= blocks; ++ob) {
    fetch(ob + stages - 2, stage + stages - 2 < stages ? stage + stages - 2 : stage - 2);
    ring_wait(stages - 2);
    fence_proxy_async_smem();
    if (__syncthreads_or(dead)) {  // block ob has landed, and the out block has been written out
      dead = true;
      break;
    }
    if (rank > 0 && ob < blocks && warp == 0) {
      tc_fence_after();
      if (elect_one()) {
        const uint32_t b_at = sm_u32 + stage * step + y_bytes;
        for (int k = 0; k < terms; ++k)
          for (int32_t j = 0; j < ranks16; ++j)
            tc_mma_bf16(tmem + kD2 + (ob & 1) * 64,
                        smem_desc_k128(sm_u32 + v_at + (uint32_t)(k * rank_blocks + j / 4) * kOperandTile + (j % 4) * 32),
                        smem_desc_k128(b_at + (uint32_t)(j / 4) * 64 * 128 + (j % 4) * 32), idesc2, (k | j) != 0);
        tc_commit(&done2[ob & 1]);
      }
      __syncwarp();
    }
    if (ob > 0) {
      if (rank > 0) {
        if (!mbar_wait(&done2[(ob - 1) & 1], ((ob - 1) >> 1) & 1, &g_lora_flags)) dead = true;
        __syncwarp();
        tc_fence_after();
      }
      finish(ob - 1, before);
      if (__syncthreads_or(dead)) {
        dead = true;
        break;
      }
      write_out(ob - 1);
    }
    before = stage;
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  ring_wait(0);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_lora_mma(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, cudaStream_t s) {
  const int32_t terms = a.out_dtype == MOE_DTYPE_BF16 ? 2 : 3;
  const int32_t rank_blocks = (a.max_rank + 63) / 64;
  const uint32_t y_size = !a.y.data ? 0 : a.y_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const uint32_t rest = 1024 + 128 * 64 * (a.out_dtype == MOE_DTYPE_F32 ? 4 : 2) + terms * rank_blocks * kOperandTile;
  const uint32_t room = 225 * 1024 - rest;
  const uint32_t step1 = mma_step1((a.max_rank + 15) / 16), step2 = std::max(mma_step2(y_size, rank_blocks), 1024u);
  const uint32_t ring = std::min(room, std::max(kMmaMaxStages * step1, 4 * step2)) / 1024 * 1024;
  static std::atomic<bool> configured[kMaxDevices];
  const cudaError_t e = raise_smem_limit(lora_mma_kernel, 225 * 1024, configured);
  if (e != cudaSuccess) return e;
  return launch_ex(lora_mma_kernel, dim3((unsigned)tiles), dim3(kLoraThreads), ring + rest, s, true, a, p, terms, ring);
}

bool lora_mma_fits(const moe_lora_args& a) {
  const uint32_t y_size = !a.y.data ? 0 : a.y_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const int32_t terms = a.out_dtype == MOE_DTYPE_BF16 ? 2 : 3, rank_blocks = (a.max_rank + 63) / 64;
  const uint32_t rest = 1024 + 128 * 64 * (a.out_dtype == MOE_DTYPE_F32 ? 4 : 2) + terms * rank_blocks * kOperandTile;
  return rest + 3 * mma_step2(y_size, rank_blocks) <= 225 * 1024 && rest + 3 * mma_step1((a.max_rank + 15) / 16) <= 225 * 1024;
}

cudaError_t lora_device_flags(int32_t* flags) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(flags, g_lora_flags, sizeof(int32_t));
  const int32_t zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_lora_flags, &zero, sizeof(int32_t));
  return e;
}

}  // namespace moe
