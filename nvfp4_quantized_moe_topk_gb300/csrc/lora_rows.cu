// lora_rows.cu -- the adapters for many tokens of ranks above 64 with an fp32
// out: a CTA, or a cluster of CTAs, takes 64 tokens of one adapter through both
// products with warp matrix instructions.
//
// With 64 tokens a tile A and B are read once per 64 rows of x and y.  Warps
// are 4 groups of 16 tokens x 2 halves.  In the first product the halves take
// alternate 64-column chunks of in_features, in the second alternate 64-column
// blocks of out_features.  The four warps of a half share its chunk of A (or B)
// in shared memory, copied by all of them and met at one barrier a step; their
// own tokens' 16-byte pieces of x (or y) go through thread-private slots of the
// same ring steps.  Every 16 tokens reread A and B from shared memory, which at
// these ranks is what bounds it: 4096 tokens, 4096 to 4096, rank 128, fp32 y and
// out 104 us, 16384 380 on a GB300 (the bytes are 27 and 102).  It is not the
// faster way: lora_mma.cu, whose three terms of v fit beside two steps of 24 KB
// here too, takes 74 and 186 in a trial, and is still to take this case over.
//
// Shared rows of A, B and v are read as 16 bytes by lane (row g, piece q); rows
// whose pitch is a multiple of 128 bytes are stored with pieces 0-3 and 4-7
// swapped in odd rows, so that eight lanes touch all banks once.
#include "lora.cuh"

namespace moe {

namespace {

constexpr int kHalf = kLoraThreads / 2;
constexpr uint32_t kHalfVec = kHalf * 16;  // one 16-byte vector of every thread of a half

__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, %1;" ::"r"(half + 1), "n"(kHalf) : "memory");
}

// Bytes of a ring step: x and A; y and B.
__host__ __device__ inline uint32_t shrink_step(int32_t ranks8) { return 2 * (4 * kHalfVec + ranks8 * 8 * 128); }
__host__ __device__ inline uint32_t expand_step(int32_t ranks32, uint32_t y_vecs) {
  return 2 * (4 * y_vecs * kHalfVec + 64 * ranks32 * 64);
}
constexpr int kPass = 64, kPartPitch = kPass + 8;  // ranks of a pass of the first product; pitch of its sums

__global__ void __launch_bounds__(kLoraThreads, 2)
    lora_rows_kernel(const moe_lora_args a, const LoraPlan plan, uint32_t ring_bytes) {
  extern __shared__ __align__(128) char sm[];
  __shared__ int32_t row[kRowsTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int group = warp & 3, half = warp >> 2, htid = tid & (kHalf - 1);
  const uint32_t C = cluster_size(), cr = cluster_rank();
  Tile t;
  if (!planned_tile<kRowsTile>(a, plan, (int32_t)(blockIdx.x / C), row, t)) return;
  const int32_t rank = t.rank;
  const float scale = t.scale;
  // ring; v [kLoraTerms][64][VP] bf16; in a cluster the CTA's sums [64][kPartPitch].  Between the loops the ring holds
  // the halves' sums [2][64][kPartPitch].
  const int32_t kwins = (rank + 31) / 32;
  const uint32_t v_pitch = (uint32_t)((a.max_rank + 63) / 64) * 128;  // bytes
  const uint32_t sm_u32 = smem_u32(sm), v_at = ring_bytes;  // (offsets in sm; cp.async takes addresses)
  char* v_base = sm + ring_bytes;
  float* part = reinterpret_cast<float*>(sm);
  float* sum = reinterpret_cast<float*>(v_base + kLoraTerms * kRowsTile * v_pitch);
  int32_t tok[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) tok[h] = row[group * 16 + h * 8 + g];
  const int64_t t0 = tok[0] >= 0 ? tok[0] : row[0], t1 = tok[1] >= 0 ? tok[1] : row[0];  // (past the count: not stored)

  if (rank > 0) {
    const char* A = reinterpret_cast<const char*>(a.a + (int64_t)t.adapter * a.max_rank * a.in_features);
    const uint32_t row_bytes = (uint32_t)a.in_features * 2;
    const int64_t xs = (a.x.stride ? a.x.stride : a.in_features) * 2;
    const char* x0 = static_cast<const char*>(a.x.data) + t0 * xs + 16 * q;
    const char* x1 = static_cast<const char*>(a.x.data) + t1 * xs + 16 * q;
    const uint32_t first = (cr * 2 + half) * 128, jump = C * 256;  // byte offsets in a row of the half's chunks
    for (int32_t r0 = 0; r0 < rank; r0 += kPass) {
      const int32_t nt = min(kPass / 8, (rank - r0 + 15) / 16 * 2);  // groups of 8 ranks, in pairs
      const int32_t a_rows = min(8 * nt, a.max_rank - r0);  // rows past the rank reach only entries of v that are set to zero
      const uint32_t step = shrink_step(nt);
      const int stages = ring_stages(ring_bytes, step);
      const uint32_t a_at = 4 * kHalfVec;  // of the half's part of a step: x, then A
      // this thread's 16-byte piece of A: row ar + 16 i, piece ap
      const int32_t ar = htid >> 3, ap = htid & 7;
      const char* Ap = A + (uint64_t)(r0 + ar) * row_bytes + 16 * ap;
      const uint32_t a_to = a_at + ar * 128 + ((ap ^ ((ar & 1) << 2)) * 16);
      auto fetch = [&](uint32_t off, int stage) {
        if (off < row_bytes) {
          const uint32_t at = stage * step + half * (step / 2);
          const uint32_t slot = at + htid * 16;
          if (off + 16 * q < row_bytes) {
            ring16(sm_u32 + slot, x0 + off);
            ring16(sm_u32 + slot + kHalfVec, x1 + off);
          }
          if (off + 64 + 16 * q < row_bytes) {
            ring16(sm_u32 + slot + 2 * kHalfVec, x0 + off + 64);
            ring16(sm_u32 + slot + 3 * kHalfVec, x1 + off + 64);
          }
          if (off + 16 * ap < row_bytes) {
            const char* src = Ap + off;
#pragma unroll
            for (int i = 0; i < kPass / 16; ++i)
              if (ar + 16 * i < a_rows) ring16(sm_u32 + at + a_to + i * 16 * 128, src + (uint64_t)(16 * i) * row_bytes);
          }
        }
        ring_commit();
      };
      float acc[kPass / 8][4] = {};
      for (int s = 0; s + 1 < stages; ++s) fetch(first + s * jump, s);
      int stage = 0;
      for (uint32_t off = first; off < row_bytes; off += jump) {
        ring_wait(stages - 2);
        half_barrier(half);  // the step is there for all, and the one before has been read
        fetch(off + (stages - 1) * jump, stage == 0 ? stages - 1 : stage - 1);
        __syncwarp();
        const uint32_t at = stage * step + half * (step / 2);
        const bool tail = off + 128 > row_bytes;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint4 xa0 = slot16(sm, at + htid * 16 + (2 * w) * kHalfVec), xa1 = slot16(sm, at + htid * 16 + (2 * w + 1) * kHalfVec);
          const bool past = tail && off + 64 * w + 16 * q >= row_bytes;
          if (past) xa0 = xa1 = make_uint4(0, 0, 0, 0);
          const uint32_t from = at + a_at + g * 128 + (((w * 4 + q) ^ ((g & 1) << 2)) * 16);
#pragma unroll
          for (int j = 0; j < kPass / 8; j += 2) {
            if (j >= nt) break;
            uint4 b0 = slot16(sm, from + j * 1024), b1 = slot16(sm, from + (j + 1) * 1024);
            if (past) b0 = b1 = make_uint4(0, 0, 0, 0);
            mma_bf16(acc[j], xa0.x, xa1.x, xa0.y, xa1.y, b0.x, b0.y);
            mma_bf16(acc[j + 1], xa0.x, xa1.x, xa0.y, xa1.y, b1.x, b1.y);
            mma_bf16(acc[j], xa0.z, xa1.z, xa0.w, xa1.w, b0.z, b0.w);
            mma_bf16(acc[j + 1], xa0.z, xa1.z, xa0.w, xa1.w, b1.z, b1.w);
          }
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
      }
      ring_wait(0);
      __syncthreads();  // the ring becomes the halves' sums
#pragma unroll
      for (int j = 0; j < kPass / 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(part + (half * kRowsTile + group * 16 + h * 8 + g) * kPartPitch + 8 * j + 2 * q) =
              make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
      __syncthreads();
      // thread: two ranks of rows warp, warp + 8, ...
      constexpr int kRows = kRowsTile / kLoraWarps;
      const int32_t r = 2 * lane;
      const bool used = r0 + r < rank;
      float2 s[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float* p = part + (warp + i * kLoraWarps) * kPartPitch + r;
        const float2 p0 = *reinterpret_cast<const float2*>(p);
        const float2 p1 = *reinterpret_cast<const float2*>(p + kRowsTile * kPartPitch);
        s[i] = make_float2(p0.x + p1.x, p0.y + p1.y);
      }
      if (C > 1) {
        if (used) {
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            *reinterpret_cast<float2*>(sum + (warp + i * kLoraWarps) * kPartPitch + r) = s[i];
        }
        cluster_sync();
        // added in the order of the cluster's CTAs, the same in each of them
#pragma unroll
        for (int i = 0; i < kRows; ++i) s[i] = make_float2(0.f, 0.f);
        for (uint32_t k = 0; used && k < C; ++k) {
          float2 p[kRows];
#pragma unroll
          for (int i = 0; i < kRows; ++i) p[i] = peer_float2(sum + (warp + i * kLoraWarps) * kPartPitch + r, k);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            s[i].x += p[i].x;
            s[i].y += p[i].y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = warp + i * kLoraWarps;
        float s0 = used ? s[i].x * scale : 0.f, s1 = r0 + r + 1 < rank ? s[i].y * scale : 0.f;
        char* to = v_base + m * v_pitch + (uint32_t)(r0 / kPass) * 128 + (((lane >> 2) ^ ((m & 1) << 2)) * 16) +
                   (lane & 3) * 4;
        for (int k = 0; k < kLoraTerms; ++k, to += kRowsTile * v_pitch)
          *reinterpret_cast<uint32_t*>(to) = take_terms(s0, s1);
      }
      if (C > 1)
        cluster_sync();  // the peers have read this CTA's sums
      else
        __syncthreads();
    }
  }

  // out = y + B v over blocks of 64 columns.  A lane's columns of each 32: 4 at c0 and 4 at c0 + next.
  const bool quads = a.y_dtype == MOE_DTYPE_F32 || a.out_dtype == MOE_DTYPE_F32;
  const bool yf = a.y_dtype == MOE_DTYPE_F32, has_y = a.y.data != nullptr;
  const int32_t lc = quads ? 4 : 8, next = quads ? 16 : 4;
  const uint32_t y_vecs = !has_y ? 0 : yf ? 2 : 1, y_size = yf ? 4 : 2;
  const char* B = reinterpret_cast<const char*>(a.b) + (rank > 0 ? (int64_t)t.adapter * a.out_features * a.max_rank * 2 : 0);
  const uint32_t b_bytes = (uint32_t)a.max_rank * 2, b_pitch = kwins * 64;  // of a row: in the bank, in shared memory
  const uint32_t swap = b_pitch % 128 == 0 ? 4 : 0;
  const int64_t ys = (a.y.stride ? a.y.stride : a.out_features) * y_size;
  const char* y0 = static_cast<const char*>(a.y.data) + t0 * ys + lc * q * y_size;
  const char* y1 = static_cast<const char*>(a.y.data) + t1 * ys + lc * q * y_size;
  const uint32_t step = max(expand_step(kwins, y_vecs), 32u);
  const int stages = ring_stages(ring_bytes, step);
  const bool odd_rank = rank & 7;  // its last 16-byte piece of B is masked where it is read
  const int32_t blocks = (a.out_features + 63) / 64, b0 = (int32_t)cr * 2 + half, bstep = (int32_t)C * 2;
  auto fetch = [&](int32_t ob, int stage) {
    if (ob < blocks) {
      const uint32_t at = stage * step + half * (step / 2);
      const int32_t left = a.out_features - ob * 64;
      if (has_y) {
        uint32_t slot = at + htid * 16;
        const uint32_t e = (uint32_t)ob * 64 * y_size;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const bool in0 = w * 32 + lc * q < left, in1 = w * 32 + lc * q + next < left;
          const uint32_t ew = e + w * 32 * y_size;
          if (yf) {
            if (in0) {
              ring16(sm_u32 + slot, y0 + ew);
              ring16(sm_u32 + slot + 2 * kHalfVec, y1 + ew);
            }
            if (in1) {
              ring16(sm_u32 + slot + kHalfVec, y0 + ew + 64);
              ring16(sm_u32 + slot + 3 * kHalfVec, y1 + ew + 64);
            }
          } else if (quads) {
            if (in0) {
              ring8(sm_u32 + slot, y0 + ew);
              ring8(sm_u32 + slot + kHalfVec, y1 + ew);
            }
            if (in1) {
              ring8(sm_u32 + slot + 8, y0 + ew + 32);
              ring8(sm_u32 + slot + kHalfVec + 8, y1 + ew + 32);
            }
          } else if (in0) {
            ring16(sm_u32 + slot, y0 + ew);
            ring16(sm_u32 + slot + kHalfVec, y1 + ew);
          }
          slot += 2 * y_vecs * kHalfVec;
        }
      }
      const uint32_t b_at = at + 4 * y_vecs * kHalfVec;
      const char* src = B + (uint64_t)((uint32_t)ob * 64) * b_bytes;
      for (int32_t k = 0; k < kwins; ++k) {
        const int32_t p = k * 4 + (htid & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int32_t o = (htid >> 2) + 32 * i;
          const uint32_t to = b_at + o * b_pitch + ((p ^ ((o & 1) * swap)) * 16);
          if (8 * p >= rank)  // what lies beyond the rank may hold anything
            *reinterpret_cast<uint4*>(sm + to) = make_uint4(0, 0, 0, 0);
          else if (o < left)
            ring16(sm_u32 + to, src + o * b_bytes + 16 * p);
        }
      }
    }
    ring_commit();
  };
  for (int s = 0; s + 1 < stages; ++s) fetch(b0 + s * bstep, s);
  int stage = 0;
  for (int32_t ob = b0; ob < blocks; ob += bstep) {
    ring_wait(stages - 2);
    half_barrier(half);
    fetch(ob + (stages - 1) * bstep, stage == 0 ? stages - 1 : stage - 1);
    const uint32_t at = stage * step + half * (step / 2);
    const uint32_t b_at = at + 4 * y_vecs * kHalfVec;
    float acc[2][4][4] = {};
    for (int32_t k = 0; k < kwins; ++k) {
      uint4 bv[2][4];
      const int32_t left = rank - (k * 32 + 8 * q);
      const uint32_t from = b_at + ((g >> 1) * lc + (g & 1)) * b_pitch + (((k * 4 + q) ^ ((g & 1) * swap)) * 16);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bv[w][j] = slot16(sm, from + (w * 32 + (j >> 1) * next + 2 * (j & 1)) * b_pitch);
          if (odd_rank && left < 8) {
            bv[w][j].x &= left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
            bv[w][j].y &= left >= 4 ? 0xffffffffu : left == 3 ? 0xffffu : 0u;
            bv[w][j].z &= left >= 6 ? 0xffffffffu : left == 5 ? 0xffffu : 0u;
            bv[w][j].w &= left == 7 ? 0xffffu : 0u;
          }
        }
      const uint32_t vp = v_at + (group * 16 + g) * v_pitch + (k / 2) * 128 + ((((k & 1) * 4 + q) ^ ((g & 1) << 2)) * 16);
      for (int i = 0; i < kLoraTerms; ++i) {
        const uint4 lo = slot16(sm, vp + i * kRowsTile * v_pitch), hi = slot16(sm, vp + (i * kRowsTile + 8) * v_pitch);
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_bf16(acc[w][j], lo.x, hi.x, lo.y, hi.y, bv[w][j].x, bv[w][j].y);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_bf16(acc[w][j], lo.z, hi.z, lo.w, hi.w, bv[w][j].z, bv[w][j].w);
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int32_t c = ob * 64 + w * 32 + lc * q;
      const bool in0 = c < a.out_features, in1 = c + next < a.out_features;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tok[h] < 0 || !in0) continue;
        float r[8] = {};
        if (has_y) {
          const uint32_t ya = at + htid * 16 + (2 * w + h) * y_vecs * kHalfVec;
          const uint4 d = slot16(sm, ya);
          if (yf) {
            const uint4 e = slot16(sm, ya + kHalfVec);
            r[0] = __uint_as_float(d.x);
            r[1] = __uint_as_float(d.y);
            r[2] = __uint_as_float(d.z);
            r[3] = __uint_as_float(d.w);
            r[4] = __uint_as_float(e.x);
            r[5] = __uint_as_float(e.y);
            r[6] = __uint_as_float(e.z);
            r[7] = __uint_as_float(e.w);
          } else {
            unpack8(d, r);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[2 * j] += acc[w][j][2 * h];
          r[2 * j + 1] += acc[w][j][2 * h + 1];
        }
        if (a.out_dtype == MOE_DTYPE_F32) {
          float* p = row_ptr<float>(a.out, tok[h], a.out_features) + c;
          *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
          if (in1) *reinterpret_cast<float4*>(p + next) = make_float4(r[4], r[5], r[6], r[7]);
        } else {
          uint16_t* p = row_ptr<uint16_t>(a.out, tok[h], a.out_features) + c;
          if (!quads) {
            store8(p, r);
          } else {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack2(r[0], r[1]), pack2(r[2], r[3]));
            if (in1) *reinterpret_cast<uint2*>(p + next) = make_uint2(pack2(r[4], r[5]), pack2(r[6], r[7]));
          }
        }
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
}

}  // namespace

cudaError_t launch_lora_rows(const moe_lora_args& a, const LoraPlan& p, int32_t tiles, int32_t expected, cudaStream_t s) {
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = raise_smem_limit(lora_rows_kernel, 225 * 1024, configured);
  if (e != cudaSuccess) return e;
  static std::atomic<int32_t> held[kMaxDevices][kLoraMaxCluster + 1];
  int32_t cluster = 1;
  e = lora_cluster(lora_rows_kernel, kLoraThreads, 225 * 1024, expected, held, &cluster);
  if (e != cudaSuccess) return e;
  const uint32_t y_vecs = !a.y.data ? 0 : a.y_dtype == MOE_DTYPE_F32 ? 2 : 1;
  const uint32_t rest = kLoraTerms * kRowsTile * ((a.max_rank + 63) / 64) * 128 +
                        (cluster > 1 ? kRowsTile * kPartPitch * 4 : 0);
  // up to four ring steps, at least two: without a cluster as many as let two CTAs share an SM if those are two or
  // more, else as many as fit one
  const uint32_t step = std::max(shrink_step(std::min(a.max_rank, kPass) / 8), expand_step((a.max_rank + 31) / 32, y_vecs));
  const uint32_t two = 112 * 1024, one = 224 * 1024;
  uint32_t ring = std::min(4 * step, (cluster == 1 && rest + 2 * step <= two ? two : one) - rest);
  ring = std::max<uint32_t>(ring, 2 * kRowsTile * kPartPitch * 4) / 128 * 128;
  return lora_launch_cluster(lora_rows_kernel, tiles, cluster, kLoraThreads, ring + rest, true, s, a, p, ring);
}

}  // namespace moe
