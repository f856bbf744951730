// tile.cuh -- the product of one NVFP4 fragment tile (decode.cu, layer_few.cu).
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cg_f32(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_cg_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int32_t atom_add_acq_rel_gpu(int32_t* p, int32_t v) {
  int32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
// One k-tile (16 rows x 64 k) of one row tile against this lane's activation
// fragments x0 (k 16t .. 16t+7) and x1 (k 16t+8 .. 16t+15) of token column g.
// c: the lane's codes; s0, s1: the scales of rows g and g + 8 (scale_bf16_2p118, both halves).
__device__ __forceinline__ void tile_mma(const uint4& c, uint32_t s0, uint32_t s1, const uint4& x0, const uint4& x1,
                                         float (&acc)[4], float (&acc2)[4]) {
  uint32_t r0, r1, r2, r3;  // row g
  uint32_t q0, q1, q2, q3;  // row g + 8
  // word 0 of each row: k blocks 0 and 1 of the MMA
  unpack_word(c.x, r0, r1, r2, r3);
  unpack_word(c.z, q0, q1, q2, q3);
  mma_bf16_16816(acc, mul_bf16x2(r0, s0), mul_bf16x2(q0, s1), mul_bf16x2(r1, s0), mul_bf16x2(q1, s1), x0.x, x0.y);
  mma_bf16_16816(acc2, mul_bf16x2(r2, s0), mul_bf16x2(q2, s1), mul_bf16x2(r3, s0), mul_bf16x2(q3, s1), x0.z, x0.w);
  // word 1 of each row: k blocks 2 and 3
  unpack_word(c.y, r0, r1, r2, r3);
  unpack_word(c.w, q0, q1, q2, q3);
  mma_bf16_16816(acc, mul_bf16x2(r0, s0), mul_bf16x2(q0, s1), mul_bf16x2(r1, s0), mul_bf16x2(q1, s1), x1.x, x1.y);
  mma_bf16_16816(acc2, mul_bf16x2(r2, s0), mul_bf16x2(q2, s1), mul_bf16x2(r3, s0), mul_bf16x2(q3, s1), x1.z, x1.w);
}

// The same from a tile in shared memory.
__device__ __forceinline__ void tile_mma(const uint8_t* tile, const uint4& x0, const uint4& x1, int lane,
                                         const uint32_t* scale_lut, float (&acc)[4], float (&acc2)[4]) {
  const int g = lane >> 2, t = lane & 3;
  tile_mma(*reinterpret_cast<const uint4*>(tile + 16 * lane), scale_lut[tile[512 + 4 * g + t]],
           scale_lut[tile[512 + 4 * (g + 8) + t]], x0, x1, acc, acc2);
}

}  // namespace moe
