// router.cuh -- how one warp routes one token (router.cu, layer.cu).
#pragma once

#include "common.cuh"

namespace moe {

// Unsigned key with the order of the fp32 value (after -0 -> +0, so that
// equal values compare equal as in the float comparison).
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Lane l's biased logits z[l + 32 i], i < SLOTS, of one token.
template <int SLOTS>
__device__ __forceinline__ void load_token(const float* __restrict__ row, const float* __restrict__ bias, int32_t E,
                                           int lane, float (&z)[SLOTS]) {
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int32_t e = lane + 32 * i;
    z[i] = 0.f;
    if (e < E) z[i] = bias ? __ldg(row + e) + __ldg(bias + e) : __ldg(row + e);
  }
}

// One warp routes one token from its loaded logits.  Each pick is the expert
// with the largest key among those not yet taken, equal keys taken lower index
// first (a max then a min over the warp).
template <int SLOTS>
__device__ __forceinline__ void route_token(const float (&z)[SLOTS], int32_t E, int32_t k, int lane,
                                            int32_t* __restrict__ ids_t, float* __restrict__ w_t, int32_t* s_hist) {
  uint32_t key[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) key[i] = lane + 32 * i < E ? order_key(z[i]) : 0u;  // 0: below every real key
  uint32_t taken = 0;
  float my_z = 0.f, z0 = 0.f;
  int32_t my_e = 0;
  for (int32_t j = 0; j < k; ++j) {
    uint32_t bk = 0u;
    int32_t be = 0x7fffffff;
    float bz = 0.f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int32_t e = lane + 32 * i;
      if (e < E && !(taken & (1u << i)) && (be == 0x7fffffff || key[i] > bk)) {
        bk = key[i];
        be = e;
        bz = z[i];
      }
    }
    const uint32_t gk = __reduce_max_sync(0xffffffffu, bk);
    const int32_t ge = (int32_t)__reduce_min_sync(0xffffffffu, (be != 0x7fffffff && bk == gk) ? (uint32_t)be
                                                                                               : 0x7fffffffu);
    const float gz = __shfl_sync(0xffffffffu, bz, ge & 31);
    if ((ge & 31) == lane) taken |= 1u << (ge >> 5);
    if (j == 0) z0 = gz;
    if (lane == j) {
      my_z = gz;
      my_e = ge;
    }
  }
  const float ex = lane < k ? expf(my_z - z0) : 0.f;
  float sum = ex;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane < k) {
    ids_t[lane] = my_e;
    w_t[lane] = ex / sum;
    if (s_hist) atomicAdd(&s_hist[my_e], 1);
  }
}

}  // namespace moe
