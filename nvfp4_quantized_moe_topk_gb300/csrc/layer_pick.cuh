// layer_pick.cuh -- a token's experts of the whole-layer call, by a warp (layer.cu, layer_few.cu).
#pragma once

#include "kernels.h"
#include "router.cuh"

namespace moe {

// One token's picks: k of the logits, then the shared experts.
// (ids, w: the token's; out: write the caller's too.)
template <int SLOTS>
__device__ __forceinline__ void pick_token(const LayerPick& a, int32_t t, int lane, int32_t* ids, float* w, bool out) {
  float z[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int32_t e = lane + 32 * i;
    z[i] = 0.f;
    if (e < a.E) z[i] = __ldcg(a.logits + (int64_t)t * a.E + e) + (a.bias ? __ldg(a.bias + e) : 0.f);
  }
  route_token<SLOTS>(z, a.E, a.k, lane, ids, w, nullptr);
  __syncwarp();
  if (out && lane < a.k) {
    if (a.ids_out) a.ids_out[(int64_t)t * a.k + lane] = ids[lane];
    if (a.w_out) a.w_out[(int64_t)t * a.k + lane] = w[lane];
  }
  if (lane < a.shared) {
    const int32_t part = a.part_of ? t / kDecPassTok : 0, more = (a.n + kDecPassTok - 1) / kDecPassTok - 1;
    ids[a.k + lane] = part == 0 ? a.E + lane : a.E + a.shared + lane * more + part - 1;
    w[a.k + lane] = 1.f;
  }
}
__device__ __noinline__ inline void pick_any(const LayerPick& a, int32_t t, int lane, int32_t* ids, float* w, bool out) {
  if (a.E <= 64)
    pick_token<2>(a, t, lane, ids, w, out);
  else if (a.E <= 128)
    pick_token<4>(a, t, lane, ids, w, out);
  else if (a.E <= 256)
    pick_token<8>(a, t, lane, ids, w, out);
  else if (a.E <= 512)
    pick_token<16>(a, t, lane, ids, w, out);
  else
    pick_token<32>(a, t, lane, ids, w, out);
}

}  // namespace moe
