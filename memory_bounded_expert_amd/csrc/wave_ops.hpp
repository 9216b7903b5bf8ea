// Wave-level helpers of the row operators (routing, layer norm, embedding,
// distillation): reductions over aligned runs of lanes and the ordering of a
// wave's own LDS traffic.
#pragma once

#include "device_common.hpp"

namespace moe {

// Orders one wave's LDS writes before its later LDS reads of other lanes' data
// (and those reads before later writes): the DS unit executes a wave's
// instructions in order, so waiting for this wave's own LDS operations and
// keeping the compiler from moving memory operations across is enough.
__device__ __forceinline__ void wave_lds_order() {
  constexpr int kWaitLgkm0 = 0xC07F;  // vmcnt 63, expcnt 7, lgkmcnt 0
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Reductions over aligned runs of G lanes by xor butterflies: commutative
// pairwise steps, so every lane of the run ends with the same bits.
template <int G>
__device__ __forceinline__ float run_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
template <int G, typename V>
__device__ __forceinline__ V run_sum64(V v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
template <int G, typename V>
__device__ __forceinline__ V run_max(V v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) {
    const V w = __shfl_xor(v, o);
    v = w > v ? w : v;
  }
  return v;
}
template <int G, typename V>
__device__ __forceinline__ V run_min(V v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) {
    const V w = __shfl_xor(v, o);
    v = w < v ? w : v;
  }
  return v;
}

}  // namespace moe
