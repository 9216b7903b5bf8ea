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

// v of the lane n places around the lane's row of 16 (a DPP operand, no LDS).
template <int n, typename V>
__device__ __forceinline__ V row_ror(V v) {
  static_assert(sizeof(V) == 4, "one register");
  return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + n, 0xf, 0xf, false));
}

// v of the lane n places before, 0 before the row's first lane.
template <int n>
__device__ __forceinline__ int row_shr(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x110 + n, 0xf, 0xf, false);
}

// Reductions over aligned runs of G = 16 or 64 lanes; every lane of the run ends
// with the same bits.  Within a row of 16 by rotations, whose pairs are
// combined commutatively step by step; the four rows through lanes 0, 16, 32,
// 48 in order.
template <int G, typename V, typename Op>
__device__ __forceinline__ V run_reduce(V v, Op op) {
  static_assert(G == 16 || G == 64, "a row or a wave");
  v = op(v, row_ror<8>(v));
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  v = op(v, row_ror<1>(v));
  if constexpr (G == 64) {
    auto lane = [&](int l) { return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
    v = op(op(lane(0), lane(16)), op(lane(32), lane(48)));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float run_sum(float v) {
  return run_reduce<G>(v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ int run_sumi(int v) {
  return run_reduce<G>(v, [](int a, int b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float run_maxf(float v) {
  return run_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float run_minf(float v) {
  return run_reduce<G>(v, [](float a, float b) { return fminf(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t run_maxu(uint32_t v) {
  return run_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t run_minu(uint32_t v) {
  return run_reduce<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t run_or(uint32_t v) {
  return run_reduce<G>(v, [](uint32_t a, uint32_t b) { return a | b; });
}

}  // namespace moe
