// What the row operators (layer norm, RMS norm) share: a row read once and held in
// registers by W waves with C vectors of 16 bytes per lane, its sums, and the sum
// over the slabs that hold shares of the weights' gradients.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "moe_internal.h"
#include "wave_ops.hpp"

namespace moe {
namespace {

constexpr int kMaxSlabs = 1024;
constexpr unsigned kMaxRowGrid = 1u << 16;
// Waves over which the rows are spread: two per SIMD, what the registers of the
// backward pass allow.  65,536 x 2048 forward, backward and 8192 x 7168 backward
// take 90, 160 and 86 us so; 116, 165 and 92 with 1,024 waves, 97, 162 and 102
// with 4,096.
constexpr int kRowWaves = 2048;

// Sum over the work-group; every thread gets it.  `red` holds one float per wave.
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = run_sum<64>(v);
  __syncthreads();  // the previous sum's reads are done
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

// One lane's part of a row: C vectors of EPC elements, vector c at c * 64 W + its
// place in the row's lanes.  TAIL: the row's last vector is short, and the lane
// that holds it moves its elements one by one.
template <typename T, int W, int C, bool TAIL>
struct RowPart {
  static constexpr int EPC = Elem<T>::kPer16B, COLS = EPC * C;
  u32x4_t raw[C];

  __device__ __forceinline__ void load(const T* row, int place, int H) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
      raw[c] = u32x4_t{0u, 0u, 0u, 0u};
      if (at + EPC <= H) raw[c] = *reinterpret_cast<const u32x4_any_t*>(row + at);
    }
    if constexpr (TAIL) {
      const int last = H / EPC;  // the short vector
      if (last % (64 * W) == place) {
        float v[EPC];
#pragma unroll
        for (int e = 0; e < EPC; ++e) v[e] = last * EPC + e < H ? Elem<T>::to_f(row[last * EPC + e]) : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c == last / (64 * W)) raw[c] = pack16(v, T());
      }
    }
  }
  __device__ __forceinline__ void get(int c, float* v) const { unpack16(raw[c], v, T()); }
  // PAST: past L2, for rows that the call does not read again
  template <bool PAST = false>
  __device__ static __forceinline__ void put(T* row, int at, int H, const float* v) {
    if (at + EPC <= H) {
      const u32x4_any_t w = pack16(v, T());
      if constexpr (PAST)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any_t*>(row + at));
      else
        *reinterpret_cast<u32x4_any_t*>(row + at) = w;
    } else if constexpr (TAIL) {
#pragma unroll
      for (int e = 0; e < EPC; ++e)
        if (at + e < H) row[at + e] = Elem<T>::from_f(v[e]);
    }
  }
};

// A lane's columns of gamma or beta; 0 past the row's end and without p.
template <int EPC, int W, int C, bool TAIL>
__device__ __forceinline__ void load_cols(const float* p, int place, int H, float* out) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * 64 * W + place) * EPC;
#pragma unroll
    for (int e = 0; e < EPC; e += 4) {
      f32x4_t v{0.f, 0.f, 0.f, 0.f};
      if (p && at + e + 4 <= H) {
        v = *reinterpret_cast<const f32x4_any_t*>(p + at + e);
      } else if (TAIL && p) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
          if (at + e + f < H) v[f] = p[at + e + f];
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) out[c * EPC + e + f] = v[f];
    }
  }
}

// Sums over the W waves of a row (a work-group of W waves, or one wave); `red`
// alternates between two halves, so one barrier per sum is enough.
template <int W, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float (*red)[NV][16], int& half) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = run_sum<64>(v[i]);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) red[half][i][threadIdx.x >> 6] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[half][i][w];
      v[i] = s;
    }
    half ^= 1;
  }
}

// The next row's loads fly ahead, except where 16 waves leave each 128 registers.
template <int W>
constexpr bool kAhead = W < 16;
template <int W>
constexpr int kGroup = W == 1 ? kThreads : 64 * W;  // threads of a work-group

// Sums of the slabs' shares, `width` columns each: the first H to dgamma, the
// rest to dbeta; latency (5 us at 512 slabs of 2048 columns).  64 columns per work-group; wave w
// takes slabs w, w + 16, ... in order, then the waves' sums are added in order.
constexpr int kFoldWaves = 16;
__global__ __launch_bounds__(64 * kFoldWaves) void slab_fold_kernel(const float* __restrict__ part,
                                                                    int slabs, int width, int H,
                                                                    float* __restrict__ dgamma,
                                                                    float* __restrict__ dbeta) {
  __shared__ float red[kFoldWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < width) {
    const float* q = part + c;
#pragma unroll 8
    for (int p = w; p < slabs; p += kFoldWaves) s += q[(int64_t)p * width];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w != 0 || c >= width) return;
#pragma unroll
  for (int v = 1; v < kFoldWaves; ++v) s += red[v][lane];
  if (c < H)
    dgamma[c] = s;
  else if (dbeta)
    dbeta[c - H] = s;
}

// How a row is held: W waves, C vectors per lane.  The smallest W, then the
// smallest C, that hold it; at most four vectors per lane, which with gamma and
// two sums fills the registers of two waves per SIMD.  Two vectors a lane and
// twice the waves take 116, 156 and 86 us where these take 90, 160 and 86 (see
// kRowWaves).  W = 0: too wide.
struct Holding {
  int W, C;
};
Holding holding(int H, int dtype) {
  const int epc = 16 / elem_bytes(dtype);
  const int64_t vecs = ceil_div(H, epc);
  for (int W : {1, 2, 4, 8, 16})
    for (int C : {1, 2, 4})
      if ((W == 1 || C == 4) && (W < 16 || epc == 4) && vecs <= 64 * W * C) return {W, C};
  return {0, 0};
}
int rows_per_group(int W) { return W == 1 ? kThreads / 64 : 1; }
int waves_per_group(int W) { return W == 1 ? kThreads / 64 : W; }

// Work-groups of a pass over the rows.
int row_groups(int64_t N, int W) {
  if (W == 0) return (int)std::min<int64_t>(N, 512);
  return (int)std::min<int64_t>(ceil_div(N, rows_per_group(W)), std::max(256, kRowWaves / waves_per_group(W)));
}

// The backward pass's work-groups: each takes kSlabRounds rows a wave (a
// work-group of several waves a row) at least, since a slab of its own costs as
// much to write and fold as the rows to read: 794 x 7808 bf16 26 us with 4 rounds,
// 35 with 1, 30 with 8.  With one slab there is no fold's launch: calls on 16 x
// 512 fp32 13.7 us and 16.3 with one, on 4 x 4096 bf16 13.7 and 16.8.
constexpr int kSlabRounds = 4;
int slab_count(int64_t N, int W) {
  const int most = row_groups(N, W);
  return W == 0 ? most : (int)std::min<int64_t>(most, ceil_div(N, kSlabRounds * rows_per_group(W)));
}

// Calls f with the holding, and whether a row's last vector is short, as
// template arguments.
template <typename T, typename F>
void with_holding(const Holding& h, int H, F f) {
  constexpr int EPC = Elem<T>::kPer16B;
  using std::bool_constant;
  using std::integral_constant;
#define HOLDING_CASE(w, c)                                                                            \
  if (h.W == w && h.C == c) {                                                                      \
    if (H % EPC) return f(integral_constant<int, w>(), integral_constant<int, c>(), bool_constant<true>()); \
    return f(integral_constant<int, w>(), integral_constant<int, c>(), bool_constant<false>());     \
  }
  HOLDING_CASE(1, 1)
  HOLDING_CASE(1, 2)
  HOLDING_CASE(1, 4)
  HOLDING_CASE(2, 4)
  HOLDING_CASE(4, 4)
  HOLDING_CASE(8, 4)
  if constexpr (EPC == 4) {
    HOLDING_CASE(16, 4)
  }
#undef HOLDING_CASE
}

}  // namespace
}  // namespace moe
