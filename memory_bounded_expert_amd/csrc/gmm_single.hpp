// The 8-bit grouped product of a few rows: Y[row][n] = sum_k X[row][k] W[e][n][k], a
// row's dot products without matrix instructions.
//
// What there is to do is read the weights once.  A wave has kSingleCols neighbouring columns
// of one row: 1 KiB of each at a time, 16 numbers a lane, U of them in flight.  A
// lane's 16 products are added up in fp32 (each is exact there) before their block's
// two powers of two multiply the sum, and the lanes' sums meet at the end, in an order
// of their own.  No part of k is another work-group's: one launch, no workspace.  1 x
// 7168 x 2048 takes 6.1 us a call in a graph, 2.4 TB/s: the time is latency, of the
// offsets, then of two rounds of loads.
#pragma once

#include "gmm_common.hpp"

namespace moe {
namespace gmm {

constexpr int kSingleCols = 2;  // of a wave (4: 1 x 7168 x 2048 7.4 us for 6.3; 1: 16,384 columns 10.1 for 9.6)

template <int U>
__global__ __launch_bounds__(kThreads) void gmm_single_kernel(const Args p) {
  constexpr int COLS = kSingleCols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // a block of columns runs for all rows on one XCD, whose L2 then holds its weights
  const int slot = (int)blockIdx.x >> 3, block = slot / p.R * 8 + ((int)blockIdx.x & 7), row = slot % p.R;
  const int n0 = (block * (kThreads / 64) + wave) * COLS;
  if (n0 >= p.N) return;
  int e = -1;
  for (int set = 0; set * 64 < p.E && e < 0; ++set) {
    const Segment s = segment(p.offsets, min(set * 64 + lane, p.E - 1), p.R);
    const unsigned long long has = __ballot(set * 64 + lane < p.E && s.lo <= row && row < s.hi);
    if (has) e = set * 64 + __ffsll((long long)has) - 1;
  }
  if (e < 0) return;  // a row of no expert
  const int kp = q8_row_pitch(p.K), sp = q8_scale_pitch(p.K);
  const unsigned char* x = (const unsigned char*)p.A + (int64_t)row * kp;
  const unsigned char* w = (const unsigned char*)p.B + ((int64_t)e * p.N + n0) * kp;
  const unsigned char* xs = (const unsigned char*)p.As + (int64_t)row * sp;
  const unsigned char* ws = (const unsigned char*)p.Bs + ((int64_t)e * q8_blocks(p.N) + n0 / kQBlock) * sp;
  float acc[COLS] = {};
  for (int k0 = 0; k0 < kp; k0 += U * 1024) {
    u32x4_t xq[U], wq[U][COLS];
    int xb[U], wb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 1024 + lane * 16;
      xq[u] = u32x4_t{0, 0, 0, 0};
      xb[u] = wb[u] = kQOne;
#pragma unroll
      for (int c = 0; c < COLS; ++c) wq[u][c] = xq[u];
      if (k < kp) {
#pragma unroll
        for (int c = 0; c < COLS; ++c) wq[u][c] = *reinterpret_cast<const u32x4_t*>(w + (int64_t)c * kp + k);
        xq[u] = *reinterpret_cast<const u32x4_t*>(x + k);
        xb[u] = xs[k / kQBlock];
        wb[u] = ws[k / kQBlock];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float xv[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) q8_values4(xq[u][q], 1.f, xv + 4 * q);
      const bool bad = xb[u] == 255 || wb[u] == 255;
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float wv[4];
          q8_values4(wq[u][c][q], 1.f, wv);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fmaf(xv[4 * q + i], wv[i], s);
        }
        acc[c] += bad ? __uint_as_float(0x7fc00000u) : ldexpf(s, xb[u] + wb[u] - 254);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c) acc[c] = run_sum<64>(acc[c]);
  if (lane < COLS) {
    float v = acc[0];
#pragma unroll
    for (int c = 1; c < COLS; ++c) v = lane == c ? acc[c] : v;
    ((bf16_t*)p.C)[(int64_t)row * p.N + n0 + lane] = f2bf(v);
  }
}

}  // namespace gmm
}  // namespace moe
