// Distillation's choice of strips and logit tiles, from sizes alone (host
// code without the GPU's headers, so that it can be compiled by itself).
// Figures here, in gemm_cce.hip's distillation and in distill.hip's plan are
// of whole passes (forward + backward, dW bf16 unless said), the accepted form
// against the other in turn on one card.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kKdCus = 256;  // compute units

// The logit tiles: rows x columns, work-groups a CU.
enum KdTile : int {
  kKdWide,   // 256 x 256, 1
  kKdFew,    // 128 x 256, 2
  kKdShort,  // 128 x 128, 3
  kKdThin,   // 64 x 128, 2
};

inline int64_t kd_ceil(int64_t n, int64_t d) { return (n + d - 1) / d; }

// The forward pass keeps no logits: its strips are wide enough for four rounds
// of 256 x 256 tiles, one per CU (32-bit offsets into W allowing), and so
// depend on N, V and H alone, as lse then does.
inline int kd_forward_strip(int64_t N, int64_t V, int H) {
  const int64_t wanted = std::min(kd_ceil(4 * kKdCus, kd_ceil(N, 256)) * 256, kd_ceil(V, 256) * 256);
  const int64_t most = (((int64_t)1 << 30) - 1) / H / 256 * 256;
  return (int)std::min(wanted, most);
}

// Whether 128-row tiles, two per CU, finish before 256-row tiles, one per CU:
// in rounds of the chip, where a CU left with one 128-row tile needs half of
// one, and the smaller tiles take a tenth longer for the same products.  They
// win where a last round of 256-row tiles is mostly empty: 300 x 4096 x 100,000
// takes 1,372 us so and 1,480 with 256-row tiles, 777 x 512 x 20,000 (Short, see
// below) 136 and 157, but 1000 x 4096 x 30,000 (1.8 full rounds) with them
// everywhere 1,000 and not 917, 2000 x 2048 x 50,000 1,750 and not 1,671.
inline bool kd_few_tiles(int64_t t256, int64_t t128) {
  if (t256 >= 4 * kKdCus) return false;
  const int64_t rest = t128 % (2 * kKdCus);
  const double half_rounds = 2.0 * (double)(t128 / (2 * kKdCus)) + (rest == 0 ? 0 : rest <= kKdCus ? 1 : 2);
  return 1.1 * half_rounds < 2.0 * (double)kd_ceil(t256, kKdCus);
}

// The tile for N rows of H by a strip of w columns (the grids cover whole 256
// columns).
// Thin for up to 64 tokens, where reading W bounds the product, and where the
// whole product is one round of it, two a CU, whose steps along K take half as
// long: 47 x 3456 x 8123 takes 81 us so and 130 with Few, 500 x 2048 x 2000 71
// and 108, 16 x 4096 x 100,000 727 and 732; past one round it gains nothing (100
// x 2048 x 50,000, 1.5 rounds, 227 us with Thin and 225 with Few).
// Short is Few's work for rows of up to 512, where a tile's first loads and its
// epilogue take as long as its products and a third work-group a CU hides them:
// 777 x 512 x 20,000 takes 136 us so and 142 with Few, 600 x 256 x 60,000 188
// and 195, but 300 x 4096 x 100,000 1,489 and not 1,372 (nothing between 512 and
// 4096 was timed).
inline KdTile kd_logit_tile(int64_t N, int H, int w) {
  const int64_t cols = kd_ceil(w, 256);
  if (N <= 64 || kd_ceil(N, 64) * 2 * cols <= 2 * kKdCus) return kKdThin;
  if (kd_few_tiles(kd_ceil(N, 256) * cols, kd_ceil(N, 128) * cols)) return H <= 512 ? kKdShort : kKdFew;
  return kKdWide;
}

}  // namespace moe
