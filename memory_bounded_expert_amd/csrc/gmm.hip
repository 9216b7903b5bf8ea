// Matrix products grouped by expert, with ragged sizes (include/gmm.h): which
// kernel, tile and split a product takes, and the calls.
#include <algorithm>

#include "gmm.h"
#include "gmm_rows.hpp"
#include "gmm_single.hpp"
#include "gmm_weights.hpp"
#include "moe_internal.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

using namespace gmm;

constexpr uint32_t kGmmMagic = 0x474d4d31u;  // "GMM1"

bool plan_ok(const gmm_plan_t* p, int operands) {
  return p != nullptr && p->magic == kGmmMagic && p->operands == operands;
}
bool aligned(const void* p, int to) { return p && (uintptr_t)p % to == 0; }
// 0: go on
int check_call(const gmm_plan_t& P, const int32_t* offsets, const void* workspace, size_t bytes,
               int64_t needed) {
  if (offsets ? (uintptr_t)offsets % 4 != 0 : P.E != 1) return MOE_EINVAL;
  if (needed > 0 && !aligned(workspace, 256)) return MOE_EINVAL;
  return bytes < (size_t)needed ? MOE_EWORKSPACE : MOE_OK;
}
int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }

// Row tiles of all experts at most.
int64_t row_tiles(int64_t R, int E, int bm) { return R / bm + std::min<int64_t>(E, R); }

// Tiles, and into how many parts k is split.
enum class Size { Large, Middle, Small, Few, Tiny, Single };
struct Choice {
  Size size;
  int splits, steps;  // steps: of a part
};

// Tiles of bm x bn that R rows over E experts come to, rows spread evenly: an
// expert's last row tile is half full.
int64_t tiles_of(int64_t R, int E, int N, int bm, int bn) {
  const int64_t experts = std::min<int64_t>(E, R), rows = ceil_div(R, std::max<int64_t>(experts, 1));
  const int64_t halves = rows <= bm ? 2 : 2 * rows / bm + 1;
  return experts * halves / 2 * ceil_div(N, bn);
}

// Microseconds with one tile and the other, in bf16 forward / dX and in e4m3:
//  * Single (dot products) for up to 4 rows in e4m3: 1 x 7168 x 2048 5.6 us in a graph
//    (Few in parts 8.4), 4 rows 8.5 (8.8), 8 rows 13.9 (8.9); 1 x 2048 x 1408 3.0 (6.6).
//    All of one matrix, which the rows share; not measured over several.
//  * Few (64 x 64, four stages) where there are fewer 64 x 128 tiles than CUs, so
//    that a step's latency counts: 64 x 4096 x 4096 17 / 15, 10 (Small 35 / 35, 13).
//  * Tiny (16 or 32 rows) for up to 16 rows an expert: 128 x 2048 x 1408 over 64
//    experts 53.8 / 55, 25.8 (Small 54.6 / 66, 26.4).
//  * Small (64 x 128) for up to 48, and where larger tiles leave CUs idle: 2048 rows
//    68.8 / 78 (Middle 80 / 68); 1500 x 2048 x 2048 22.7 / 21.7, 12.6 (Middle 24 / 24, 14).
//  * Middle (128 x 128, two work-groups a CU) for up to 96, in e4m3 up to 512:
//    4096 rows 83 / 72, 36 (Large 97 / 81, 41); 16,384 rows 146 / 147, 62 (Large 157 /
//    130, 78).
//  * Large (256 x 256) for more: 8192 rows 106 / 86 (Middle 107 / 100); 32,768 rows 223 /
//    214, 112 (Middle 246 / 259, 110).
// Few tiles and a long k: parts of at least eight steps, up to a work-group a CU (1 x
// 7168 x 2048 21 -> 11.5; 64 x 4096 x 4096 17.3 -> 16.6).
Choice choose_rows(bool q8, int64_t R, int K, int N, int E) {
  if (q8 && R <= 4) return Choice{Size::Single, 1, 0};
  const int64_t rows = ceil_div(R, std::max<int64_t>(std::min<int64_t>(E, R), 1));
  const int64_t few = tiles_of(R, E, N, 64, 64);
  if (tiles_of(R, E, N, 64, 128) <= kCus) {
    const int steps = (int)ceil_div(K, q8 ? 128 : 64);
    const int64_t parts = std::min<int64_t>(few < 64 ? kCus / std::max<int64_t>(few, 1) : 1, steps / 8);
    if (parts < 2) return Choice{Size::Few, 1, 0};
    const int each = (int)(ceil_div(ceil_div(steps, parts), 4) * 4);  // the scales' words hold four steps
    return Choice{Size::Few, (int)ceil_div(steps, each), each};
  }
  if (rows <= 16) return Choice{Size::Tiny, 1, 0};
  if (rows > (q8 ? 512 : 96) && tiles_of(R, E, N, 256, 256) >= 160) return Choice{Size::Large, 1, 0};
  if (rows > 48 && tiles_of(R, E, N, 128, 128) >= kCus) return Choice{Size::Middle, 1, 0};
  return Choice{Size::Small, 1, 0};
}

// Large (256 x 256) from 160 tiles on, otherwise Middle (128 x 128, two work-groups a
// CU): 8192 x 2048 x 2048, 64 large tiles, 167 us and 69.  Few tiles over many rows:
// parts of at least eight steps, up to a work-group a CU (32,768 x 512 x 512 219 -> 38
// us with 8 parts and more).
Choice choose_weights(int64_t R, int K, int N, int E) {
  if (E * ceil_div(K, 256) * ceil_div(N, 256) >= 160) return Choice{Size::Large, 1, 0};
  const int64_t tiles = E * ceil_div(K, 128) * ceil_div(N, 128);
  const int64_t steps = ceil_div(ceil_div(R, std::max(E, 1)), 32);
  const int64_t parts = std::min(kCus / std::max<int64_t>(tiles, 1), steps / 8);
  return Choice{Size::Middle, (int)std::max<int64_t>(parts, 1), 0};
}

int64_t part_bytes(const Choice& c, int64_t values) { return c.splits > 1 ? c.splits * values * 4 : 0; }

template <Form F, class S>
int rows_launch(const Args& a, const Choice& c, hipStream_t st) {
  const int ntiles = (int)ceil_div(a.N, S::BN);
  const dim3 grid((unsigned)(row_tiles(a.R, a.E, S::BM) * ntiles), c.splits);
  constexpr int lds = RowsCfg<F, S>::LDS;
  static uint64_t whole = 0;
  (void)hipGetLastError();
  if constexpr (S::NS == 4) {  // Few: the only one that is split
    if (c.splits > 1) {
      static uint64_t part = 0;
      auto kern = gmm_rows_kernel<F, S, true>;
      if (set_lds_attr(kern, lds, part) != hipSuccess) return MOE_EHIP;
      kern<<<grid, S::THREADS, lds, st>>>(a, ntiles, c.steps);
      if (const int bad = launched()) return bad;
      const unsigned groups = (unsigned)std::min<int64_t>(ceil_div((int64_t)a.R * a.N / 8, kThreads), 2048);
      gmm_join_kernel<<<groups, kThreads, 0, st>>>(a.part, (bf16_t*)a.C, a.offsets, a.E, a.R, a.N, c.splits);
      return launched();
    }
  }
  auto kern = gmm_rows_kernel<F, S, false>;
  if (set_lds_attr(kern, lds, whole) != hipSuccess) return MOE_EHIP;
  kern<<<grid, S::THREADS, lds, st>>>(a, ntiles, 0);
  return launched();
}

int single_launch(const Args& a, hipStream_t st) {
  (void)hipGetLastError();
  const unsigned grid = (unsigned)(ceil_div(ceil_div(a.N, kSingleCols * (kThreads / 64)), 8) * 8 * a.R);
  // (1 x 2048 x 1408 2.96 us with two KiB of a row in flight, 3.22 with four; 1 x 7168 x
  // 2048 6.3 and 6.1)
  auto kern = a.K <= 4096 ? gmm_single_kernel<2> : gmm_single_kernel<4>;
  kern<<<grid, kThreads, 0, st>>>(a);
  return launched();
}

// Calls g with the tile of a size.
template <Form F, typename G>
auto with_rows_shape(Size size, G g) {
  switch (size) {
    // (waves of 64 x 128, or in bf16 128 x 64, of which the transposing reads want
    // fewer columns: 16,384 x 4096 x 4096 forward 410 us and 397)
    case Size::Large: return g(std::conditional_t<F == Form::Q8, GShape<256, 256, 4, 2, 2>, GShape<256, 256, 2, 4, 2>>());
    case Size::Middle: return g(GShape<128, 128, 2, 2, 2>());
    case Size::Small: return g(GShape<64, 128, 2, 2, 2>());
    case Size::Few: return g(GShape<64, 64, 2, 2, 4>());
    default: return g(GShape<F == Form::Q8 ? 32 : 16, 128, 1, 4, 2>());
  }
}
template <typename G>
auto with_weights_shape(Size size, G g) {
  if (size == Size::Large) return g(GShape<256, 256, 4, 2, 4>());
  return g(GShape<128, 128, 2, 2, 4>());
}

// Whether a product's launch has fewer than 2^32 threads along x (HIP refuses others).
constexpr int64_t kLaunchThreads = (int64_t)1 << 32;
template <Form F>
bool rows_launchable(const Choice& c, int64_t R, int N, int E) {
  return c.size == Size::Single || with_rows_shape<F>(c.size, [&](auto s) {
           return row_tiles(R, E, s.BM) * ceil_div(N, s.BN) * s.THREADS < kLaunchThreads;
         });
}
bool weights_launchable(const Choice& c, int K, int N, int E) {
  return with_weights_shape(c.size, [&](auto s) {
    return weights_groups(E * ceil_div(K, s.BM) * ceil_div(N, s.BN)) * s.THREADS < kLaunchThreads;
  });
}

template <Form F>
int rows_product(Args a, void* workspace, hipStream_t st) {
  const Choice c = choose_rows(F == Form::Q8, a.R, a.K, a.N, a.E);
  a.part = (float*)workspace;
  if constexpr (F == Form::Q8)
    if (c.size == Size::Single) return single_launch(a, st);
  return with_rows_shape<F>(c.size, [&](auto s) { return rows_launch<F, decltype(s)>(a, c, st); });
}

template <Form F, class S>
int weights_launch(const Args& a, const Choice& c, hipStream_t st) {
  const int mtiles = (int)ceil_div(a.K, S::BM), ntiles = (int)ceil_div(a.N, S::BN);
  const dim3 grid((unsigned)weights_groups((int64_t)a.E * mtiles * ntiles), c.splits);
  constexpr int lds = WeightsCfg<F, S>::LDS;
  static uint64_t whole = 0;
  (void)hipGetLastError();
  if constexpr (S::BM == 128) {  // Middle: the only one that is split
    if (c.splits > 1) {
      static uint64_t part = 0;
      auto kern = gmm_weights_kernel<F, S, true>;
      if (set_lds_attr(kern, lds, part) != hipSuccess) return MOE_EHIP;
      kern<<<grid, S::THREADS, lds, st>>>(a, mtiles, ntiles);
      if (const int bad = launched()) return bad;
      const int64_t vecs = (int64_t)a.E * a.K * a.N / 4;
      gmm_join_weights_kernel<<<(unsigned)std::min<int64_t>(ceil_div(vecs, kThreads), 4096), kThreads, 0, st>>>(
          a.part, (float*)a.C, vecs, c.splits, a.accumulate);
      return launched();
    }
  }
  auto kern = gmm_weights_kernel<F, S, false>;
  if (set_lds_attr(kern, lds, whole) != hipSuccess) return MOE_EHIP;
  kern<<<grid, S::THREADS, lds, st>>>(a, mtiles, ntiles);
  return launched();
}

template <Form F>
int weights_product(Args a, void* workspace, hipStream_t st) {
  const Choice c = choose_weights(a.R, a.K, a.N, a.E);
  a.part = (float*)workspace;
  return with_weights_shape(c.size, [&](auto s) { return weights_launch<F, decltype(s)>(a, c, st); });
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int gmm_plan(int64_t R, int32_t K, int32_t N, int32_t E, int32_t operands, gmm_plan_t* out) {
  if (!out || R < 0 || K < 1 || N < 1 || E < 0 || (E == 0 && R > 0)) return MOE_EINVAL;
  if (operands != GMM_BF16 && operands != GMM_Q8) return MOE_EINVAL;
  if (N % 8 || (operands == GMM_BF16 && K % 8)) return MOE_EINVAL;
  if (K > 65536 || N > 65536 || E > 1024 || R >= ((int64_t)1 << 31) - 65536) return MOE_EUNSUPPORTED;
  if (2 * (int64_t)K * N >= ((int64_t)1 << 31) || R * std::max(K, N) >= ((int64_t)1 << 40)) return MOE_EUNSUPPORTED;
  gmm_plan_t p{};
  p.magic = kGmmMagic;
  p.operands = operands;
  p.R = R;
  p.K = K;
  p.N = N;
  p.E = E;
  p.row_pitch = operands == GMM_BF16 ? 2 * K : q8_row_pitch(K);
  const bool q8 = operands == GMM_Q8;
  const Choice dw = choose_weights(R, K, N, E);
  if (!weights_launchable(dw, K, N, E)) return MOE_EUNSUPPORTED;
  if (R > 0) {
    const Choice y = choose_rows(q8, R, K, N, E);
    if (!(q8 ? rows_launchable<Form::Q8>(y, R, N, E) : rows_launchable<Form::NN>(y, R, N, E))) return MOE_EUNSUPPORTED;
    p.fwd_workspace_bytes = part_bytes(y, R * N);
    if (!q8) {
      const Choice dx = choose_rows(false, R, N, K, E);
      if (!rows_launchable<Form::NT>(dx, R, K, E)) return MOE_EUNSUPPORTED;
      p.fwd_workspace_bytes = std::max(p.fwd_workspace_bytes, part_bytes(dx, R * K));
    }
    p.bwd_workspace_bytes = part_bytes(dw, (int64_t)E * K * N);
  }
  *out = p;
  return MOE_OK;
}

MOE_API int gmm_forward(const gmm_plan_t* plan, const void* X, const void* W, const int32_t* offsets,
                        void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::NN>(Args{X, nullptr, W, nullptr, Y, offsets, (int)P.R, P.E, P.K, P.N, 0, nullptr}, workspace, (hipStream_t)stream);
}

MOE_API int gmm_backward_dx(const gmm_plan_t* plan, const void* dY, const void* W, const int32_t* offsets,
                            void* dX, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(dY, 16) || !aligned(W, 16) || !aligned(dX, 16)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::NT>(Args{dY, nullptr, W, nullptr, dX, offsets, (int)P.R, P.E, P.N, P.K, 0, nullptr}, workspace, (hipStream_t)stream);
}

MOE_API int gmm_backward_dw(const gmm_plan_t* plan, const void* X, const void* dY, const int32_t* offsets,
                            float* dW, int32_t accumulate, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.E == 0) return MOE_OK;
  if (!aligned(dW, 16) || (P.R > 0 && (!aligned(X, 16) || !aligned(dY, 16)))) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.bwd_workspace_bytes)) return bad;
  return weights_product<Form::TN>(Args{X, nullptr, dY, nullptr, dW, offsets, (int)P.R, P.E, P.K, P.N, accumulate != 0, nullptr}, workspace, (hipStream_t)stream);
}

MOE_API int gmm8_forward(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* Wq,
                         const void* Ws, const int32_t* offsets, void* Y, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_Q8)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(Xs, 4) || !aligned(Ws, 4)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::Q8>(Args{Xq, Xs, Wq, Ws, Y, offsets, (int)P.R, P.E, P.K, P.N, 0, nullptr}, workspace, (hipStream_t)stream);
}

MOE_API int gmm8_backward_dw(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* dY,
                             const int32_t* offsets, float* dW, int32_t accumulate, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_Q8)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.E == 0) return MOE_OK;
  if (!aligned(dW, 16) || (P.R > 0 && (!aligned(Xq, 16) || !aligned(Xs, 4) || !aligned(dY, 16)))) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.bwd_workspace_bytes)) return bad;
  return weights_product<Form::TN8>(Args{Xq, Xs, dY, nullptr, dW, offsets, (int)P.R, P.E, P.K, P.N, accumulate != 0, nullptr}, workspace, (hipStream_t)stream);
}
