// Contractions of the vocabulary-strip cross-entropy (bf16, LDS pipeline):
// the strip's logits X W_s^T with the statistics or gradient epilogue, the
// running sum dX += G W_s, and the strip's weight gradient dW_s = G^T X.
#include "gemm_kernel.hpp"
#include "gemm_lds.hpp"
#include "kd_shapes.hpp"

namespace moe {
using namespace gemm;

namespace {
// 256 x 256 tiles of 4 x 2 waves; each wave's 64 x 128 block is one
// 128-column vocabulary slice of the statistics.
using Logit = Shape<256, 256, 4, 2, 32, 1>;
// Distillation's smaller tiles (kd_shapes.hpp says which when).
using LogitFew = Shape<128, 256, 2, 2, 32, 2>;
using LogitShort = Shape<128, 128, 4, 1, 32, 3>;
using LogitThin = Shape<64, 128, 4, 1, 64, 2>;
static_assert(kKdCus == kCus, "one chip");
static_assert(Logit::BN / Logit::WGN == kCceSlice, "statistics slice = one wave's columns");
static_assert(LogitFew::BN / LogitFew::WGN == kCceSlice, "statistics slice = one wave's columns");
static_assert(LogitShort::BN / LogitShort::WGN == kCceSlice, "statistics slice = one wave's columns");
static_assert(LogitThin::BN / LogitThin::WGN == kCceSlice, "statistics slice = one wave's columns");
}  // namespace

hipError_t gemm_cce_logits(bool grad, const void* X, const void* Ws, int64_t N, int H, int w,
                           int64_t col0, const int32_t* targets, float* pmax, float* psum,
                           float* ytgt, const float* lse, const float* dl, void* G, int ldg,
                           hipStream_t st) {
  if (N == 0 || w == 0) return hipSuccess;
  Params p{};
  p.A = X; p.lda = H;
  p.B = Ws; p.ldb = H;
  p.M = (int)N; p.N = w; p.K = H;
  p.ce_targets = targets; p.ce_col0 = col0;
  const dim3 grid((unsigned)ceil_div(N, Logit::BM), (unsigned)ceil_div(w, Logit::BN));
  if (!grad) {
    p.ce_pmax = pmax; p.ce_psum = psum; p.ce_ytgt = ytgt;
    return launch_lds<Mode::Dense, Logit, false, true, true, false, Epi::CEStats>(p, grid, st);
  }
  p.ce_lse = lse; p.ce_dl = dl;
  p.C = G; p.ldc = ldg;
  return launch_lds<Mode::Dense, Logit, false, true, true, false, Epi::CEGrad>(p, grid, st);
}

hipError_t gemm_cce_dx(const void* G, int ldg, const void* Ws, int64_t N, int H, int w,
                       float* dx, bool first, hipStream_t st) {
  if (N == 0) return hipSuccess;
  Params p{};
  p.A = G; p.lda = ldg;
  p.B = Ws; p.ldb = H;
  p.C = dx; p.ldc = H;
  p.M = (int)N; p.N = H; p.K = w;
  p.acc_init = first ? 1 : 0;
  p.acc_chain = 1;
  const int bn = H % 256 == 0 ? 256 : 128;
  const dim3 grid((unsigned)ceil_div(N, 256), (unsigned)(H / bn));
  if (bn == 256)
    return launch_lds<Mode::Dense, Shape<256, 256, 4, 2, 32, 1>, false, true, false, false, Epi::AccF32>(p, grid, st);
  return launch_lds<Mode::Dense, Shape<256, 128, 4, 2, 32, 1>, false, true, false, false, Epi::AccF32>(p, grid, st);
}

hipError_t gemm_cce_dw(const void* G, int ldg, const void* X, int64_t N, int H, int w, float* dws,
                       hipStream_t st) {
  if (w == 0) return hipSuccess;
  Params p{};
  p.A = G; p.lda = ldg;
  p.B = X; p.ldb = H;
  p.C = dws; p.ldc = H; p.c_estride = 0;
  p.M = w; p.N = H; p.K = (int)N;  // one segment: rows [0, N) of G and X (no offsets)
  p.acc_init = 1;
  // K = N rows is long: 8 x 8 blocks of tiles run together and share their
  // K-tiles through L2 (the N-tile-fastest order re-reads all of X per M-tile)
  p.tile_group = kCceDwGroup;
  const int bn = H % 256 == 0 ? 256 : 128;
  const dim3 grid((unsigned)ceil_div(w, 128), (unsigned)(H / bn), 1u);
  if (bn == 256)
    return launch_lds<Mode::Expert, Shape<128, 256, 2, 2, 32, 2>, false, false, false, false, Epi::AccF32>(p, grid, st);
  return launch_lds<Mode::Expert, Shape<128, 128, 2, 4, 64, 1>, false, false, false, false, Epi::AccF32>(p, grid, st);
}

hipError_t gemm_kd_logits(bool grad, const void* X, const void* Ws, int64_t N, int H, int w,
                          float T, float* pmax, float* psum, const float* lse, const float* dloss,
                          void* G, int ldg, hipStream_t st) {
  if (N == 0 || w == 0) return hipSuccess;
  Params p{};
  p.A = X; p.lda = H;
  p.B = Ws; p.ldb = H;
  p.M = (int)N; p.N = w; p.K = H;
  p.ce_scale = 1.f / T;
  if (!grad) {
    p.ce_pmax = pmax; p.ce_psum = psum;
  } else {
    p.ce_lse = lse; p.ce_dl = dloss; p.ce_up = T;
    p.C = G; p.ldc = ldg;
  }
  const unsigned cols = (unsigned)ceil_div(w, 256);  // the statistics and G go to whole 256 columns
  auto run = [&](auto shape) {
    using S = decltype(shape);
    dim3 g((unsigned)ceil_div(N, S::BM), cols * (256 / S::BN));
    // Few row tiles: those of a column tile on one XCD, whose L2 then reads W
    // once.  In the plain order each is on another: 777 x 512 x 20,000 takes 142
    // us so and 136 in this order, 500 x 4096 x 30,000 528 and 518, 1000 x 4096 x
    // 30,000 938 and 917, 2000 x 2048 x 50,000 1,688 and 1,671; of 16 tiles the
    // rows themselves no longer fit beside W (4000 x 4096 x 20,000 2,271 and 2,291).
    if (g.x > 1 && g.x <= 8) {
      p.tile_group = (int)g.y;
      g.y = (g.y + 7) / 8 * 8;
    }
    return grad ? launch_lds<Mode::Dense, S, false, true, true, false, Epi::KDGrad>(p, g, st)
                : launch_lds<Mode::Dense, S, false, true, true, false, Epi::KDStats>(p, g, st);
  };
  switch (kd_logit_tile(N, H, w)) {
    case kKdThin: return run(LogitThin());
    case kKdShort: return run(LogitShort());
    case kKdFew: return run(LogitFew());
    default: return run(Logit());
  }
}

hipError_t gemm_kd_dx(const void* G, int ldg, const void* Ws, int64_t N, int H, int w, int64_t v0,
                      float* sums, int range, int slots, hipStream_t st) {
  Params p{};
  p.lda = ldg;
  p.ldb = H;
  p.C = sums; p.ldc = H; p.c_estride = N * H;
  p.M = (int)N; p.N = H;
  p.range = range;
  p.range_slots = slots;
  const int bn = H % 256 == 0 ? 256 : 128;
  // at most `slots` ranges a launch, so that each has a sum of its own
  for (int64_t v = v0; v < v0 + w;) {
    const int64_t first = v / range, end = std::min(v0 + w, (first + slots) * range);
    p.A = (const bf16_t*)G + (v - v0);
    p.B = (const bf16_t*)Ws + (v - v0) * H;
    p.K = (int)(end - v);
    p.range_first = (int)first;
    p.range_off = (int)(v - first * range);
    const dim3 grid((unsigned)ceil_div(N, 256), (unsigned)(H / bn), (unsigned)ceil_div(end - first * range, range));
    const hipError_t err =
        bn == 256 ? launch_lds<Mode::Dense, Shape<256, 256, 4, 2, 32, 1>, false, true, false, false, Epi::AccRanges>(p, grid, st)
                  : launch_lds<Mode::Dense, Shape<256, 128, 4, 2, 32, 1>, false, true, false, false, Epi::AccRanges>(p, grid, st);
    if (err != hipSuccess) return err;
    v = end;
  }
  return hipSuccess;
}

hipError_t gemm_kd_dw(bool bf16, const void* G, int ldg, const void* X, int64_t N, int H, int w,
                      void* dws, hipStream_t st) {
  if (w == 0) return hipSuccess;
  Params p{};
  p.A = G; p.lda = ldg;
  p.B = X; p.ldb = H;
  p.C = dws; p.ldc = H;
  p.M = w; p.N = H; p.K = (int)N;
  p.acc_init = 1;
  p.tile_group = kCceDwGroup;  // as gemm_cce_dw
  // Few tokens: writing dW bounds it, and three small work-groups a CU write
  // more steadily (16 x 4096 x 100,000 727 us so and 746 with the wide tiles,
  // 333 x 2048 x 50,000 395 and 398, but 1000 x 4096 x 30,000 932 and 917; nothing
  // between 333 and 777 tokens was timed).  So too where the wide tiles do not
  // fill the chip (8000 x 512 x 20,000, 66 a strip, 1,093 and 1,263, 7778 x 256 x
  // 1813 153 and 189), and where H is no multiple of 256 (16 x 4224 x 100,000 714
  // and 904 with one 512-thread work-group a CU, 4000 x 4224 x 20,000 2,680 and
  // 2,855).
  const bool wide = H % 256 == 0 && N > 512 && ceil_div(w, 128) * (H / 256) >= 2 * kCus;
  auto run = [&](auto shape) {
    using S = decltype(shape);
    const dim3 grid((unsigned)ceil_div(w, S::BM), (unsigned)(H / S::BN), 1u);
    return bf16 ? launch_lds<Mode::Expert, S, false, false, false, false, Epi::Store>(p, grid, st)
                : launch_lds<Mode::Expert, S, false, false, false, false, Epi::AccF32>(p, grid, st);
  };
  return wide ? run(Shape<128, 256, 2, 2, 32, 2>()) : run(Shape<128, 128, 2, 2, 32, 3>());
}

}  // namespace moe
