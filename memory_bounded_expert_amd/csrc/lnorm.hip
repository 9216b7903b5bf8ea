// Layer norm and its gradient (include/lnorm.h).
//
// Both passes move a few bytes per operation and are bound by HBM, so a row is
// read once and held in registers: W waves per row, C vectors of 16 bytes per
// lane.  A
// work-group walks over rows with gamma, beta (or the shares of dgamma and
// dbeta) in registers and the next row's loads in flight.  The backward pass
// writes each work-group's shares of dgamma and dbeta to the workspace, and a
// second launch adds them up in order.  Rows wider than the registers hold go
// through kernels that read the row again for each step.
#include <algorithm>
#include <cmath>

#include "device_common.hpp"
#include "lnorm.h"
#include "moe_internal.h"
#include "row_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kLnormMagic = 0x4c4e4d31u;  // "LNM1"

// Measured: 65,536 x 2048 bf16 90 us, 6.0 TB/s of reads and writes; one row of
// 2048 2.9 us.
template <typename T, int W, int C, bool TAIL>
__global__ __launch_bounds__(kGroup<W>) void lnorm_rows_forward_kernel(
    const T* X, const float* __restrict__ gamma, const float* __restrict__ beta, T* Y,
    float* __restrict__ mean, float* __restrict__ rstd, int64_t N, int H, float eps) {
  using Part = RowPart<T, W, C, TAIL>;
  constexpr int EPC = Part::EPC;
  __shared__ float red[2][1][16];
  constexpr int RPG = kGroup<W> / (64 * W);  // rows of a work-group at a time
  const int place = threadIdx.x % (64 * W);
  const float inv = 1.f / H;
  float ga[Part::COLS], be[Part::COLS];
  load_cols<EPC, W, C, TAIL>(gamma, place, H, ga);
  load_cols<EPC, W, C, TAIL>(beta, place, H, be);
  int half = 0;
  int64_t t = (int64_t)blockIdx.x * RPG + threadIdx.x / (64 * W);
  const int64_t step = (int64_t)gridDim.x * RPG;
  Part cur;
  if (kAhead<W> && t < N) cur.load(X + t * H, place, H);
  for (; t < N; t += step) {
    Part next;
    if constexpr (kAhead<W>) {
      if (t + step < N) next.load(X + (t + step) * H, place, H);
    } else {
      cur.load(X + t * H, place, H);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[EPC];
      cur.get(c, v);
#pragma unroll
      for (int e = 0; e < EPC; ++e) s[0] += v[e];
    }
    row_sums<W>(s, red, half);
    const float m = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
      if (at < H) {
        float v[EPC];
        cur.get(c, v);
#pragma unroll
        for (int e = 0; e < EPC; ++e)
          if (!TAIL || at + e < H) s[0] = fmaf(v[e] - m, v[e] - m, s[0]);
      }
    }
    row_sums<W>(s, red, half);
    const float r = 1.f / sqrtf(s[0] * inv + eps);
    if (place == 0) {
      mean[t] = m;
      rstd[t] = r;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
      if (at < H) {
        float v[EPC];
        cur.get(c, v);
#pragma unroll
        for (int e = 0; e < EPC; ++e) v[e] = fmaf((v[e] - m) * r, ga[c * EPC + e], be[c * EPC + e]);
        Part::put(Y + t * H, at, H, v);
      }
    }
    if constexpr (kAhead<W>) cur = next;
  }
}

// Where work-group g's rows' shares of dgamma and dbeta go: g 2H floats past
// these.  One work-group writes dgamma and dbeta themselves.
struct Slabs {
  float *dgamma, *dbeta;
};

// Measured:
// 65,536 x 2048 bf16 160 us, 5.0 TB/s (the copy rate); 8192 x 7168 86 us, 4.1
// TB/s, 16 rows a work-group, two work-groups a CU and a barrier a row.
template <typename T, int W, int C, bool TAIL>
__global__ __launch_bounds__(kGroup<W>) void lnorm_rows_backward_kernel(
    const T* __restrict__ X, const float* __restrict__ gamma, const T* dY,
    const float* __restrict__ mean, const float* __restrict__ rstd, T* dX,
    const Slabs part, int64_t N, int H) {
  using Part = RowPart<T, W, C, TAIL>;
  constexpr int EPC = Part::EPC;
  constexpr int RPG = kGroup<W> / (64 * W);
  __shared__ float red[2][2][16];
  const int place = threadIdx.x % (64 * W);
  const float inv = 1.f / H;
  float ga[Part::COLS], dg[Part::COLS], db[Part::COLS];
  load_cols<EPC, W, C, TAIL>(gamma, place, H, ga);
#pragma unroll
  for (int i = 0; i < Part::COLS; ++i) dg[i] = db[i] = 0.f;
  int half = 0;
  int64_t t = (int64_t)blockIdx.x * RPG + threadIdx.x / (64 * W);
  const int64_t step = (int64_t)gridDim.x * RPG;
  Part x, dy;
  float m = 0.f, r = 0.f;
  auto load = [&](int64_t u, Part& px, Part& pd, float& pm, float& pr) {
    px.load(X + u * H, place, H);
    pd.load(dY + u * H, place, H);
    pm = mean[u];
    pr = rstd[u];
  };
  if (kAhead<W> && t < N) load(t, x, dy, m, r);
  for (; t < N; t += step) {
    Part x2, dy2;
    float m2 = 0.f, r2 = 0.f;
    if constexpr (kAhead<W>) {
      if (t + step < N) load(t + step, x2, dy2, m2, r2);
    } else {
      load(t, x, dy, m, r);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      // lanes past the row's end hold x = dy = gamma = 0
      float v[EPC], d[EPC];
      x.get(c, v);
      dy.get(c, d);
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const int i = c * EPC + e;
        const float xh = (v[e] - m) * r, q = d[e] * ga[i];
        s[0] += q;
        s[1] = fmaf(q, xh, s[1]);
        dg[i] = fmaf(d[e], xh, dg[i]);
        db[i] += d[e];
      }
    }
    row_sums<W>(s, red, half);
    const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
      if (at < H) {
        float v[EPC], d[EPC];
        x.get(c, v);
        dy.get(c, d);
#pragma unroll
        for (int e = 0; e < EPC; ++e)
          d[e] = r * (fmaf(d[e], ga[c * EPC + e], -a) - (v[e] - m) * r * b);
        Part::put(dX + t * H, at, H, d);
      }
    }
    if constexpr (kAhead<W>) {
      x = x2;
      dy = dy2;
      m = m2;
      r = r2;
    }
  }
  float* pg = part.dgamma + (int64_t)blockIdx.x * 2 * H;
  float* pb = part.dbeta + (int64_t)blockIdx.x * 2 * H;
  if constexpr (RPG == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
#pragma unroll
      for (int e = 0; e < EPC; ++e)
        if (at + e < H) {
          pg[at + e] = dg[c * EPC + e];
          pb[at + e] = db[c * EPC + e];
        }
    }
  } else {
    // the work-group's waves add their shares up in order
    __shared__ float sum[2][64 * C * EPC];
    for (int w = 0; w < RPG; ++w) {
      if ((int)threadIdx.x >> 6 == w) {
#pragma unroll
        for (int i = 0; i < Part::COLS; ++i) {
          // column of element i of this lane
          const int at = (i / EPC * 64 + place) * EPC + i % EPC;
          sum[0][at] = w == 0 ? dg[i] : sum[0][at] + dg[i];
          sum[1][at] = w == 0 ? db[i] : sum[1][at] + db[i];
        }
      }
      __syncthreads();
    }
    for (int h = threadIdx.x; h < H; h += kThreads) {
      pg[h] = sum[0][h];
      pb[h] = sum[1][h];
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void lnorm_forward_kernel(
    const T* X, const float* __restrict__ gamma, const float* __restrict__ beta, T* Y,
    float* __restrict__ mean, float* __restrict__ rstd, int64_t N, int H, float eps) {
  __shared__ float red[kThreads / 64];
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const T* x = X + t * H;
    float s = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) s += Elem<T>::to_f(x[h]);
    const float m = group_sum(s, red) / H;
    float q = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float d = Elem<T>::to_f(x[h]) - m;
      q = fmaf(d, d, q);
    }
    const float r = 1.f / sqrtf(group_sum(q, red) / H + eps);
    if (threadIdx.x == 0) {
      mean[t] = m;
      rstd[t] = r;
    }
    for (int h = threadIdx.x; h < H; h += kThreads)
      Y[t * H + h] = Elem<T>::from_f(fmaf((Elem<T>::to_f(x[h]) - m) * r, gamma[h], beta ? beta[h] : 0.f));
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void lnorm_backward_kernel(
    const T* __restrict__ X, const float* __restrict__ gamma, const T* dY,
    const float* __restrict__ mean, const float* __restrict__ rstd, T* dX,
    const Slabs part, int64_t N, int H) {
  __shared__ float red[kThreads / 64];
  float* pg = part.dgamma + (int64_t)blockIdx.x * 2 * H;
  float* pb = part.dbeta + (int64_t)blockIdx.x * 2 * H;
  for (int h = threadIdx.x; h < H; h += kThreads) pg[h] = pb[h] = 0.f;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const T* x = X + t * H;
    const T* dy = dY + t * H;
    const float m = mean[t], r = rstd[t];
    float a = 0.f, b = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float d = Elem<T>::to_f(dy[h]), xh = (Elem<T>::to_f(x[h]) - m) * r;
      const float dg = d * gamma[h];
      a += dg;
      b = fmaf(dg, xh, b);
      pg[h] = fmaf(d, xh, pg[h]);
      pb[h] += d;
    }
    a = group_sum(a, red) / H;
    b = group_sum(b, red) / H;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float dg = Elem<T>::to_f(dy[h]) * gamma[h], xh = (Elem<T>::to_f(x[h]) - m) * r;
      dX[t * H + h] = Elem<T>::from_f(r * (dg - a - xh * b));
    }
  }
}

template <typename T>
hipError_t run_forward(const lnorm_plan_t& P, const void* X, const float* gamma, const float* beta,
                       void* Y, float* mean, float* rstd, hipStream_t st) {
  const Holding h = holding(P.H, P.dtype);
  if (h.W == 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(P.N, kMaxRowGrid);
    lnorm_forward_kernel<T><<<grid, kThreads, 0, st>>>((const T*)X, gamma, beta, (T*)Y, mean, rstd,
                                                       P.N, P.H, P.eps);
  } else {
    const int grid = row_groups(P.N, h.W);
    with_holding<T>(h, P.H, [&](auto w, auto c, auto tail) {
      lnorm_rows_forward_kernel<T, w.value, c.value, tail.value><<<grid, kGroup<w.value>, 0, st>>>(
          (const T*)X, gamma, beta, (T*)Y, mean, rstd, P.N, P.H, P.eps);
    });
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run_backward(const lnorm_plan_t& P, const void* X, const float* gamma, const void* dY,
                        const float* mean, const float* rstd, void* dX, Slabs part, int slabs,
                        hipStream_t st) {
  const Holding h = holding(P.H, P.dtype);
  const int grid = slabs;
  if (h.W == 0) {
    lnorm_backward_kernel<T><<<grid, kThreads, 0, st>>>((const T*)X, gamma, (const T*)dY, mean, rstd,
                                                        (T*)dX, part, P.N, P.H);
  } else {
    with_holding<T>(h, P.H, [&](auto w, auto c, auto tail) {
      lnorm_rows_backward_kernel<T, w.value, c.value, tail.value><<<grid, kGroup<w.value>, 0, st>>>(
          (const T*)X, gamma, (const T*)dY, mean, rstd, (T*)dX, part, P.N, P.H);
    });
  }
  return hipGetLastError();
}

bool plan_ok(const lnorm_plan_t* p) { return p != nullptr && p->magic == kLnormMagic; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int lnorm_plan(int64_t N, int32_t H, int32_t dtype, float eps, lnorm_plan_t* out) {
  if (!out || N < 0 || H < 1 || !(eps > 0.f) || !std::isfinite(eps)) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (H > 65536 || N >= ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
  lnorm_plan_t p{};
  p.magic = kLnormMagic;
  p.dtype = dtype;
  p.N = N;
  p.H = H;
  p.eps = eps;
  p.bwd_workspace_bytes = std::min<int64_t>(N, kMaxSlabs) * 2 * H * sizeof(float);
  *out = p;
  return MOE_OK;
}

MOE_API int lnorm_forward(const lnorm_plan_t* plan, const void* X, const float* gamma,
                          const float* beta, void* Y, float* mean, float* rstd, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const lnorm_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!X || !gamma || !Y || !mean || !rstd) return MOE_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const hipError_t err = P.dtype == MOE_BF16
                             ? run_forward<bf16_t>(P, X, gamma, beta, Y, mean, rstd, st)
                             : run_forward<float>(P, X, gamma, beta, Y, mean, rstd, st);
  return err == hipSuccess ? MOE_OK : MOE_EHIP;
}

MOE_API int lnorm_backward(const lnorm_plan_t* plan, const void* X, const float* gamma,
                           const void* dY, const float* mean, const float* rstd, void* dX,
                           float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const lnorm_plan_t& P = *plan;
  if (!dgamma) return MOE_EINVAL;
  if (P.N > 0 && (!X || !gamma || !dY || !mean || !rstd || !dX || !workspace)) return MOE_EINVAL;
  if (P.N > 0 && (uintptr_t)workspace % 256) return MOE_EINVAL;
  if (workspace_bytes < (size_t)P.bwd_workspace_bytes) return MOE_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int slabs = P.N > 0 ? slab_count(P.N, holding(P.H, P.dtype).W) : 0;
  float* part = (float*)workspace;
  if (P.N > 0) {
    const Slabs to = slabs == 1 ? Slabs{dgamma, dbeta ? dbeta : part} : Slabs{part, part + P.H};
    const hipError_t err =
        P.dtype == MOE_BF16
            ? run_backward<bf16_t>(P, X, gamma, dY, mean, rstd, dX, to, slabs, st)
            : run_backward<float>(P, X, gamma, dY, mean, rstd, dX, to, slabs, st);
    if (err != hipSuccess) return MOE_EHIP;
    if (slabs == 1) return MOE_OK;
  }
  slab_fold_kernel<<<(unsigned)ceil_div(2 * (int64_t)P.H, 64), 64 * kFoldWaves, 0, st>>>(
      part, slabs, 2 * P.H, P.H, dgamma, dbeta);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
