// Root-mean-square norm with the residual's addition, and its gradient
// (include/rms.h).
//
// As layer norm's (lnorm.hip), both passes are bound by HBM: a row is read once
// and held in registers by W waves, C vectors of 16 bytes per lane, the next row's
// loads in flight.  A block of 128 columns lies in 16 lanes (bf16) or 32 (fp32),
// so an 8-bit output takes its scale from a reduction within the wave and costs no
// pass of its own.  The backward pass needs one sum per row; shares of dgamma go
// to slabs that a second launch adds up in order.  Rows are written past L2 (65,536 x
// 2048 bf16 into 8 bits 190 us, 177 so; backward 207, 198; 60,000 x 1000 89, 74).  Rows
// wider than the registers hold go through kernels that read the row again for each
// step.
#include <algorithm>
#include <cmath>

#include "device_common.hpp"
#include "moe_internal.h"
#include "q8_ops.hpp"
#include "rms.h"
#include "row_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kRmsMagic = 0x524d5331u;  // "RMS1"

// Where a row's output goes: Y of the rows' type, or q and s of 8 bits.
struct RowsOut {
  void *y, *q, *s;
  int row_pitch, scale_pitch;
};

// A row's sum over its W waves, from 16 lanes on in 64 bits; `red` alternates between
// two halves, so one barrier is enough.
template <int W>
__device__ __forceinline__ double row_sum64(float v, double (*red)[16], int& half) {
  v = run_sum<16>(v);
  auto lane = [&](int l) { return (double)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l)); };
  double s = (lane(0) + lane(16)) + (lane(32) + lane(48));
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[half][threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[half][w];
    half ^= 1;
  }
  return s;
}
// Sum over the work-group, in 64 bits; `red` as in row_sum64.
__device__ __forceinline__ double group_sum64(double v, double (*red)[16], int& half) {
#pragma unroll
  for (int n = 32; n > 0; n /= 2) v += __shfl_xor(v, n);
  if ((threadIdx.x & 63) == 0) red[half][threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += red[half][w];
  half ^= 1;
  return v;
}
// 1 / sqrt(m) from r, which is that in 32 bits, by a Newton step.
__device__ __forceinline__ double rstd64(double m, float r) {
  return fma(0.5 * r, fma(-m * r, (double)r, 1.0), (double)r);
}
// A value for 8 bits, y = v r g in 32 bits.  (65,536 x 2048: 15 to 23 of 134 million numbers are not
// those of 64 bits; all in 32 bits 67 to 109.)
__device__ __forceinline__ float exact8(float y, float v, float g, double r64) {
  return q8_border(y) ? q8_to_odd((double)v * r64 * (double)g) : y;
}

// 65,536 x 2048 with a residual into 8 bits: bf16 178 us, 5.3 TB/s; fp32 338 us, 5.2 TB/s.
template <typename T, int W, int C, bool TAIL, bool Q8>
__global__ __launch_bounds__(kGroup<W>) void rms_rows_forward_kernel(
    const T* X, const T* residual, const float* __restrict__ gamma, T* S, const RowsOut out,
    float* __restrict__ rstd, int64_t N, int H, float eps) {
  using Part = RowPart<T, W, C, TAIL>;
  constexpr int EPC = Part::EPC;
  __shared__ double red[2][16];
  constexpr int RPG = kGroup<W> / (64 * W);  // rows of a work-group at a time
  const int place = threadIdx.x % (64 * W);
  const double inv = 1.0 / H;
  float ga[Part::COLS];
  load_cols<EPC, W, C, TAIL>(gamma, place, H, ga);
  int half = 0;
  int64_t t = (int64_t)blockIdx.x * RPG + threadIdx.x / (64 * W);
  const int64_t step = (int64_t)gridDim.x * RPG;
  Part cur, res;
  auto load = [&](int64_t u, Part& x, Part& r) {
    x.load(X + u * H, place, H);
    if (residual) r.load(residual + u * H, place, H);
  };
  if (kAhead<W> && t < N) load(t, cur, res);
  for (; t < N; t += step) {
    Part next, nres;
    if constexpr (kAhead<W>) {
      if (t + step < N) load(t + step, next, nres);
    } else {
      load(t, cur, res);
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[EPC];
      cur.get(c, v);
      if (residual) {
        // the sum as the rows' type holds it: what is written, normed and read back
        float r[EPC];
        res.get(c, r);
#pragma unroll
        for (int e = 0; e < EPC; ++e) v[e] += r[e];
        cur.raw[c] = pack16(v, T());
        cur.get(c, v);
        Part::template put<true>(S + t * H, (c * 64 * W + place) * EPC, H, v);
      }
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < EPC; ++e) part = fmaf(v[e], v[e], part);
      sum += part;
    }
    const double m = fma(row_sum64<W>(sum, red, half), inv, (double)eps);
    const float r = 1.f / sqrtf((float)m);
    const double r64 = rstd64(m, r);
    if (place == 0) rstd[t] = r;
    if constexpr (Q8) {
      uint8_t* q = (uint8_t*)out.q + t * out.row_pitch;
      uint8_t* sc = (uint8_t*)out.s + t * out.scale_pitch;
      const int blocks = q8_blocks(H);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = (c * 64 * W + place) * EPC;
        float v[EPC];
        cur.get(c, v);
        float y[EPC];
        bool border = false;
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          y[e] = v[e] * r * ga[c * EPC + e];
          // past the row's end x and gamma are 0, but r may be NaN
          if (at + e >= H) y[e] = 0.f;
          border |= q8_border(y[e]);
        }
        if (border) {
#pragma unroll
          for (int e = 0; e < EPC; ++e) y[e] = exact8(y[e], v[e], ga[c * EPC + e], r64);
        }
        const uint32_t byte = q8_scale_byte(q8_amax<EPC>(y, [](float m) {
          m = run_maxf<16>(m);
          return EPC == 4 ? fmaxf(m, __shfl_xor(m, 16)) : m;
        }));
        const float qi = q8_inverse(byte);
        if (at < out.row_pitch) {
          if constexpr (EPC == 8)
            __builtin_nontemporal_store((uint64_t)q8_round4(y, qi) | (uint64_t)q8_round4(y + 4, qi) << 32,
                                        reinterpret_cast<uint64_t*>(q + at));
          else
            __builtin_nontemporal_store(q8_round4(y, qi), reinterpret_cast<uint32_t*>(q + at));
          if (at % kQBlock == 0) sc[at / kQBlock] = (uint8_t)byte;
        }
      }
      if (place < out.scale_pitch - blocks) sc[blocks + place] = kQOne;
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = (c * 64 * W + place) * EPC;
        if (at < H) {
          float v[EPC];
          cur.get(c, v);
#pragma unroll
          for (int e = 0; e < EPC; ++e) v[e] = v[e] * r * ga[c * EPC + e];
          Part::template put<true>((T*)out.y + t * H, at, H, v);
        }
      }
    }
    if constexpr (kAhead<W>) {
      cur = next;
      res = nres;
    }
  }
}

// dS + rstd (d - xh mean(d xh)), d = dY gamma.  65,536 x 2048 with dS: bf16 198 us, 5.4
// TB/s; fp32 415 us, 5.2 TB/s, the slabs' sum among them.
template <typename T, int W, int C, bool TAIL>
__global__ __launch_bounds__(kGroup<W>) void rms_rows_backward_kernel(
    const T* __restrict__ S, const float* __restrict__ gamma, const T* dY,
    const float* __restrict__ rstd, const T* dS, T* dX, float* __restrict__ part, int64_t N, int H) {
  using Part = RowPart<T, W, C, TAIL>;
  constexpr int EPC = Part::EPC;
  constexpr int RPG = kGroup<W> / (64 * W);
  __shared__ float red[2][1][16];
  const int place = threadIdx.x % (64 * W);
  const float inv = 1.f / H;
  float ga[Part::COLS], dg[Part::COLS];
  load_cols<EPC, W, C, TAIL>(gamma, place, H, ga);
#pragma unroll
  for (int i = 0; i < Part::COLS; ++i) dg[i] = 0.f;
  int half = 0;
  int64_t t = (int64_t)blockIdx.x * RPG + threadIdx.x / (64 * W);
  const int64_t step = (int64_t)gridDim.x * RPG;
  Part x, dy, ds;
  float r = 0.f;
  auto load = [&](int64_t u, Part& px, Part& pd, Part& ps, float& pr) {
    px.load(S + u * H, place, H);
    pd.load(dY + u * H, place, H);
    if (dS) ps.load(dS + u * H, place, H);
    pr = rstd[u];
  };
  if (kAhead<W> && t < N) load(t, x, dy, ds, r);
  for (; t < N; t += step) {
    Part x2, dy2, ds2;
    float r2 = 0.f;
    if constexpr (kAhead<W>) {
      if (t + step < N) load(t + step, x2, dy2, ds2, r2);
    } else {
      load(t, x, dy, ds, r);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      // lanes past the row's end hold x = dy = gamma = 0
      float v[EPC], d[EPC];
      x.get(c, v);
      dy.get(c, d);
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const int i = c * EPC + e;
        const float xh = v[e] * r;
        s[0] = fmaf(d[e] * ga[i], xh, s[0]);
        dg[i] = fmaf(d[e], xh, dg[i]);
      }
    }
    row_sums<W>(s, red, half);
    const float b = s[0] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
      if (at < H) {
        float v[EPC], d[EPC];
        x.get(c, v);
        dy.get(c, d);
#pragma unroll
        for (int e = 0; e < EPC; ++e) d[e] = r * fmaf(d[e], ga[c * EPC + e], -(v[e] * r * b));
        if (dS) {
          ds.get(c, v);
#pragma unroll
          for (int e = 0; e < EPC; ++e) d[e] += v[e];
        }
        Part::template put<true>(dX + t * H, at, H, d);
      }
    }
    if constexpr (kAhead<W>) {
      x = x2;
      dy = dy2;
      ds = ds2;
      r = r2;
    }
  }
  float* pg = part + (int64_t)blockIdx.x * H;
  if constexpr (RPG == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * 64 * W + place) * EPC;
#pragma unroll
      for (int e = 0; e < EPC; ++e)
        if (at + e < H) pg[at + e] = dg[c * EPC + e];
    }
  } else {
    // the work-group's waves add their shares up in order
    __shared__ float sum[64 * C * EPC];
    for (int w = 0; w < RPG; ++w) {
      if ((int)threadIdx.x >> 6 == w) {
#pragma unroll
        for (int i = 0; i < Part::COLS; ++i) {
          const int at = (i / EPC * 64 + place) * EPC + i % EPC;  // column of this lane's element i
          sum[at] = w == 0 ? dg[i] : sum[at] + dg[i];
        }
      }
      __syncthreads();
    }
    for (int h = threadIdx.x; h < H; h += kThreads) pg[h] = sum[h];
  }
}

// Rows wider than the registers hold, two or four bytes a lane at a time, their sums in 64
// bits throughout (a lane adds up to 256 numbers).  4096 x 20,000 bf16 with a residual into
// 8 bits: 353 us, 1.6 TB/s.
template <typename T, bool Q8>
__global__ __launch_bounds__(kThreads) void rms_forward_kernel(
    const T* X, const T* residual, const float* __restrict__ gamma, T* S, const RowsOut out,
    float* __restrict__ rstd, int64_t N, int H, float eps) {
  __shared__ double red[2][16];
  int half = 0;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const T* x = X + t * H;
    double q = 0.0;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      float v = Elem<T>::to_f(x[h]);
      if (residual) {
        const T sum = Elem<T>::from_f(v + Elem<T>::to_f(residual[t * H + h]));
        S[t * H + h] = sum;
        v = Elem<T>::to_f(sum);
      }
      q = fma((double)v, (double)v, q);
    }
    if (residual) x = S + t * H;  // each thread reads back what it wrote
    const double m = group_sum64(q, red, half) / H + (double)eps;
    const float r = 1.f / sqrtf((float)m);
    const double r64 = rstd64(m, r);
    if (threadIdx.x == 0) rstd[t] = r;
    if constexpr (Q8) {
      // a block of 128 columns in 32 lanes, four columns each; the sum's rows are
      // read by other threads than wrote them
      __syncthreads();
      uint8_t* qo = (uint8_t*)out.q + t * out.row_pitch;
      uint8_t* sc = (uint8_t*)out.s + t * out.scale_pitch;
      const int blocks = q8_blocks(H);
      for (int b = threadIdx.x / 32; b < blocks; b += kThreads / 32) {
        const int at = b * kQBlock + (threadIdx.x & 31) * 4;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float xe = at + e < H ? Elem<T>::to_f(x[at + e]) : 0.f, g = at + e < H ? gamma[at + e] : 0.f;
          v[e] = at + e < H ? exact8(xe * r * g, xe, g, r64) : 0.f;
        }
        const uint32_t byte = q8_scale_byte(q8_amax<4>(v, [](float m) {
          m = run_maxf<16>(m);
          return fmaxf(m, __shfl_xor(m, 16));
        }));
        *reinterpret_cast<uint32_t*>(qo + at) = q8_round4(v, q8_inverse(byte));
        if ((threadIdx.x & 31) == 0) sc[b] = (uint8_t)byte;
      }
      if ((int)threadIdx.x < out.scale_pitch - blocks) sc[blocks + threadIdx.x] = kQOne;
    } else {
      T* y = (T*)out.y;
      for (int h = threadIdx.x; h < H; h += kThreads)
        y[t * H + h] = Elem<T>::from_f(Elem<T>::to_f(x[h]) * r * gamma[h]);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rms_backward_kernel(
    const T* __restrict__ S, const float* __restrict__ gamma, const T* dY,
    const float* __restrict__ rstd, const T* dS, T* dX, float* __restrict__ part, int64_t N, int H) {
  __shared__ float red[kThreads / 64];
  float* pg = part + (int64_t)blockIdx.x * H;
  for (int h = threadIdx.x; h < H; h += kThreads) pg[h] = 0.f;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const T* x = S + t * H;
    const T* dy = dY + t * H;
    const float r = rstd[t];
    float b = 0.f;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const float d = Elem<T>::to_f(dy[h]), xh = Elem<T>::to_f(x[h]) * r;
      b = fmaf(d * gamma[h], xh, b);
      pg[h] = fmaf(d, xh, pg[h]);
    }
    b = group_sum(b, red) / H;
    for (int h = threadIdx.x; h < H; h += kThreads) {
      float d = r * fmaf(Elem<T>::to_f(dy[h]), gamma[h], -(Elem<T>::to_f(x[h]) * r * b));
      if (dS) d += Elem<T>::to_f(dS[t * H + h]);
      dX[t * H + h] = Elem<T>::from_f(d);
    }
  }
}

template <typename T, bool Q8>
hipError_t run_forward(const rms_plan_t& P, const void* X, const void* residual, const float* gamma,
                       void* S, const RowsOut& out, float* rstd, hipStream_t st) {
  const Holding h = holding(P.H, P.dtype);
  if (h.W == 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(P.N, kMaxRowGrid);
    rms_forward_kernel<T, Q8><<<grid, kThreads, 0, st>>>((const T*)X, (const T*)residual, gamma, (T*)S,
                                                         out, rstd, P.N, P.H, P.eps);
  } else {
    const int grid = row_groups(P.N, h.W);
    with_holding<T>(h, P.H, [&](auto w, auto c, auto tail) {
      rms_rows_forward_kernel<T, w.value, c.value, tail.value, Q8><<<grid, kGroup<w.value>, 0, st>>>(
          (const T*)X, (const T*)residual, gamma, (T*)S, out, rstd, P.N, P.H, P.eps);
    });
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run_backward(const rms_plan_t& P, const void* S, const float* gamma, const void* dY,
                        const float* rstd, const void* dS, void* dX, float* part, int slabs,
                        hipStream_t st) {
  const Holding h = holding(P.H, P.dtype);
  if (h.W == 0) {
    rms_backward_kernel<T><<<slabs, kThreads, 0, st>>>((const T*)S, gamma, (const T*)dY, rstd,
                                                       (const T*)dS, (T*)dX, part, P.N, P.H);
  } else {
    with_holding<T>(h, P.H, [&](auto w, auto c, auto tail) {
      rms_rows_backward_kernel<T, w.value, c.value, tail.value><<<slabs, kGroup<w.value>, 0, st>>>(
          (const T*)S, gamma, (const T*)dY, rstd, (const T*)dS, (T*)dX, part, P.N, P.H);
    });
  }
  return hipGetLastError();
}

bool plan_ok(const rms_plan_t* p) { return p != nullptr && p->magic == kRmsMagic; }

template <bool Q8>
int forward(const rms_plan_t* plan, const void* X, const void* residual, const float* gamma, void* S,
            const RowsOut& out, float* rstd, void* stream) {
  const rms_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!X || !gamma || !rstd || (Q8 ? !out.q || !out.s : !out.y)) return MOE_EINVAL;
  if ((residual == nullptr) != (S == nullptr)) return MOE_EINVAL;
  if (Q8 && ((uintptr_t)out.q % 16 || (uintptr_t)out.s % 4)) return MOE_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const hipError_t err = P.dtype == MOE_BF16
                             ? run_forward<bf16_t, Q8>(P, X, residual, gamma, S, out, rstd, st)
                             : run_forward<float, Q8>(P, X, residual, gamma, S, out, rstd, st);
  return err == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int rms_plan(int64_t N, int32_t H, int32_t dtype, float eps, rms_plan_t* out) {
  if (!out || N < 0 || H < 1 || !(eps > 0.f) || !std::isfinite(eps)) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (H > 65536 || N >= ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
  rms_plan_t p{};
  p.magic = kRmsMagic;
  p.dtype = dtype;
  p.N = N;
  p.H = H;
  p.eps = eps;
  p.row_pitch = q8_row_pitch(H);
  p.scale_pitch = q8_scale_pitch(H);
  p.bwd_workspace_bytes = std::min<int64_t>(N, kMaxSlabs) * H * sizeof(float);
  *out = p;
  return MOE_OK;
}

MOE_API int rms_forward(const rms_plan_t* plan, const void* X, const void* residual,
                        const float* gamma, void* S, void* Y, float* rstd, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  return forward<false>(plan, X, residual, gamma, S, RowsOut{Y, nullptr, nullptr, 0, 0}, rstd, stream);
}

MOE_API int rms_forward_q8(const rms_plan_t* plan, const void* X, const void* residual,
                           const float* gamma, void* S, void* Yq, void* Ys, float* rstd,
                           void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  return forward<true>(plan, X, residual, gamma, S,
                       RowsOut{nullptr, Yq, Ys, plan->row_pitch, plan->scale_pitch}, rstd, stream);
}

MOE_API int rms_backward(const rms_plan_t* plan, const void* S, const float* gamma, const void* dY,
                         const float* rstd, const void* dS, void* dX, float* dgamma,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const rms_plan_t& P = *plan;
  if (!dgamma) return MOE_EINVAL;
  if (P.N > 0 && (!S || !gamma || !dY || !rstd || !dX || !workspace)) return MOE_EINVAL;
  if (P.N > 0 && (uintptr_t)workspace % 256) return MOE_EINVAL;
  if (workspace_bytes < (size_t)P.bwd_workspace_bytes) return MOE_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int slabs = P.N > 0 ? slab_count(P.N, holding(P.H, P.dtype).W) : 0;
  if (P.N > 0) {
    // one work-group writes dgamma itself
    float* part = slabs == 1 ? dgamma : (float*)workspace;
    const hipError_t err = P.dtype == MOE_BF16
                               ? run_backward<bf16_t>(P, S, gamma, dY, rstd, dS, dX, part, slabs, st)
                               : run_backward<float>(P, S, gamma, dY, rstd, dS, dX, part, slabs, st);
    if (err != hipSuccess) return MOE_EHIP;
    if (slabs == 1) return MOE_OK;
  }
  slab_fold_kernel<<<(unsigned)ceil_div(P.H, 64), 64 * kFoldWaves, 0, st>>>(
      (const float*)workspace, slabs, P.H, P.H, dgamma, nullptr);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
