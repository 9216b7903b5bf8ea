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
#include <type_traits>

#include "device_common.hpp"
#include "lnorm.h"
#include "moe_internal.h"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kLnormMagic = 0x4c4e4d31u;  // "LNM1"
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
  __device__ static __forceinline__ void put(T* row, int at, int H, const float* v) {
    if (at + EPC <= H) {
      *reinterpret_cast<u32x4_any_t*>(row + at) = pack16(v, T());
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

// dgamma, dbeta = sum of the slabs' shares; latency (5 us at 512 slabs of 2048
// columns).  64 columns per work-group; wave w
// takes slabs w, w + 16, ... in order, then the waves' sums are added in order.
constexpr int kFoldWaves = 16;
__global__ __launch_bounds__(64 * kFoldWaves) void lnorm_fold_kernel(const float* __restrict__ part,
                                                                     int slabs, int H,
                                                                     float* __restrict__ dgamma,
                                                                     float* __restrict__ dbeta) {
  __shared__ float red[kFoldWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const int width = 2 * H;
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
Holding holding(const lnorm_plan_t& P) {
  const int epc = 16 / elem_bytes(P.dtype);
  const int64_t vecs = ceil_div(P.H, epc);
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
#define LNORM_CASE(w, c)                                                                            \
  if (h.W == w && h.C == c) {                                                                      \
    if (H % EPC) return f(integral_constant<int, w>(), integral_constant<int, c>(), bool_constant<true>()); \
    return f(integral_constant<int, w>(), integral_constant<int, c>(), bool_constant<false>());     \
  }
  LNORM_CASE(1, 1)
  LNORM_CASE(1, 2)
  LNORM_CASE(1, 4)
  LNORM_CASE(2, 4)
  LNORM_CASE(4, 4)
  LNORM_CASE(8, 4)
  if constexpr (EPC == 4) {
    LNORM_CASE(16, 4)
  }
#undef LNORM_CASE
}

template <typename T>
hipError_t run_forward(const lnorm_plan_t& P, const void* X, const float* gamma, const float* beta,
                       void* Y, float* mean, float* rstd, hipStream_t st) {
  const Holding h = holding(P);
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
  const Holding h = holding(P);
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
  const int slabs = P.N > 0 ? slab_count(P.N, holding(P).W) : 0;
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
  lnorm_fold_kernel<<<(unsigned)ceil_div(2 * (int64_t)P.H, 64), 64 * kFoldWaves, 0, st>>>(
      part, slabs, P.H, dgamma, dbeta);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
