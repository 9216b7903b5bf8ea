// Layer norm and its gradient (include/lnorm.h).
//
// Forward: one work-group per row; the mean, then the centred squares, then
// the output.  Backward: one work-group per slab of rows keeps the slab's
// shares of dgamma and dbeta in the workspace and writes dX row by row; a
// second launch adds the slabs up in order.
#include <algorithm>
#include <cmath>

#include "device_common.hpp"
#include "lnorm.h"
#include "moe_internal.h"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kLnormMagic = 0x4c4e4d31u;  // "LNM1"
constexpr int kMaxSlabs = 512;
constexpr unsigned kMaxRowGrid = 1u << 16;

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

// part: [slab][2][H], this slab's shares of dgamma and dbeta.
template <typename T>
__global__ __launch_bounds__(kThreads) void lnorm_backward_kernel(
    const T* __restrict__ X, const float* __restrict__ gamma, const T* dY,
    const float* __restrict__ mean, const float* __restrict__ rstd, T* dX,
    float* __restrict__ part, int64_t N, int H) {
  __shared__ float red[kThreads / 64];
  float* pg = part + (int64_t)blockIdx.x * 2 * H;
  float* pb = pg + H;
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

// dgamma, dbeta = sum of the slabs' shares, slabs in order.  64 columns per
// work-group, its waves taking every fourth slab.
__global__ __launch_bounds__(kThreads) void lnorm_fold_kernel(const float* __restrict__ part,
                                                              int slabs, int H,
                                                              float* __restrict__ dgamma,
                                                              float* __restrict__ dbeta) {
  __shared__ float red[kThreads];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  const int width = 2 * H;
  float s = 0.f;
  if (c < width)
    for (int p = w; p < slabs; p += kThreads / 64) s += part[(int64_t)p * width + c];
  red[threadIdx.x] = s;
  __syncthreads();
  if (w != 0 || c >= width) return;
#pragma unroll
  for (int v = 1; v < kThreads / 64; ++v) s += red[v * 64 + threadIdx.x];
  if (c < H)
    dgamma[c] = s;
  else if (dbeta)
    dbeta[c - H] = s;
}

int slabs_of(int64_t N) { return (int)std::min<int64_t>(N, kMaxSlabs); }

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
  p.bwd_workspace_bytes = (int64_t)slabs_of(N) * 2 * H * sizeof(float);
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
  const unsigned grid = (unsigned)std::min<int64_t>(P.N, kMaxRowGrid);
  if (P.dtype == MOE_BF16)
    lnorm_forward_kernel<bf16_t><<<grid, kThreads, 0, st>>>(
        (const bf16_t*)X, gamma, beta, (bf16_t*)Y, mean, rstd, P.N, P.H, P.eps);
  else
    lnorm_forward_kernel<float><<<grid, kThreads, 0, st>>>((const float*)X, gamma, beta, (float*)Y,
                                                           mean, rstd, P.N, P.H, P.eps);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
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
  const int slabs = slabs_of(P.N);
  float* part = (float*)workspace;
  if (P.N > 0) {
    if (P.dtype == MOE_BF16)
      lnorm_backward_kernel<bf16_t><<<slabs, kThreads, 0, st>>>(
          (const bf16_t*)X, gamma, (const bf16_t*)dY, mean, rstd, (bf16_t*)dX, part, P.N, P.H);
    else
      lnorm_backward_kernel<float><<<slabs, kThreads, 0, st>>>(
          (const float*)X, gamma, (const float*)dY, mean, rstd, (float*)dX, part, P.N, P.H);
    if (hipGetLastError() != hipSuccess) return MOE_EHIP;
  }
  lnorm_fold_kernel<<<(unsigned)ceil_div(2 * (int64_t)P.H, 64), kThreads, 0, st>>>(part, slabs, P.H,
                                                                                  dgamma, dbeta);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
