// Distillation from a teacher's top logits through the vocabulary projection
// (include/distill.h).
//
// The scheme is the cross-entropy's (cce.hip, gemm_cce.hip): strips of logits,
// here scaled by 1 / T, formed twice and never kept.  Strips, tiles and the
// order of dX's sums have rules of their own (kd_shapes.hpp, strip_of,
// dx_ranges).  What the teacher's list adds is sparse, K of V entries per token:
// the forward pass takes their logits as dot products of gathered rows of W, and
// the backward pass overwrites their values in the strip's logit gradient from
// those logits, in fp32 before the one rounding.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.hpp"
#include "distill.h"
#include "kd_shapes.hpp"
#include "moe_internal.h"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kKdMagic = 0x4b445331u;  // "KDS1"
constexpr int kMaxList = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kDots = 4;             // rows of W a wave multiplies at a time

struct KdArgs {
  const bf16_t* X;
  const bf16_t* W;
  const int32_t* t_idx;
  const float* t_logit;
  const float* lse;
  int64_t N, V;
  int H, K;
  float T;
};

// The teacher's probabilities of token t's list: lane l holds entries l + 64 q,
// q < kPer (K <= 64 kPer).  Differences to the largest logit are divided by T,
// not the logits: a quotient of a finite logit may overflow where T < 1.
// p is -1 for an entry that is no part of the list; returns whether any is.
template <int kPer>
__device__ __forceinline__ bool list_softmax(const KdArgs& a, int64_t t, int lane, int32_t (&id)[kPer],
                                             float (&p)[kPer], float (&logp)[kPer]) {
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int j = lane + 64 * q;
    id[q] = -1;
    logp[q] = -INFINITY;
    if (j < a.K) {
      const int32_t v = a.t_idx[t * a.K + j];
      const float l = a.t_logit[t * a.K + j];
      if (v >= 0 && v < a.V && l > -INFINITY) {
        id[q] = v;
        logp[q] = l;
      }
    }
    top = fmaxf(top, logp[q]);
  }
  top = run_maxf<64>(top);
  const bool any = top > -INFINITY;
  float z = 0.f;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    logp[q] = (logp[q] - top) / a.T;
    p[q] = id[q] >= 0 ? expf(logp[q]) : 0.f;
    z += p[q];
  }
  z = run_sum<64>(z);
  const float logz = any ? logf(z) : 0.f;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    p[q] = id[q] >= 0 ? p[q] / z : -1.f;
    logp[q] -= logz;
  }
  return any;
}

// Adds (a, b), b = sum of exp(y - a), to (m, z): the larger maximum stays, the
// other's sum is rescaled by one exponential.  A slice past the vocabulary has
// a = -inf.
__device__ __forceinline__ void fold(float a, float b, float& m, float& z) {
  if (a == -INFINITY) return;
  const float far = __expf(-fabsf(a - m));
  z = a > m ? fmaf(z, far, b) : fmaf(b, far, z);
  m = fmaxf(m, a);
}

// Folds a strip's slice pairs into the running state (m, z).  A work-group takes
// 16 tokens, 16 threads each: every thread folds each 16th slice in order, then
// one thread a token its state and the 16 results in order.  The last strip's are
// folded by kd_loss_kernel.  Latency bounds it: 64 slices of 8192 tokens 5.1 us.
constexpr int kFoldTokens = 16, kFoldWays = kThreads / kFoldTokens, kFoldAhead = 4;
__global__ __launch_bounds__(kThreads) void kd_fold_kernel(
    const float* __restrict__ pmax, const float* __restrict__ psum, int nslices, int64_t N,
    float* __restrict__ m, float* __restrict__ z, int first) {
  __shared__ float ms[kFoldWays][kFoldTokens], zs[kFoldWays][kFoldTokens];
  const int i = threadIdx.x % kFoldTokens, way = threadIdx.x / kFoldTokens;
  const int64_t t = (int64_t)blockIdx.x * kFoldTokens + i, tc = min(t, N - 1);
  float mm = -INFINITY, zz = 0.f;
  for (int s0 = way; s0 < nslices; s0 += kFoldAhead * kFoldWays) {
    float a[kFoldAhead], b[kFoldAhead];
#pragma unroll
    for (int u = 0; u < kFoldAhead; ++u) {
      const int s = min(s0 + u * kFoldWays, nslices - 1);
      a[u] = pmax[(int64_t)s * N + tc];
      b[u] = psum[(int64_t)s * N + tc];
    }
#pragma unroll
    for (int u = 0; u < kFoldAhead; ++u)
      if (s0 + u * kFoldWays < nslices) fold(a[u], b[u], mm, zz);
  }
  ms[way][i] = mm;
  zs[way][i] = zz;
  __syncthreads();
  if (way != 0 || t >= N) return;
  mm = first ? -INFINITY : m[t];
  zz = first ? 0.f : z[t];
#pragma unroll
  for (int v = 0; v < kFoldWays; ++v) fold(ms[v][i], zs[v][i], mm, zz);
  m[t] = mm;
  z[t] = zz;
}

// One work-group per token: the last strip's slices folded in, which gives lse,
// the list entries' logits, a wave taking kDots rows of W at a time, then the
// loss.  (With a fold of its own launch 777 x 512 x 20,000 takes 142 us instead of
// 136, 25 x 256 x 43,363 56 and 50.)  Bound by the gathered rows: 8192 tokens, 32
// entries of 7168, 590 us for 3.8 GB (6.4 TB/s, partly from cache), 0.8% of the
// pass.
template <int kPer>
__global__ __launch_bounds__(kThreads) void kd_loss_kernel(
    const KdArgs a, const float* __restrict__ pmax, const float* __restrict__ psum, int nslices,
    const float* __restrict__ m, const float* __restrict__ z, int first, float* __restrict__ lse,
    float* __restrict__ loss, float* __restrict__ y_top) {
  __shared__ float ys[kMaxList], ms[kWaves], zs[kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  float mm = -INFINITY, zz = 0.f;
  for (int s = threadIdx.x; s < nslices; s += kThreads)
    fold(pmax[(int64_t)s * a.N + t], psum[(int64_t)s * a.N + t], mm, zz);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {  // the same way round for both lanes of a pair
    const float m2 = __shfl_xor(mm, o), z2 = __shfl_xor(zz, o);
    fold(m2, z2, mm, zz);
  }
  ms[w] = mm;
  zs[w] = zz;
  const u32x4_t* x = reinterpret_cast<const u32x4_t*>(a.X + t * a.H);
  for (int j0 = w * kDots; j0 < a.K; j0 += kWaves * kDots) {
    const u32x4_t* row[kDots];
    bool real[kDots];
    float acc[kDots];
#pragma unroll
    for (int u = 0; u < kDots; ++u) {
      const int32_t v = j0 + u < a.K ? a.t_idx[t * a.K + j0 + u] : -1;
      real[u] = v >= 0 && v < a.V && a.t_logit[t * a.K + j0 + u] > -INFINITY;
      row[u] = reinterpret_cast<const u32x4_t*>(a.W + (int64_t)(real[u] ? v : 0) * a.H);
      acc[u] = 0.f;
    }
    for (int c = lane; c < a.H / 8; c += 64) {
      u32x4_t raw[kDots];
#pragma unroll
      for (int u = 0; u < kDots; ++u) raw[u] = row[u][c];
      float xv[8], wv[8];
      unpack16(x[c], xv, bf16_t());
#pragma unroll
      for (int u = 0; u < kDots; ++u) {
        unpack16(raw[u], wv, bf16_t());
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[u] = fmaf(xv[e], wv[e], acc[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kDots; ++u) {
      acc[u] = real[u] ? run_sum<64>(acc[u]) : 0.f;
      if (lane == 0 && j0 + u < a.K) {
        ys[j0 + u] = acc[u];
        y_top[t * a.K + j0 + u] = acc[u];
      }
    }
  }
  __syncthreads();
  if (w != 0) return;
  mm = first ? -INFINITY : m[t];
  zz = first ? 0.f : z[t];
#pragma unroll
  for (int v = 0; v < kWaves; ++v) fold(ms[v], zs[v], mm, zz);
  const float lse_t = mm + logf(zz);
  if (lane == 0) lse[t] = lse_t;
  int32_t id[kPer];
  float p[kPer], logp[kPer];
  const bool any = list_softmax(a, t, lane, id, p, logp);
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (p[q] > 0.f) s = fmaf(p[q], logp[q] - (ys[lane + 64 * q] / a.T - lse_t), s);
  s = run_sum<64>(s);
  if (lane == 0) loss[t] = any ? a.T * a.T * s : 0.f;
}

// The teacher's part of the strip's logit gradient, a wave per token: for each
// list entry in the strip G[t][i - v0] = dl (q - the sum of p over the entries
// with its index), dl = dloss T, from the entry's own logit (entries of one
// index write the same value); a token whose list is empty gets a row of zeros.
// Latency: 4.9 us, 8192 tokens of 32 entries 5.6.  (The sums formed once for all
// strips by a launch of their own: 734 x 384 x 1006 49.8 us instead of 46.5.)
template <int kPer>
__global__ __launch_bounds__(kThreads) void kd_entries_kernel(const KdArgs a, const float* __restrict__ y_top,
                                                              const float* __restrict__ dloss, int64_t v0,
                                                              int w, bf16_t* __restrict__ G, int ldg) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= a.N) return;  // whole wave leaves together
  int32_t id[kPer];
  float p[kPer], logp[kPer];
  bf16_t* row = G + t * ldg;
  if (!list_softmax(a, t, lane, id, p, logp)) {
    for (int c = lane; c < (w + 255) / 256 * 32; c += 64)  // as wide as the products read it
      reinterpret_cast<u32x4_t*>(row)[c] = u32x4_t{0u, 0u, 0u, 0u};
    return;
  }
  bool in[kPer], some = false;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    in[q] = id[q] >= v0 && id[q] < v0 + w;
    some |= in[q];
  }
  if (!__any(some)) return;
  float sum[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) sum[q] = 0.f;
#pragma unroll
  for (int r = 0; r < kPer; ++r)
    for (uint64_t left = __ballot(in[r]); left; left &= left - 1) {  // equal ones are in the strip too
      const int l = __builtin_ctzll(left);
      const int32_t v = __builtin_amdgcn_readlane(id[r], l);
      const float pv = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p[r]), l));
#pragma unroll
      for (int q = 0; q < kPer; ++q) sum[q] += id[q] == v ? pv : 0.f;
    }
  const float dl = dloss[t] * a.T, lse = a.lse[t];
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (in[q]) row[id[q] - v0] = f2bf(dl * (expf(y_top[t * a.K + lane + 64 * q] / a.T - lse) - sum[q]));
}

// dX [N][H] = bf16 of the slots' sums: a wave adds a quarter of the slots in
// order, then the waves' sums are added in order.  4 values per lane.
__global__ __launch_bounds__(kThreads) void kd_fold_dx_kernel(const float* __restrict__ sums,
                                                              int slots, int64_t n4,
                                                              bf16_t* __restrict__ dX) {
  __shared__ f32x4_t part[kWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t i = (int64_t)blockIdx.x * 64 + lane, ic = min(i, n4 - 1);
  const int share = (slots + kWaves - 1) / kWaves;
  f32x4_t s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int v = w * share; v < min(slots, (w + 1) * share); ++v)
    s += reinterpret_cast<const f32x4_t*>(sums)[v * n4 + ic];
  part[w][lane] = s;
  __syncthreads();
  if (w != 0 || i >= n4) return;
#pragma unroll
  for (int v = 1; v < kWaves; ++v) s += part[v][lane];
  reinterpret_cast<ushort4*>(dX)[i] = make_ushort4(f2bf(s[0]), f2bf(s[1]), f2bf(s[2]), f2bf(s[3]));
}

// The same of one sum; 4 values per thread.
__global__ __launch_bounds__(kThreads) void kd_round_dx_kernel(const float* __restrict__ sum,
                                                               int64_t n4, bf16_t* __restrict__ dX) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n4) return;
  const f32x4_t s = reinterpret_cast<const f32x4_t*>(sum)[i];
  reinterpret_cast<ushort4*>(dX)[i] = make_ushort4(f2bf(s[0]), f2bf(s[1]), f2bf(s[2]), f2bf(s[3]));
}

// Calls f with the list entries per lane as a template argument.
template <typename F>
void with_list(int K, F f) {
  if (K <= 64) return f(std::integral_constant<int, 1>());
  return f(std::integral_constant<int, kMaxList / 64>());
}

// Columns of a strip's buffers: whole 256-column logit tiles.
int strip_cols(int64_t V, int strip) {
  return (int)std::min<int64_t>(strip, ceil_div(V, 256) * 256);
}

// The backward pass's strips: v_chunk, times what KD_STRIP_BYTES leaves (and
// 32-bit offsets into W), evened out over the vocabulary.  777 x 512 x 20,000 at
// v_chunk 4096 takes 136 us so and 281 with strips of v_chunk, at 8192 100 x 2048
// x 50,000 225 and 484, 2000 x 2048 x 50,000 1,671 and 1,838.
int strip_of(int64_t N, int64_t V, int H, int v_chunk) {
  const int64_t cols = ceil_div(V, 256) * 256;
  const int64_t most = std::min<int64_t>((int64_t)KD_STRIP_BYTES / 2 / std::max<int64_t>(N, 1),
                                         (((int64_t)1 << 30) - 1) / H);
  if (cols <= most) return (int)(ceil_div(cols, v_chunk) * v_chunk);
  const int64_t strips = ceil_div(V, std::max<int64_t>(most / v_chunk, 1) * v_chunk);
  return (int)(ceil_div(ceil_div(V, strips), v_chunk) * v_chunk);
}

// dX's ranges: with fewer than 256 tiles of dX, as many sums side by side as
// fill the CUs once, each range at least 512 entries (16 K-tiles).  Depends on
// N, H and V alone, so dX does not depend on the strips.  The passes above take
// 460, 742 and 2,114 us with one sum.
struct DxRanges {
  int range, slots;
};
DxRanges dx_ranges(int64_t N, int64_t V, int H) {
  const int64_t tiles = ceil_div(N, 256) * (H / (H % 256 == 0 ? 256 : 128));
  const int64_t want = 256 / tiles;
  if (want < 2) return {0, 1};
  const int64_t span = std::min<int64_t>(V, (int64_t)KD_STRIP_BYTES / 2 / N);
  const int range = (int)std::max<int64_t>(512, ceil_div(ceil_div(span, want), 256) * 256);
  return {range, (int)std::min(want, ceil_div(V, range))};
}

struct KdLayout {
  size_t pmax = 0, psum = 0, m = 0, z = 0;      // forward
  size_t g = 0, dx = 0;                         // backward
  size_t total = 0;
};

// cols: the pass's strip columns (strip_cols).
KdLayout kd_layout(int64_t N, int64_t V, int H, int cols, bool backward) {
  KdLayout L;
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) & ~(size_t)255;
    return o;
  };
  const size_t n = (size_t)N;
  if (!backward) {
    const size_t nsl = (size_t)cols / kCceSlice;
    L.pmax = take(nsl * n * 4);
    L.psum = take(nsl * n * 4);
    L.m = take(n * 4);
    L.z = take(n * 4);
  } else {
    L.g = take(n * (size_t)cols * 2);
    L.dx = take((size_t)dx_ranges(N, V, H).slots * n * (size_t)H * 4);
  }
  L.total = cur;
  return L;
}

bool plan_ok(const kd_plan_t* p) { return p != nullptr && p->magic == kKdMagic; }

// The matrices move in vectors of 16 bytes.
bool off16(const void* a, const void* b) { return ((uintptr_t)a | (uintptr_t)b) % 16 != 0; }

KdArgs kd_args(const kd_plan_t& P, const void* X, const void* W, const int32_t* t_idx,
               const float* t_logit, const float* lse) {
  return KdArgs{(const bf16_t*)X, (const bf16_t*)W, t_idx, t_logit, lse, P.N, P.V, P.H, P.K,
                P.temperature};
}

}  // namespace
}  // namespace moe

using namespace moe;

#define KD_CHECK(call)                         \
  do {                                         \
    if ((call) != hipSuccess) return MOE_EHIP; \
  } while (0)

MOE_API int kd_plan(int64_t N, int32_t H, int64_t V, int32_t v_chunk, int32_t K, float temperature,
                    int32_t dtype, int32_t dw_dtype, kd_plan_t* out) {
  if (!out || N < 0 || V < 1 || H < 1 || v_chunk < 1 || K < 1) return MOE_EINVAL;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature)) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (dw_dtype != MOE_F32 && dw_dtype != MOE_BF16) return MOE_EINVAL;
  if (dtype != MOE_BF16 || H % 128 != 0 || v_chunk % 256 != 0 || K > kMaxList) return MOE_EUNSUPPORTED;
  const int64_t lim = (int64_t)1 << 30;
  if (N >= lim || N * (int64_t)H >= lim || N * (int64_t)v_chunk >= lim ||
      (int64_t)v_chunk * H >= lim || V >= 2 * lim)
    return MOE_EUNSUPPORTED;
  kd_plan_t p{};
  p.magic = kKdMagic;
  p.dtype = dtype;
  p.N = N;
  p.V = V;
  p.H = H;
  p.v_chunk = v_chunk;
  p.K = K;
  p.temperature = temperature;
  p.dw_dtype = dw_dtype;
  p.strip = strip_of(N, V, H, v_chunk);
  p.S = N == 0 ? 0 : (int32_t)ceil_div(V, p.strip);
  p.strip_bound_bytes = N * std::min<int64_t>(p.strip, V) * 2;
  if (N > 0) {  // without tokens there are no tiles to count, and no workspaces
    const int fcols = strip_cols(V, kd_forward_strip(N, V, H)), cols = strip_cols(V, p.strip);
    p.fwd_workspace_bytes = (int64_t)kd_layout(N, V, H, fcols, false).total;
    p.bwd_workspace_bytes = (int64_t)kd_layout(N, V, H, cols, true).total;
  }
  *out = p;
  return MOE_OK;
}

MOE_API int kd_forward(const kd_plan_t* plan, const void* X, const void* W, const int32_t* t_idx,
                       const float* t_logit, float* loss, float* lse, float* y_top,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const kd_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!X || !W || !t_idx || !t_logit || !loss || !lse || !y_top || !workspace) return MOE_EINVAL;
  if ((uintptr_t)workspace % 256 || off16(X, W)) return MOE_EINVAL;
  if (workspace_bytes < (size_t)P.fwd_workspace_bytes) return MOE_EWORKSPACE;
  const int strip = kd_forward_strip(P.N, P.V, P.H);
  const KdLayout L = kd_layout(P.N, P.V, P.H, strip_cols(P.V, strip), false);
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  float* pmax = (float*)(ws + L.pmax);
  float* psum = (float*)(ws + L.psum);
  (void)hipGetLastError();
  for (int64_t v0 = 0; v0 < P.V; v0 += strip) {
    const int w = (int)std::min<int64_t>(strip, P.V - v0);
    KD_CHECK(gemm_kd_logits(false, X, (const bf16_t*)W + v0 * P.H, P.N, P.H, w, P.temperature,
                            pmax, psum, nullptr, nullptr, nullptr, 0, st));
    const int nsl = (int)ceil_div(w, 256) * (256 / kCceSlice);
    float *m = (float*)(ws + L.m), *z = (float*)(ws + L.z);
    if (v0 + w < P.V)
      kd_fold_kernel<<<(unsigned)ceil_div(P.N, kFoldTokens), kThreads, 0, st>>>(pmax, psum, nsl, P.N, m, z, v0 == 0);
    else
      with_list(P.K, [&](auto per) {
        kd_loss_kernel<per.value><<<(unsigned)P.N, kThreads, 0, st>>>(
            kd_args(P, X, W, t_idx, t_logit, nullptr), pmax, psum, nsl, m, z, v0 == 0, lse, loss, y_top);
      });
    KD_CHECK(hipGetLastError());
  }
  return MOE_OK;
}

MOE_API int kd_backward(const kd_plan_t* plan, const void* X, const void* W, const int32_t* t_idx,
                        const float* t_logit, const float* lse, const float* y_top,
                        const float* dloss, void* dX, void* dW, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const kd_plan_t& P = *plan;
  if (!dW) return MOE_EINVAL;
  if (P.N > 0 && (!X || !W || !t_idx || !t_logit || !lse || !y_top || !dloss || !dX || !workspace))
    return MOE_EINVAL;
  if (P.N > 0 && ((uintptr_t)workspace % 256 || off16(X, W) || off16(dX, dW))) return MOE_EINVAL;
  if (workspace_bytes < (size_t)P.bwd_workspace_bytes) return MOE_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  const size_t dwb = P.dw_dtype == MOE_BF16 ? 2 : 4;
  (void)hipGetLastError();
  if (P.N == 0) {  // no tokens: dW = 0
    KD_CHECK(launch_fill_zero(dW, (size_t)P.V * P.H * dwb, st));
    return MOE_OK;
  }
  const int cols = strip_cols(P.V, P.strip);
  const KdLayout L = kd_layout(P.N, P.V, P.H, cols, true);
  const DxRanges R = dx_ranges(P.N, P.V, P.H);
  char* ws = (char*)workspace;
  bf16_t* G = (bf16_t*)(ws + L.g);
  float* dx = (float*)(ws + L.dx);
  const KdArgs a = kd_args(P, X, W, t_idx, t_logit, lse);
  for (int s = 0; s < P.S; ++s) {
    const int64_t v0 = (int64_t)s * P.strip;
    const int w = (int)std::min<int64_t>(P.strip, P.V - v0);
    const bf16_t* Ws = (const bf16_t*)W + v0 * P.H;
    KD_CHECK(gemm_kd_logits(true, X, Ws, P.N, P.H, w, P.temperature, nullptr, nullptr, lse, dloss,
                            G, cols, st));
    with_list(P.K, [&](auto per) {
      kd_entries_kernel<per.value><<<(unsigned)ceil_div(P.N, kWaves), kThreads, 0, st>>>(a, y_top, dloss, v0,
                                                                                        w, G, cols);
    });
    KD_CHECK(hipGetLastError());
    if (R.slots > 1)
      KD_CHECK(gemm_kd_dx(G, cols, Ws, P.N, P.H, w, v0, dx, R.range, R.slots, st));
    else
      KD_CHECK(gemm_cce_dx(G, cols, Ws, P.N, P.H, w, dx, s == 0, st));
    KD_CHECK(gemm_kd_dw(P.dw_dtype == MOE_BF16, G, cols, X, P.N, P.H, w, (char*)dW + v0 * P.H * dwb, st));
  }
  const int64_t n4 = P.N * P.H / 4;
  if (R.slots > 1)
    kd_fold_dx_kernel<<<(unsigned)ceil_div(n4, 64), kThreads, 0, st>>>(dx, R.slots, n4, (bf16_t*)dX);
  else
    kd_round_dx_kernel<<<(unsigned)ceil_div(n4, kThreads), kThreads, 0, st>>>(dx, n4, (bf16_t*)dX);
  KD_CHECK(hipGetLastError());
  return MOE_OK;
}
