// Routing by scores (include/route.h): selection of k experts per token by
// softmax or sigmoid scores with a bias and a group limit, the gates, and the
// gradient of the logits.
//
// One wave per token; lane l holds the logits of experts l, l + 64, ....  The
// selection runs k rounds; a round takes the largest remaining rank over the
// wave, then the lowest expert index that holds it.  Ranks are compared as
// unsigned integers that order as the values do (0: not to be selected), so
// any input, NaN included, gives k distinct experts.
#include <climits>
#include <cmath>

#include "device_common.hpp"
#include "moe_internal.h"
#include "route.h"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kRouteMagic = 0x52545331u;  // "RTS1"
constexpr int kRouteMaxE = 1024, kRouteMaxK = 64, kRouteMaxGroups = 64;
constexpr int kWaves = kThreads / 64;

struct RouteArgs {
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* gates;
  int64_t N;
  int E, k, sigmoid, n_group, topk_group, group_top, renorm;
  float scale;
};

// Unsigned integers in the order of the values; -0.0 as +0.0, never 0.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t o = b ^ ((b >> 63) ? ~0ull : 1ull << 63);
  return o ? o : 1ull;
}

__device__ __forceinline__ bool is_masked(float l) { return !(l > -INFINITY); }

template <int V>
__global__ __launch_bounds__(kThreads) void route_forward_kernel(const RouteArgs a) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + w;
  if (t >= a.N) return;  // whole wave leaves together; no work-group barrier below
  const float* row = a.logits + t * a.E;
  const int per = a.E / a.n_group;
  float l[V];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 64 * j;
    l[j] = e < a.E ? row[e] : -INFINITY;
    if (is_masked(l[j])) l[j] = -INFINITY;
    top = fmaxf(top, l[j]);
  }
  top = run_max<64>(top);
  // v_e, in 64 bits
  double v[V], z = 0.0;
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 1.0 / (1.0 + exp(-(double)l[j]));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = is_masked(l[j]) ? 0.0 : exp((double)l[j] - (double)top);
      z += v[j];
    }
    z = run_sum64<64>(z);
    const double inv = z > 0.0 ? 1.0 / z : 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= inv;
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 64 * j < a.E) v[j] += (double)a.bias[lane + 64 * j];
  }
  uint64_t rank[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
    rank[j] = lane + 64 * j >= a.E ? 0ull
              : is_masked(l[j])    ? order_of(-INFINITY)
                                   : order_of(a.bias ? v[j] : (double)l[j]);
  if (a.n_group > 1) {
    // group strengths: lane g sums group g's best values out of LDS
    double* val = smem + w * (kRouteMaxE + kRouteMaxGroups);
    double* strength = val + kRouteMaxE;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 64 * j < a.E) val[lane + 64 * j] = is_masked(l[j]) ? -INFINITY : v[j];
    wave_lds_order();
    double mine = -INFINITY;
    if (lane < a.n_group) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double x = val[lane * per + i];
        b2 = fmax(b2, fmin(b1, x));
        b1 = fmax(b1, x);
      }
      mine = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      strength[lane] = mine;
    }
    wave_lds_order();
    int before = 0;
    for (int h = 0; h < a.n_group; ++h)
      before += strength[h] > mine || (!(mine > strength[h]) && h < lane) ? 1 : 0;
    const uint64_t kept = __ballot(lane < a.n_group && before < a.topk_group);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 64 * j < a.E && !((kept >> ((lane + 64 * j) / per)) & 1)) rank[j] = 0ull;
  }
  int my_i = 0;
  for (int s = 0; s < a.k; ++s) {
    uint64_t best = 0ull;
#pragma unroll
    for (int j = 0; j < V; ++j) best = rank[j] > best ? rank[j] : best;
    best = run_max<64>(best);
    int at = INT_MAX;
#pragma unroll
    for (int j = V - 1; j >= 0; --j)
      if (rank[j] == best) at = lane + 64 * j;
    at = run_min<64>(at);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (at == lane + 64 * j) rank[j] = 0ull;
    if (lane == s) my_i = at;
  }
  // gates of the selected, lane s for slot s
  float ls = -INFINITY;
  if (lane < a.k) {
    ls = row[my_i];
    if (is_masked(ls)) ls = -INFINITY;
  }
  float g;
  if (a.renorm) {
    // scores relative to the largest one selected: no sum underflows
    const float m = run_max<64>(ls);
    const float c = a.sigmoid ? fminf(m, 0.f) : m;
    float r = 0.f;
    if (ls > -INFINITY)
      r = !a.sigmoid ? expf(ls - c) : ls < 0.f ? expf(ls - c) / (1.f + expf(ls)) : 1.f / (1.f + expf(-ls));
    const float sum = run_sum<64>(r);
    g = sum > 0.f ? a.scale * (r / sum) : 0.f;
  } else if (a.sigmoid) {
    g = a.scale * (ls < 0.f ? expf(ls) / (1.f + expf(ls)) : 1.f / (1.f + expf(-ls)));
  } else {
    g = ls > -INFINITY ? a.scale * (expf(ls - top) / (float)z) : 0.f;
  }
  if (lane < a.k) {
    a.idx[t * a.k + lane] = my_i;
    a.gates[t * a.k + lane] = g;
  }
}

struct RouteBwdArgs {
  const float* logits;
  const int32_t* idx;
  const float* dgates;
  float* dlogits;
  int64_t N;
  int E, k, sigmoid, renorm;
  float scale;
};

// One wave per token: lane s works out slot s's share, the row goes through
// LDS (zeros or the softmax's dense part, then the selected experts' shares
// added) and out.
template <int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const RouteBwdArgs a) {
  __shared__ float out[kWaves][kRouteMaxE];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + w;
  if (t >= a.N) return;  // whole wave leaves together
  const float* row = a.logits + t * a.E;
  const bool dense = !a.sigmoid && !a.renorm;
  float l[V], top = -INFINITY, z = 0.f;
  if (dense) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = lane + 64 * j < a.E ? row[lane + 64 * j] : -INFINITY;
      if (is_masked(l[j])) l[j] = -INFINITY;
      top = fmaxf(top, l[j]);
    }
    top = run_max<64>(top);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = is_masked(l[j]) ? 0.f : expf(l[j] - top);
      z += l[j];
    }
    z = run_sum<64>(z);
    z = z > 0.f ? 1.f / z : 0.f;
  }
  int e = -1;
  float ls = -INFINITY, dg = 0.f;
  if (lane < a.k) {
    e = a.idx[t * a.k + lane];
    if ((unsigned)e < (unsigned)a.E) {
      ls = row[e];
      if (is_masked(ls)) ls = -INFINITY;
    } else {
      e = -1;
    }
    dg = a.dgates[t * a.k + lane];
  }
  const bool live = ls > -INFINITY;
  if (!live) dg = 0.f;  // a gate fixed at 0
  const float sig = ls < 0.f ? expf(ls) / (1.f + expf(ls)) : 1.f / (1.f + expf(-ls));
  const float one_less = ls < 0.f ? 1.f / (1.f + expf(ls)) : expf(-ls) / (1.f + expf(-ls));
  float wgt = 0.f;  // g / scale
  if (a.renorm) {
    const float m = run_max<64>(ls);
    const float c = a.sigmoid ? fminf(m, 0.f) : m;
    float r = 0.f;
    if (live) r = !a.sigmoid ? expf(ls - c) : ls < 0.f ? expf(ls - c) / (1.f + expf(ls)) : sig;
    const float sum = run_sum<64>(r);
    wgt = sum > 0.f ? r / sum : 0.f;
  } else if (live) {
    wgt = a.sigmoid ? sig : expf(ls - top) * z;
  }
  // d_s = scale dg_s - sum_j g_j dg_j
  const float dot = a.sigmoid && !a.renorm ? 0.f : a.scale * run_sum<64>(wgt * dg);
  float d = wgt * (a.scale * dg - (dense ? 0.f : dot));
  if (a.sigmoid) d *= one_less;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (lane + 64 * j < a.E) out[w][lane + 64 * j] = dense ? -(l[j] * z) * dot : 0.f;
  wave_lds_order();
  if (e >= 0 && live) out[w][e] += d;
  wave_lds_order();
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (lane + 64 * j < a.E) a.dlogits[t * a.E + lane + 64 * j] = out[w][lane + 64 * j];
}

bool plan_ok(const route_plan_t* p) { return p != nullptr && p->magic == kRouteMagic; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int route_plan(int64_t N, int32_t E, int32_t k, int32_t score, int32_t n_group,
                       int32_t topk_group, int32_t group_top, int32_t renorm, float scale,
                       route_plan_t* out) {
  if (!out || N < 0 || E < 1 || k < 1 || k > E) return MOE_EINVAL;
  if (score != ROUTE_SOFTMAX && score != ROUTE_SIGMOID) return MOE_EINVAL;
  if (n_group < 1 || E % n_group || topk_group < 1 || topk_group > n_group) return MOE_EINVAL;
  if ((int64_t)k > (int64_t)topk_group * (E / n_group)) return MOE_EINVAL;
  if ((group_top != 1 && group_top != 2) || (renorm != 0 && renorm != 1)) return MOE_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MOE_EINVAL;
  if (E > kRouteMaxE || k > kRouteMaxK || n_group > kRouteMaxGroups || N >= ((int64_t)1 << 26))
    return MOE_EUNSUPPORTED;
  route_plan_t p{};
  p.magic = kRouteMagic;
  p.score = score;
  p.N = N;
  p.E = E;
  p.k = k;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.group_top = group_top;
  p.renorm = renorm;
  p.scale = scale;
  *out = p;
  return MOE_OK;
}

MOE_API int route_forward(const route_plan_t* plan, const float* logits, const float* bias,
                          int32_t* topk_idx, float* gates, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const route_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!logits || !topk_idx || !gates) return MOE_EINVAL;
  const RouteArgs a{logits, bias,      topk_idx,     gates,       P.N,      P.E,    P.k,
                    P.score, P.n_group, P.topk_group, P.group_top, P.renorm, P.scale};
  const unsigned grid = (unsigned)ceil_div(P.N, kWaves);
  const size_t lds = P.n_group > 1 ? kWaves * (kRouteMaxE + kRouteMaxGroups) * sizeof(double) : 0;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int vpl = (P.E + 63) / 64;
  if (vpl <= 1)
    route_forward_kernel<1><<<grid, kThreads, lds, st>>>(a);
  else if (vpl <= 4)
    route_forward_kernel<4><<<grid, kThreads, lds, st>>>(a);
  else
    route_forward_kernel<16><<<grid, kThreads, lds, st>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

MOE_API int route_backward(const route_plan_t* plan, const float* logits, const int32_t* topk_idx,
                           const float* dgates, float* dlogits, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const route_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!logits || !topk_idx || !dgates || !dlogits) return MOE_EINVAL;
  const RouteBwdArgs a{logits, topk_idx, dgates, dlogits, P.N, P.E, P.k, P.score, P.renorm, P.scale};
  const unsigned grid = (unsigned)ceil_div(P.N, kWaves);
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int vpl = (P.E + 63) / 64;
  if (vpl <= 1)
    route_backward_kernel<1><<<grid, kThreads, 0, st>>>(a);
  else if (vpl <= 4)
    route_backward_kernel<4><<<grid, kThreads, 0, st>>>(a);
  else
    route_backward_kernel<16><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
