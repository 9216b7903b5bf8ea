// Routing by scores (include/route.h): selection of k experts per token by
// softmax or sigmoid scores with a bias and a group limit, the gates, and the
// gradient of the logits.
//
// The bytes are few (a row of logits in, k pairs out), so the selection's
// instructions decide.  A token takes 16 lanes of up to 16 experts each (a wave
// past 256 experts or 16 slots), so that a wave selects for four tokens at once
// and every reduction stays inside a row of lanes, in DPP operands.  The lanes'
// largest ranks give a threshold that few experts pass; those, one a lane, count
// the ones before them.  Where more pass than there are lanes (many equal ones,
// or more slots than a row's lanes) the selection runs k rounds: the largest
// remaining rank, then the lowest expert that holds it.
//
// Ranks are the values, -inf for a masked expert and NaN for what is not to be
// selected, which no maximum and no comparison takes: any input gives k
// distinct experts.  Logits rank exactly as they are.  Scores with a bias, and
// group strengths, are formed in 32 bits first; where two values that decide
// something are nearer than their error bound, the candidates, or the token by
// its whole wave (route_exact), are ranked again in 64 bits.
#include <algorithm>
#include <cmath>
#include <type_traits>

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
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t o = b ^ ((b >> 31) ? ~0u : 1u << 31);
  return o ? o : 1u;
}
// The value that ranks as o (o != 0).
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 1u << 31 : ~0u));
}

__device__ __forceinline__ bool is_masked(float l) { return !(l > -INFINITY); }

// The hardware exponential's argument is rounded (a step per unit of it) and
// its result within a step, as the reciprocal's.
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// A selected expert's score: relative to exp(c), c <= 0 and c = the largest
// logit if that is below 0, so that the largest neither under- nor overflows
// (c = 0: the score itself); and 1 - sigmoid.
__device__ __forceinline__ float sigmoid_rel(float l, float c, float* one_less) {
  const float r = rcp(1.f + __expf(-fabsf(l)));
  const float far = __expf(-fabsf(l)) * r;
  if (one_less) *one_less = l < 0.f ? r : far;
  return l < 0.f ? __expf(l - c) * r : r;
}

// How near two scores (group strengths: sums of two) may be for 32 bits to tell
// them apart.  A sigmoid is off by less than 3e-7 (0.25 of its exponential's
// relative error of 1.2e-7 + 6e-8 |l|, |l| s (1 - s) <= 0.23; a step each of
// 1 + x and the reciprocal).  A softmax's own error is no larger, but the sum
// of up to 1024 terms is off by up to 22 roundings, 1.3e-6, which moves two
// scores apart by as much of their distance.  Adding the bias rounds by half a step of the result.
__device__ __forceinline__ float nearness(int sigmoid, float x) {
  return (sigmoid ? 7e-7f : 2e-6f) * (1.f + fabsf(x));
}

// The sum of exp(l - top) in 64 bits over a row, G lanes taking every G-th expert
// from `first` on.  (A loop: unrolled, its registers would halve the waves.)
template <int G>
__device__ __forceinline__ double softmax_sum64(const float* row, int E, int first, float top) {
  double z = 0.0;
#pragma unroll 2
  for (int e = first; e < E; e += G) z += is_masked(row[e]) ? 0.0 : exp((double)row[e] - (double)top);
#pragma unroll
  for (int o = 1; o < G; o <<= 1) z += __shfl_xor(z, o);
  return z;
}

// One token's selection in 64 bits by the whole wave (every lane of it calls):
// lane s returns slot s's expert.  lds: E + n_group doubles of the wave's own.
// The values stay there, not in registers: few tokens come here, and the kernel
// around it is to keep its waves (E > 512 with a bias: 2 a SIMD with registers).
__device__ __forceinline__ int route_exact(const RouteArgs& a, int64_t t, double* lds) {
  const int lane = threadIdx.x & 63;
  const float* row = a.logits + t * a.E;
  float top = -INFINITY;
  double inv = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 64) top = fmaxf(top, row[e]);
    top = run_maxf<64>(top);
    const double z = softmax_sum64<64>(row, a.E, lane, top);
    inv = z > 0.0 ? 1.0 / z : 0.0;
  }
  wave_lds_order();  // earlier uses of the wave's LDS are done
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float l = row[e];
    double v = -INFINITY;
    if (!is_masked(l)) {
      v = exp(a.sigmoid ? -(double)l : (double)l - (double)top);
      v = a.sigmoid ? 1.0 / (1.0 + v) : v * inv;
      if (a.bias) v = fmax(v + (double)a.bias[e], -INFINITY);  // a NaN bias masks, as in 32 bits
    }
    lds[e] = v;
  }
  const int per = a.E / a.n_group;
  uint64_t kept = ~0ull;
  if (a.n_group > 1) {
    // group strengths: lane g sums group g's best values
    double* strength = lds + a.E;
    wave_lds_order();
    double mine = -INFINITY;
    if (lane < a.n_group) {
      double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 8
      for (int i = 0; i < per; ++i) {
        const double x = lds[lane * per + i];
        b2 = fmax(b2, fmin(b1, x));
        b1 = fmax(b1, x);
      }
      mine = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      strength[lane] = mine;
    }
    wave_lds_order();
    int before = 0;
    for (int h = 0; h < a.n_group; ++h)
      before += strength[h] > mine || (strength[h] == mine && h < lane) ? 1 : 0;
    kept = __ballot(lane < a.n_group && before < a.topk_group);
  }
  // a lane's experts from here on are its own: ranks in the values' place, and
  // the largest, at the lowest expert, in registers
  uint64_t* rank = reinterpret_cast<uint64_t*>(lds);
  uint64_t own = 0ull;
  int own_e = 0;
  for (int e = lane; e < a.E; e += 64) {
    const double x = lds[e];
    const bool in = a.n_group == 1 || (kept >> (e / per)) & 1;
    const uint64_t r = in ? order_of(a.bias || x == -INFINITY ? x : (double)row[e]) : 0ull;
    rank[e] = r;
    if (r > own) own = r, own_e = e;
  }
  int my_i = 0;
  for (int s = 0; s < a.k; ++s) {
    // the largest over the wave, its high half first
    const uint32_t hi = run_maxu<64>((uint32_t)(own >> 32));
    const uint32_t lo = run_maxu<64>((uint32_t)(own >> 32) == hi ? (uint32_t)own : 0u);
    const bool holds = own == ((uint64_t)hi << 32 | lo);
    const uint32_t at = run_minu<64>(holds ? (uint32_t)own_e : ~0u);
    if (lane == s) my_i = (int)at;
    if ((int)(at % 64) == lane) {
      rank[at] = 0ull;
      own = 0ull;
#pragma unroll 8
      for (int e = lane; e < a.E; e += 64) {
        const uint64_t r = rank[e];
        own_e = r > own ? e : own_e;
        own = r > own ? r : own;
      }
    }
  }
  return my_i;
}

// How many lanes of the lane's row of 16 hold more than it (below 2^31): the
// signs of the differences, shifted together.  (A sum with the negative: as a
// subtraction with a DPP operand the compiler's code had the other sign here.)
__device__ __forceinline__ int lanes_above(uint32_t v) {
  uint32_t signs = 0u;
  const uint32_t less = 0u - v;
#define ROUTE_ROTATE(n) signs = __builtin_amdgcn_alignbit(signs, v + row_ror<n>(less), 31);
  ROUTE_ROTATE(1) ROUTE_ROTATE(2) ROUTE_ROTATE(3) ROUTE_ROTATE(4) ROUTE_ROTATE(5)
  ROUTE_ROTATE(6) ROUTE_ROTATE(7) ROUTE_ROTATE(8) ROUTE_ROTATE(9) ROUTE_ROTATE(10)
  ROUTE_ROTATE(11) ROUTE_ROTATE(12) ROUTE_ROTATE(13) ROUTE_ROTATE(14) ROUTE_ROTATE(15)
#undef ROUTE_ROTATE
  return __popc(signs);
}

// kByScore: with a bias.  kQuads: groups, and every four experts that a lane
// holds next to each other are of one group.
enum RouteMode { kByLogit, kByScore, kGrouped, kQuads };

// LDS of one wave: four tokens' values, padded by one a group so that lanes
// that read one group each meet different banks, and strengths; or
// route_exact's doubles.
template <int G>
size_t route_lds(int E, int n_group) {
  const size_t fast = (64 / G) * (size_t)(E + 2 * n_group) * sizeof(float);
  const size_t exact = (size_t)(E + n_group) * sizeof(double);
  return (std::max(fast, exact) + 15) / 16 * 16;
}

// G lanes per token, V experts and at most one slot per lane.
// Measured (logits read once; the copy rate would take 4, 4 and 6 us): 65,536 x
// 64, k 8: 9.7 us, 257 vector instructions per wave of four tokens, which alone
// take 6.7 us; 16,384 x 256 in groups, k 8, biased: 13.2 us, 1,020 a wave, 6.8
// us, after one wave's own latency of 2 and the loads'; 8192 x 896, k 16: 11.7
// us, 549 a wave of one token, 7.2 us.  Against a wave per token with 64-bit
// ranks throughout: 120, 50 and 60 us.  k rounds over all experts in the place
// of candidates: 14.7, 32.8 and 31.2 us.  Lane ln
// holds expert (j / 4) 4 G + (vec ? 4 ln + j % 4 : ln + (j % 4) G) as its j-th:
// ascending in j, and 16 bytes at a time where rows start on 16-byte steps.
template <int G, int V, int MODE>
__global__ __launch_bounds__(kThreads) void route_forward_kernel(const RouteArgs a, int vec,
                                                                 uint32_t per_mul, int wave_lds) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ __attribute__((aligned(16))) uint2 lists[kWaves][64 + 8];
  constexpr int TPW = 64 / G;
  const float kNone = __builtin_nanf("");  // a rank that nothing takes
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int ln = lane % G, sub = lane / G;
  const int64_t t0 = ((int64_t)blockIdx.x * kWaves + w) * TPW;
  if (t0 >= a.N) return;  // whole wave leaves together; no work-group barrier below
  const bool valid = t0 + sub < a.N;
  const int64_t t = min(t0 + sub, a.N - 1);
  const float* row = a.logits + t * a.E;
  const int mine = vec ? 4 * ln : ln, step = vec ? 1 : G;
  auto place = [&](int j) { return (j / 4) * 4 * G + (j % 4) * step; };  // expert j's index, less `mine`

  float l[V];  // -inf: masked, NaN: past the last expert
  if (vec) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const f32x4_t q = *reinterpret_cast<const f32x4_t*>(row + min(mine + place(j), a.E - 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) l[j + i] = mine + place(j) < a.E ? fmaxf(q[i], -INFINITY) : kNone;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = row[min(mine + place(j), a.E - 1)];
      l[j] = mine + place(j) < a.E ? fmaxf(l[j], -INFINITY) : kNone;
    }
  }
  float top = -INFINITY, inv_z = 0.f;
  if (!a.sigmoid && (MODE != kByLogit || !a.renorm)) {
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, l[j]);
    top = run_maxf<G>(top);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) z += fmaxf(__expf(l[j] - top), 0.f);  // 0 of NaN
    z = run_sum<G>(z);
    inv_z = z > 0.f ? 1.f / z : 0.f;
  }

  float rank[V];
  bool near = false;  // 32 bits do not tell: select again with route_exact
  if constexpr (MODE == kByLogit) {
#pragma unroll
    for (int j = 0; j < V; ++j) rank[j] = l[j];
  } else {
    // v_e.  Loads and the choice of score stand outside the loops: a branch per
    // element would wait for each load by itself.
    float v[V], b[V];
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = logistic(l[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = fmaxf(__expf(l[j] - top) * inv_z, 0.f);
    }
    if (a.bias) {
      if (vec) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const f32x4_t q = *reinterpret_cast<const f32x4_t*>(a.bias + min(mine + place(j), a.E - 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) b[j + i] = q[i];
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = a.bias[min(mine + place(j), a.E - 1)];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += b[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = l[j] > -INFINITY ? fmaxf(v[j], -INFINITY) : l[j];  // a NaN bias masks its expert
      rank[j] = a.bias ? v[j] : l[j];
    }
    if constexpr (MODE >= kGrouped) {
      // Lane g adds up group g's best out of LDS: from the values, or from the
      // two best of each four.
      constexpr int Q = MODE == kQuads ? 4 : 1, NQ = V / Q;
      const int per = a.E / a.n_group / Q;
      float* val = reinterpret_cast<float*>(smem + w * wave_lds) + sub * (a.E + 2 * a.n_group);
      float* strength = val + a.E + a.n_group;
      int grp[NQ];
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        const int e = (mine + place(j * Q)) / Q;
        grp[j] = (int)(((uint32_t)e * per_mul) >> 20);
        if constexpr (MODE == kQuads) {
          const float* x = v + 4 * j;
          float b1 = fmaxf(x[0], x[1]), b2 = fminf(x[0], x[1]);
#pragma unroll
          for (int i = 2; i < 4; ++i) {
            b2 = __builtin_amdgcn_fmed3f(b2, b1, x[i]);
            b1 = fmaxf(b1, x[i]);
          }
          if (e * 4 < a.E) reinterpret_cast<float2*>(val)[e + grp[j]] = make_float2(b1, b2);
        } else {
          if (e < a.E) val[e + grp[j]] = v[j];
        }
      }
      wave_lds_order();
      float size = 0.f;  // of the values summed
      for (int g = ln; g < a.n_group; g += G) {
        float b1 = -INFINITY, b2 = -INFINITY;  // b2 <= b1: med3 is the second of the three
        if constexpr (MODE == kQuads) {
          const float2* q = reinterpret_cast<const float2*>(val) + g * (per + 1);
#pragma unroll 8
          for (int i = 0; i < per; ++i) {
            b2 = fmaxf(__builtin_amdgcn_fmed3f(b2, b1, q[i].x), q[i].y);
            b1 = fmaxf(b1, q[i].x);
          }
        } else {
          const float* q = val + g * (per + 1);
#pragma unroll 8
          for (int i = 0; i < per; ++i) {
            b2 = __builtin_amdgcn_fmed3f(b2, b1, q[i]);
            b1 = fmaxf(b1, q[i]);
          }
        }
        strength[g] = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        if (b1 > -INFINITY) size = fmaxf(size, fmaxf(fabsf(b1), b2 > -INFINITY ? fabsf(b2) : 0.f));
      }
      wave_lds_order();
      uint32_t lo = 0u, hi = 0u;
      float weakest = INFINITY, next = -INFINITY;  // of the kept, the best of the others
      for (int g = ln; g < a.n_group; g += G) {
        const float x = strength[g];
        int before = 0;
        for (int h = 0; h < a.n_group; ++h)
          before += strength[h] > x || (strength[h] == x && h < g) ? 1 : 0;
        if (before < a.topk_group) {
          weakest = fminf(weakest, x);
          if (g < 32) lo |= 1u << g; else hi |= 1u << (g - 32);
        } else {
          next = fmaxf(next, x);
        }
      }
      lo = run_or<G>(lo);
      hi = run_or<G>(hi);
      weakest = run_minf<G>(weakest);
      next = run_maxf<G>(next);
      near = next > -INFINITY && !(weakest - next > 2.f * nearness(a.sigmoid, run_maxf<G>(size)));
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        const bool keep = ((grp[j] < 32 ? lo : hi) >> (grp[j] & 31)) & 1;
#pragma unroll
        for (int i = 0; i < Q; ++i) rank[Q * j + i] = keep ? rank[Q * j + i] : kNone;
      }
    }
  }

  int my_i = 0;
  float my_v = -INFINITY;  // the value it ranks by
  const bool close = MODE != kByLogit && a.bias;  // ranks are scores, not exact
  bool done = false;
  // The wanted ranks are among few candidates: with `want` of the lanes'
  // largest at or above T, so are the `want` largest of all.  T is taken per
  // row of 16 lanes, from how many of the row's lanes have a larger largest.
  // The candidates, one a lane, then count those before them.
  constexpr int ROWS = G / 16;
  const int want = (a.k + (close ? 1 : 0) + ROWS - 1) / ROWS;
  if (want <= 16) {
    float best = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) best = fmaxf(best, rank[j]);
    // how many of the row's lanes have more: signs of differences, the lowest
    // bit left out (a lane too many with that much is as good)
    const int above = lanes_above(order_of(best) >> 1);
    // with close, whatever may turn out to be ahead of T belongs to the candidates
    auto below = [&](float x) __attribute__((always_inline)) {
      return close && fabsf(x) < INFINITY ? x - nearness(a.sigmoid, x) : x;
    };
    float T = below(run_minf<G>(above < want ? best : INFINITY));
    // (value, ~expert) of each candidate; larger is earlier
    uint2* list = lists[w] + sub * (G + 2);
    int held = 0;
    auto count_from = [&](float from) __attribute__((always_inline)) {
      held = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) held += rank[j] >= from ? 1 : 0;
      return run_sumi<G>(held);
    };
    int count = count_from(T);
    if (__any(count > G)) {
      // the best sit in few lanes (kept groups do): halve the way from T to
      // the largest until what is left fits, from the lowest lane's largest if
      // that will do (-inf is many halvings away)
      const float some = run_minf<G>(best > -INFINITY ? best : INFINITY);
      const int with_some = count_from(some);
      const bool enough = T == -INFINITY && with_some >= want * ROWS;
      uint32_t low = order_of(enough ? some : T), high = order_of(run_maxf<G>(best)) + 1u;
      bool open = count > G;
      for (int i = 0; i < 12 && __any(open); ++i) {
        const uint32_t mid = low + (high - low) / 2;
        const int c = count_from(value_of(mid));
        if (open) {
          if (c >= want * ROWS) low = mid; else high = mid;
          open = c < want * ROWS || c >= G;
        }
      }
      if (count > G) T = below(value_of(low));
      count = count_from(T);
    }
    int at = held;  // inclusive sums over the token's lanes
    at += row_shr<1>(at);
    at += row_shr<2>(at);
    at += row_shr<4>(at);
    at += row_shr<8>(at);
    if constexpr (G == 64) {
      int rows[3];
#pragma unroll
      for (int r = 0; r < 3; ++r) rows[r] = __builtin_amdgcn_readlane(at, 16 * r + 15);
      at += (ln >= 16 ? rows[0] : 0) + (ln >= 32 ? rows[1] : 0) + (ln >= 48 ? rows[2] : 0);
    }
    if (!__any(count > G)) {
      done = true;
      uint2* to = list + (at - held);
      const uint32_t last = ~(uint32_t)mine;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (rank[j] >= T) *to++ = make_uint2(__float_as_uint(rank[j]), last - place(j));
      if (G == 64 && ln < 8) list[count + ln].x = __float_as_uint(kNone);  // read by eights
      wave_lds_order();
      const bool in = ln < count;
      const uint2 c0 = list[ln];
      const float x0 = in ? __uint_as_float(c0.x) : -INFINITY;
      int before = 0;
      if constexpr (G == 64) {
        const int n = __builtin_amdgcn_readfirstlane(count);
        for (int c = 0; c < n; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 q = reinterpret_cast<const uint4*>(list + c)[u];
            before += __uint_as_float(q.x) > x0 ? 1 : 0;
            before += __uint_as_float(q.z) > x0 ? 1 : 0;
          }
      } else {
        before = lanes_above(in ? order_of(x0) >> 1 : 0u);
      }
      if (__any(run_sumi<G>(in ? before : 0) != count * (count - 1) / 2)) {
        // equal values (or a lowest bit apart): by value, then expert
        const uint64_t cand = in ? (uint64_t)order_of(x0) << 32 | c0.y : 0ull;
        before = 0;
        if constexpr (G == 64) {
          const int n = __builtin_amdgcn_readfirstlane(count);
          for (int c = 0; c < n; ++c) {
            const uint64_t o = (uint64_t)__builtin_amdgcn_readlane((int)(cand >> 32), c) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)cand, c);
            before += o > cand ? 1 : 0;
          }
        } else {
#define ROUTE_ROTATE(n)                                                                       \
  before += ((uint64_t)row_ror<n>((uint32_t)(cand >> 32)) << 32 | row_ror<n>((uint32_t)cand)) > cand ? 1 : 0;
          ROUTE_ROTATE(1) ROUTE_ROTATE(2) ROUTE_ROTATE(3) ROUTE_ROTATE(4) ROUTE_ROTATE(5)
          ROUTE_ROTATE(6) ROUTE_ROTATE(7) ROUTE_ROTATE(8) ROUTE_ROTATE(9) ROUTE_ROTATE(10)
          ROUTE_ROTATE(11) ROUTE_ROTATE(12) ROUTE_ROTATE(13) ROUTE_ROTATE(14) ROUTE_ROTATE(15)
#undef ROUTE_ROTATE
        }
      }
      wave_lds_order();
      if (in) list[before] = c0;
      wave_lds_order();
      uint2 sel = list[ln];
      if (close) {
        // in order now: are neighbours that matter too near?
        const float x = in ? __uint_as_float(sel.x) : -INFINITY;
        const float y = ln + 1 < count ? __uint_as_float(list[ln + 1].x) : -INFINITY;
        if (__any(ln < a.k && y > -INFINITY && !(x - y > nearness(a.sigmoid, y)))) {
          // then all candidates rank by their values in 64 bits
          double z = 1.0;
          if (!a.sigmoid) z = softmax_sum64<G>(row, a.E, ln, top);
          const int e = in ? (int)~c0.y : 0;
          const float le = row[e];
          const double s64 = a.sigmoid ? 1.0 / (1.0 + exp(-(double)le)) : exp((double)le - (double)top) / z;
          const uint64_t o64 = order_of(is_masked(le) ? -(double)INFINITY : fmax(s64 + (double)a.bias[e], -INFINITY));
          before = 0;
          for (int c = 0; c < G; ++c) {
            const int from = sub * G + c;
            const uint64_t o = __shfl(o64, from);
            const uint32_t oid = __shfl(c0.y, from);
            before += c < count && (o > o64 || (o == o64 && oid > c0.y)) ? 1 : 0;
          }
          wave_lds_order();
          if (in) list[before] = c0;
          wave_lds_order();
          sel = list[ln];
        }
      }
      if (ln < a.k) {
        my_i = (int)~sel.y;
        my_v = __uint_as_float(sel.x);
      }
    }
  }
  float prev = INFINITY;
  for (int s = 0; !done && s < a.k + (close ? 1 : 0); ++s) {
    float x = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) x = fmaxf(x, rank[j]);
    x = run_maxf<G>(x);
    if (close) {
      near |= x > -INFINITY && !(prev - x > nearness(a.sigmoid, x));
      prev = x;
      if (s == a.k) break;
    }
    uint32_t at = ~0u;
#pragma unroll
    for (int j = V - 1; j >= 0; --j)
      if (rank[j] == x) at = place(j);
    at = run_minu<G>(at == ~0u ? at : at + mine);
    const uint32_t mine_at = at - mine;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if ((int)mine_at == place(j)) rank[j] = kNone;
    if (ln == s) my_i = (int)at, my_v = x;
  }
  bool by_logit = MODE == kByLogit || !a.bias;  // my_v holds logits
  if constexpr (MODE != kByLogit) {
    uint64_t again = __ballot(near && valid && ln == 0);
    while (again) {
      const int first = __builtin_ctzll(again);
      again &= again - 1;
      const int at = route_exact(a, t0 + first / G, reinterpret_cast<double*>(smem + w * wave_lds));
      const int mine_at = __shfl(at, ln);
      if (sub == first / G) my_i = mine_at;
      by_logit = false;
    }
  }

  // gates, lane ln for slot ln
  const bool slot = ln < a.k;
  const float ls = !slot ? -INFINITY : fmaxf(by_logit ? my_v : row[my_i], -INFINITY);
  float g;
  if (a.renorm) {
    // scores relative to the largest one selected: no sum underflows
    const float m = run_maxf<G>(ls);
    const float c = a.sigmoid ? fminf(m, 0.f) : m;
    g = 0.f;
    if (ls > -INFINITY) g = a.sigmoid ? sigmoid_rel(ls, c, nullptr) : __expf(ls - c);
    const float sum = run_sum<G>(g);
    g *= sum > 0.f ? a.scale * rcp(sum) : 0.f;
  } else if (a.sigmoid) {
    g = a.scale * sigmoid_rel(ls, 0.f, nullptr);
  } else {
    g = ls > -INFINITY ? a.scale * (__expf(ls - top) * inv_z) : 0.f;
  }
  if (valid && slot) {
    a.idx[t * a.k + ln] = my_i;
    a.gates[t * a.k + ln] = g;
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

// Writing the row of dlogits bounds it: 65,536 x 64 takes 6.9 us (2.4 TB/s
// written), 16,384 x 256 5.6 us (3.0), 8192 x 896 with the dense part 9.0 us
// (3.3, as much read).  G lanes per token as in the forward pass: lane ln works
// out slot ln's share, the row goes through LDS (zeros or the softmax's dense
// part, then the selected experts' shares added) and out.
template <int G, int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const RouteBwdArgs a, int vec) {
  constexpr int TPW = 64 / G;
  __shared__ __attribute__((aligned(16))) float rows[kWaves * TPW][G * V];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int ln = lane % G, sub = lane / G;
  const int64_t t0 = ((int64_t)blockIdx.x * kWaves + w) * TPW;
  if (t0 >= a.N) return;  // whole wave leaves together
  const bool valid = t0 + sub < a.N;
  const int64_t t = min(t0 + sub, a.N - 1);
  const float* row = a.logits + t * a.E;
  float* out = rows[w * TPW + sub];
  const int mine = vec ? 4 * ln : ln, step = vec ? 1 : G;
  auto place = [&](int j) { return (j / 4) * 4 * G + (j % 4) * step; };

  int e = -1;
  float ls = -INFINITY, dg = 0.f;
  if (ln < a.k) {
    const int at = a.idx[t * a.k + ln];
    const float up = a.dgates[t * a.k + ln];
    if ((unsigned)at < (unsigned)a.E) ls = fmaxf(row[at], -INFINITY);
    if (ls > -INFINITY) {  // else a gate fixed at 0
      e = at;
      dg = up;
    }
  }
  const bool dense = !a.sigmoid && !a.renorm;
  float l[V], top = -INFINITY, inv_z = 0.f;
  if (dense) {
    if (vec) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        f32x4_t q{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (mine + place(j) < a.E) q = *reinterpret_cast<const f32x4_t*>(row + mine + place(j));
#pragma unroll
        for (int i = 0; i < 4; ++i) l[j + i] = q[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) l[j] = mine + place(j) < a.E ? row[mine + place(j)] : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (is_masked(l[j])) l[j] = -INFINITY;
      top = fmaxf(top, l[j]);
    }
    top = run_maxf<G>(top);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      l[j] = is_masked(l[j]) ? 0.f : __expf(l[j] - top);
      z += l[j];
    }
    z = run_sum<G>(z);
    inv_z = z > 0.f ? 1.f / z : 0.f;
  }
  float w_s, one_less = 0.f;  // g_s / scale, 1 - s
  if (a.renorm) {
    const float m = run_maxf<G>(ls);
    const float c = a.sigmoid ? fminf(m, 0.f) : m;
    w_s = a.sigmoid ? sigmoid_rel(ls, c, &one_less) : __expf(ls - c);
    if (e < 0) w_s = 0.f;
    const float sum = run_sum<G>(w_s);
    w_s *= sum > 0.f ? rcp(sum) : 0.f;
  } else if (a.sigmoid) {
    w_s = sigmoid_rel(ls, 0.f, &one_less);
  } else {
    w_s = e >= 0 ? __expf(ls - top) * inv_z : 0.f;
  }
  float dot = 0.f;  // sum_j g_j dg_j
  if (!a.sigmoid || a.renorm) dot = a.scale * run_sum<G>(w_s * dg);
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    f32x4_t q{0.f, 0.f, 0.f, 0.f};
    if (dense)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = -(l[j + i] * inv_z) * dot;
    if (vec) {
      *reinterpret_cast<f32x4_t*>(out + mine + place(j)) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[mine + place(j + i)] = q[i];
    }
  }
  wave_lds_order();
  if (e >= 0) {
    float d = w_s * (a.scale * dg - (dense ? 0.f : dot));
    if (a.sigmoid) d *= one_less;
    out[e] += d;
  }
  wave_lds_order();
  if (!valid) return;
  float* to = a.dlogits + t * a.E;
  if (vec) {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      if (mine + place(j) < a.E)
        *reinterpret_cast<f32x4_t*>(to + mine + place(j)) = *reinterpret_cast<const f32x4_t*>(out + mine + place(j));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (mine + place(j) < a.E) to[mine + place(j)] = out[mine + place(j)];
  }
}

// Calls f with lanes per token and experts per lane, for a selection among the
// `wanted` largest.  A row of 16 lanes while 16 experts each (what keeps a lane
// to a fifth of a SIMD's registers) and one slot each do; a wave past that:
// 20,000 x 250, k 32 takes 16.4 us so and took 35.6 with four slots a lane in k
// rounds, k 16 with a bias 25 and 42.
template <typename F>
void with_shape(int E, int wanted, F f) {
  using std::integral_constant;
#define ROUTE_SHAPE(g, v) f(integral_constant<int, g>(), integral_constant<int, v>())
  if (E > 512) return ROUTE_SHAPE(64, 16);
  if (E > 256) return ROUTE_SHAPE(64, 8);
  if (wanted > 16) return ROUTE_SHAPE(64, 4);
  if (E > 128) return ROUTE_SHAPE(16, 16);
  if (E > 64) return ROUTE_SHAPE(16, 8);
  return ROUTE_SHAPE(16, 4);
#undef ROUTE_SHAPE
}

bool rows_aligned(int E, const void* p, const void* q) {
  return E % 4 == 0 && ((uintptr_t)p | (uintptr_t)q) % 16 == 0;
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
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int vec = rows_aligned(P.E, logits, bias);
  // groups of whole fours: 20.6 against 22.1 us at 16,384 x 256 one by one
  const bool quads = vec && P.E / P.n_group % 4 == 0;
  const int mode = P.n_group > 1 ? (quads ? kQuads : kGrouped) : bias ? kByScore : kByLogit;
  // e / per as a product: exact for e < 1024, per < 1024
  const int per = P.E / P.n_group / (mode == kQuads ? 4 : 1);
  const uint32_t per_mul = ((1u << 20) + per - 1) / per;
  with_shape(P.E, P.k + (bias ? 1 : 0), [&](auto g, auto v) {
    constexpr int G = g.value, V = v.value;
    const unsigned grid = (unsigned)ceil_div(P.N, kWaves * (64 / G));
    const size_t lds = route_lds<G>(P.E, P.n_group);
    if (mode == kByLogit)
      route_forward_kernel<G, V, kByLogit><<<grid, kThreads, 0, st>>>(a, vec, per_mul, 0);
    else if (mode == kByScore)
      route_forward_kernel<G, V, kByScore><<<grid, kThreads, kWaves * lds, st>>>(a, vec, per_mul, (int)lds);
    else if (mode == kGrouped)
      route_forward_kernel<G, V, kGrouped><<<grid, kThreads, kWaves * lds, st>>>(a, vec, per_mul, (int)lds);
    else
      route_forward_kernel<G, V, kQuads><<<grid, kThreads, kWaves * lds, st>>>(a, 1, per_mul, (int)lds);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

MOE_API int route_backward(const route_plan_t* plan, const float* logits, const int32_t* topk_idx,
                           const float* dgates, float* dlogits, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const route_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!logits || !topk_idx || !dgates || !dlogits) return MOE_EINVAL;
  const RouteBwdArgs a{logits, topk_idx, dgates, dlogits, P.N, P.E, P.k, P.score, P.renorm, P.scale};
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int vec = rows_aligned(P.E, logits, dlogits);
  with_shape(P.E, P.k, [&](auto g, auto v) {
    constexpr int G = g.value, V = v.value;
    const unsigned grid = (unsigned)ceil_div(P.N, kWaves * (64 / G));
    route_backward_kernel<G, V><<<grid, kThreads, 0, st>>>(a, vec);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
