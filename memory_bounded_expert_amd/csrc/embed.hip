// Token embedding with scaling and its gradient (include/embed.h).
//
// Forward: a gather of rows, one vector per thread.  Backward: the positions
// are sorted by id with a stable radix sort, the sorted rows are summed in
// tiles of kTileRows positions, and runs of one id that cross tiles are
// joined in order by a last launch.
#include <algorithm>
#include <cmath>

#include "device_common.hpp"
#include "embed.h"
#include "moe_internal.h"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kEmbedMagic = 0x454d4231u;  // "EMB1"
constexpr int kTileRows = 32;                  // sorted positions per summing tile
constexpr int kSortTile = 2048;                // keys per work-group of a sort pass
constexpr int kSortRounds = kSortTile / kThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxDigit = 10;                  // bits of a sort pass's digit
constexpr int kScanThreads = 1024;

// ---- forward

// VEC: one 16-byte vector per thread, else one element.
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(const T* __restrict__ W,
                                                                 const int32_t* __restrict__ ids,
                                                                 T* __restrict__ Y, int64_t N,
                                                                 int64_t V, int H, float scale) {
  constexpr int EPC = VEC ? Elem<T>::kPer16B : 1;
  const int cpr = H / EPC;
  const int64_t total = N * cpr;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < total;
       q += (int64_t)gridDim.x * kThreads) {
    const int64_t t = q / cpr;
    const int c = (int)(q - t * cpr);
    const int64_t id = ids[t];
    const bool real = id >= 0 && id < V;
    if constexpr (VEC) {
      u32x4_t raw{0u, 0u, 0u, 0u};
      if (real) {
        float v[EPC];
        unpack16(reinterpret_cast<const u32x4_t*>(W + id * H)[c], v, T());
#pragma unroll
        for (int e = 0; e < EPC; ++e) v[e] *= scale;
        raw = pack16(v, T());
      }
      reinterpret_cast<u32x4_t*>(Y + t * H)[c] = raw;
    } else {
      Y[t * H + c] = real ? Elem<T>::from_f(Elem<T>::to_f(W[id * H + c]) * scale) : Elem<T>::from_f(0.f);
    }
  }
}

// ---- sort: positions by id, stable; ids outside [0, V) as V, so last

struct SortPass {
  const int32_t* ids;   // first pass: keys from the ids, positions as they stand
  const uint32_t* key;  // later passes
  const uint32_t* pos;
  uint32_t* key_out;
  uint32_t* pos_out;
  int32_t* hist;        // [bins][tiles]: counts, then first output positions
  int64_t N, V;
  int tiles, shift, bits;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& a, int64_t i) {
  if (!a.ids) return a.key[i];
  const int64_t id = a.ids[i];
  return id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

__global__ __launch_bounds__(kThreads) void sort_count_kernel(const SortPass a) {
  __shared__ int32_t cnt[1 << kMaxDigit];
  const int bins = 1 << a.bits;
  for (int b = threadIdx.x; b < bins; b += kThreads) cnt[b] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = (int64_t)blockIdx.x * kSortTile + r * kThreads + threadIdx.x;
    if (i < a.N) atomicAdd(&cnt[(sort_key(a, i) >> a.shift) & (bins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) a.hist[(int64_t)b * a.tiles + blockIdx.x] = cnt[b];
}

// Exclusive scan of n counts in place, one work-group.
__global__ __launch_bounds__(kScanThreads) void sort_scan_kernel(int32_t* __restrict__ v, int n) {
  __shared__ int32_t sums[kScanThreads / 64];
  const int per = (n + kScanThreads - 1) / kScanThreads;
  const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
  int s = 0;
  for (int i = lo; i < hi; ++i) s += v[i];
  int inc = s;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 63) sums[w] = inc;
  __syncthreads();
  int run = inc - s;
  for (int x = 0; x < w; ++x) run += sums[x];
  for (int i = lo; i < hi; ++i) {
    const int c = v[i];
    v[i] = run;
    run += c;
  }
}

// Each wave places its kSortTile / kWaves consecutive keys in order: within 64
// keys, equal digits rank by lane (one ballot per digit bit).
__global__ __launch_bounds__(kThreads) void sort_place_kernel(const SortPass a) {
  __shared__ int32_t next[kWaves][1 << kMaxDigit];
  const int bins = 1 << a.bits;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int b = lane; b < bins; b += 64) next[w][b] = 0;
  wave_lds_order();
  const int64_t base = (int64_t)blockIdx.x * kSortTile + w * (kSortTile / kWaves);
  uint32_t key[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    key[r] = i < a.N ? sort_key(a, i) : 0u;
    if (i < a.N) atomicAdd(&next[w][(key[r] >> a.shift) & (bins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) {
    int run = a.hist[(int64_t)b * a.tiles + blockIdx.x];
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const int c = next[v][b];
      next[v][b] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    const bool in = i < a.N;
    const uint32_t d = (key[r] >> a.shift) & (bins - 1);
    uint64_t same = __ballot(in);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? m : ~m;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    const int at = in ? next[w][d] + before : 0;
    wave_lds_order();  // every lane has read its start
    if (in && (same >> lane) == 1) next[w][d] = at + 1;  // the digit's last lane
    wave_lds_order();
    if (in) {
      a.key_out[at] = key[r];
      a.pos_out[at] = a.ids ? (uint32_t)i : a.pos[i];
    }
  }
}

// ---- sums over runs of equal ids

struct SumArgs {
  const uint32_t* key;
  const uint32_t* pos;
  const void* dY;
  float* dW;
  float* part;  // [tile][2][H]: a run continued from an earlier tile; one that goes on
  int64_t N, V;
  int H, accumulate;
  float scale;
};

template <int EPC>
__device__ __forceinline__ void store_row(float* p, const float* v) {
  if constexpr (EPC == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int e = 0; e < EPC; e += 4)
      *reinterpret_cast<f32x4_t*>(p + e) = f32x4_t{v[e], v[e + 1], v[e + 2], v[e + 3]};
  }
}
template <int EPC>
__device__ __forceinline__ void write_dw(const SumArgs& a, uint32_t id, int64_t col, const float* acc) {
  float* p = a.dW + (int64_t)id * a.H + col;
  float v[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) v[e] = a.accumulate ? p[e] + a.scale * acc[e] : a.scale * acc[e];
  store_row<EPC>(p, v);
}

// One tile of sorted positions by a block of columns.
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(const SumArgs a) {
  constexpr int EPC = VEC ? Elem<T>::kPer16B : 1;
  const int64_t i0 = (int64_t)blockIdx.x * kTileRows, i1 = min(a.N, i0 + kTileRows);
  const int64_t col = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * EPC;
  if (col >= a.H) return;
  uint32_t cur = a.key[i0];
  bool head = i0 > 0 && a.key[i0 - 1] == cur;
  float acc[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) acc[e] = 0.f;
  auto flush = [&](bool goes_on) {
    if (cur >= a.V) return;
    if (head || goes_on)
      store_row<EPC>(a.part + (blockIdx.x * 2 + (head ? 0 : 1)) * (int64_t)a.H + col, acc);
    else
      write_dw<EPC>(a, cur, col, acc);
  };
  for (int64_t i = i0; i < i1; ++i) {
    const uint32_t k = a.key[i];
    if (k != cur) {
      flush(false);
      cur = k;
      head = false;
#pragma unroll
      for (int e = 0; e < EPC; ++e) acc[e] = 0.f;
    }
    if (k >= a.V) return;  // the padded positions come last
    const T* row = static_cast<const T*>(a.dY) + (int64_t)a.pos[i] * a.H + col;
    float v[EPC];
    if constexpr (VEC)
      unpack16(*reinterpret_cast<const u32x4_t*>(row), v, T());
    else
      v[0] = Elem<T>::to_f(*row);
#pragma unroll
    for (int e = 0; e < EPC; ++e) acc[e] += v[e];
  }
  flush(i1 < a.N && a.key[i1] == cur);
}

// Joins the run that starts in this tile and goes on past it, tile by tile.
template <int EPC>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const SumArgs a) {
  const int64_t i0 = (int64_t)blockIdx.x * kTileRows, i1 = i0 + kTileRows;
  const int64_t col = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * EPC;
  if (i1 >= a.N || col >= a.H) return;
  const uint32_t cur = a.key[i1];
  if (cur >= a.V || a.key[i1 - 1] != cur) return;             // nothing goes on
  if (i0 > 0 && a.key[i0 - 1] == cur) return;  // it started earlier
  float acc[EPC];
  const float* p = a.part + (blockIdx.x * 2 + 1) * (int64_t)a.H + col;
#pragma unroll
  for (int e = 0; e < EPC; ++e) acc[e] = p[e];
  for (int64_t c = blockIdx.x + 1; c * kTileRows < a.N && a.key[c * kTileRows] == cur; ++c) {
    const float* q = a.part + c * 2 * (int64_t)a.H + col;
#pragma unroll
    for (int e = 0; e < EPC; ++e) acc[e] += q[e];
  }
  write_dw<EPC>(a, cur, col, acc);
}

struct EmbedLayout {
  size_t key[2], pos[2], hist, part, total;
  int tiles, passes, bits;
};

EmbedLayout embed_layout(int64_t N, int64_t V, int H) {
  EmbedLayout L{};
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) & ~(size_t)255;
    return o;
  };
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V
  L.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  L.bits = (bits + L.passes - 1) / L.passes;
  L.tiles = (int)ceil_div(N, kSortTile);
  for (int i = 0; i < 2; ++i) L.key[i] = take((size_t)N * 4);
  for (int i = 0; i < 2; ++i) L.pos[i] = take((size_t)N * 4);
  L.hist = take(((size_t)L.tiles << L.bits) * 4);
  L.part = take((size_t)ceil_div(N, kTileRows) * 2 * H * 4);
  L.total = cur;
  return L;
}

template <typename T>
hipError_t sum_and_join(const SumArgs& a, bool vec, hipStream_t st) {
  const int epc = vec ? Elem<T>::kPer16B : 1;
  const dim3 grid((unsigned)ceil_div(a.N, kTileRows), (unsigned)ceil_div(a.H, kThreads * epc));
  if (vec) {
    embed_sum_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
    embed_join_kernel<Elem<T>::kPer16B><<<grid, kThreads, 0, st>>>(a);
  } else {
    embed_sum_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
    embed_join_kernel<1><<<grid, kThreads, 0, st>>>(a);
  }
  return hipGetLastError();
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

bool plan_ok(const embed_plan_t* p) { return p != nullptr && p->magic == kEmbedMagic; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int embed_plan(int64_t N, int64_t V, int32_t H, int32_t dtype, float scale,
                       embed_plan_t* out) {
  if (!out || N < 0 || V < 1 || H < 1 || !std::isfinite(scale)) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (N >= ((int64_t)1 << 26) || V >= ((int64_t)1 << 30) || H > 65536) return MOE_EUNSUPPORTED;
  embed_plan_t p{};
  p.magic = kEmbedMagic;
  p.dtype = dtype;
  p.N = N;
  p.V = V;
  p.H = H;
  p.scale = scale;
  p.bwd_workspace_bytes = N == 0 ? 0 : (int64_t)embed_layout(N, V, H).total;
  *out = p;
  return MOE_OK;
}

MOE_API int embed_forward(const embed_plan_t* plan, const void* W, const int32_t* ids, void* Y,
                          void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const embed_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!W || !ids || !Y) return MOE_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const int epc = 16 / elem_bytes(P.dtype);
  const bool vec = P.H % epc == 0 && aligned16(W) && aligned16(Y);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(P.N * (P.H / (vec ? epc : 1)), kThreads), 1 << 20);
  auto run = [&](auto kern, auto* w, auto* y) { kern<<<grid, kThreads, 0, st>>>(w, ids, y, P.N, P.V, P.H, P.scale); };
  if (P.dtype == MOE_BF16)
    run(vec ? embed_forward_kernel<bf16_t, true> : embed_forward_kernel<bf16_t, false>, (const bf16_t*)W, (bf16_t*)Y);
  else
    run(vec ? embed_forward_kernel<float, true> : embed_forward_kernel<float, false>, (const float*)W, (float*)Y);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

MOE_API int embed_backward(const embed_plan_t* plan, const int32_t* ids, const void* dY, float* dW,
                           int32_t accumulate, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const embed_plan_t& P = *plan;
  if (!dW || (P.N > 0 && (!ids || !dY || !workspace))) return MOE_EINVAL;
  if (P.N > 0 && (uintptr_t)workspace % 256) return MOE_EINVAL;
  if (workspace_bytes < (size_t)P.bwd_workspace_bytes) return MOE_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  if (!accumulate && launch_fill_zero(dW, (size_t)P.V * P.H * sizeof(float), st) != hipSuccess)
    return MOE_EHIP;
  if (P.N == 0) return MOE_OK;
  const EmbedLayout L = embed_layout(P.N, P.V, P.H);
  char* ws = (char*)workspace;
  SortPass s{};
  s.ids = ids;
  s.hist = (int32_t*)(ws + L.hist);
  s.N = P.N;
  s.V = P.V;
  s.tiles = L.tiles;
  s.bits = L.bits;
  for (int i = 0; i < L.passes; ++i) {
    s.shift = i * L.bits;
    s.key_out = (uint32_t*)(ws + L.key[i & 1]);
    s.pos_out = (uint32_t*)(ws + L.pos[i & 1]);
    sort_count_kernel<<<L.tiles, kThreads, 0, st>>>(s);
    sort_scan_kernel<<<1, kScanThreads, 0, st>>>(s.hist, L.tiles << L.bits);
    sort_place_kernel<<<L.tiles, kThreads, 0, st>>>(s);
    s.ids = nullptr;
    s.key = s.key_out;
    s.pos = s.pos_out;
  }
  if (hipGetLastError() != hipSuccess) return MOE_EHIP;
  const SumArgs a{s.key, s.pos, dY, dW, (float*)(ws + L.part), P.N, P.V, P.H, accumulate != 0, P.scale};
  const bool vec = P.H % (16 / elem_bytes(P.dtype)) == 0 && aligned16(dY) && aligned16(dW);
  const hipError_t err = P.dtype == MOE_BF16 ? sum_and_join<bf16_t>(a, vec, st) : sum_and_join<float>(a, vec, st);
  return err == hipSuccess ? MOE_OK : MOE_EHIP;
}
