// Token embedding with scaling and its gradient (include/embed.h).
//
// Forward: a gather of rows, one vector per thread, bound by HBM: 8192 rows of
// 7168 bf16 out of 200,000 take 39.5 us (85 MB read, the rest of the rows being
// repeats, and 117 MB written: 5.1 TB/s).
//
// Backward: what it cannot do without is reading dY and writing dW whole, zeros
// for the most part.  The positions are sorted by id with a stable radix sort
// of two or three passes; the sorted rows are summed in tiles of consecutive
// positions by blocks of columns, and runs of one id that cross tiles are
// joined in order by a last launch.  Up to kSmallSort positions are sorted by
// one work-group in LDS.  The sort's launches are short and fill few
// CUs, so each also zeroes a slice of dW on the others; the rest is zeroed in
// the summing launch, which knows the ids and skips the rows it writes itself.
// Measured, 65,536 positions of 2048 bf16 into 200,000 rows: sort 60 us with 192
// MB zeroed beside it (33 us without), sums and zeros 327 us (1.73 GB, 5.3 TB/s;
// zeros alone 6.1, sums alone 130 us), joins 13 us.
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
// Sorted positions per summing tile, one a lane at most.  A tile's rows follow
// one another, so small batches take short tiles: 516 positions of 2304 columns
// sum in 22 us by 64 and in 14 us by 32; 65,536 of 2048 in 329 and 327 us, but
// their runs join in 13 and 20 us.
constexpr int kTileRows = 64, kFewRows = 16;
constexpr int kSortTile = 1024;                // keys per work-group of a sort pass
constexpr int kSortRounds = kSortTile / kThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxDigit = 10;                  // bits of a sort pass's digit
constexpr int kScanThreads = 1024;
// Bytes of dW that a sort launch zeroes beside its own work: what the chip
// writes in the 5 us that such a launch takes.  The pass above takes 402 us so,
// 411 without, 415 with 96 MB; 1024 positions of 1024 into 5000 rows 16.7 and
// 20.4 us.
constexpr int64_t kSliceBytes = 32 << 20;
// The same beside sort_small_kernel, which takes 8 to 20 us on one CU: calls on
// 4000 x 512 into 100,000 rows 38.5 us so and 50 with 32 MB, 8 x 512 30 and 34,
// 1861 x 320 into 123,874 29 and 37, 44 x 128 into 132,469 17.9 and 18.6.
constexpr int64_t kSmallSlice = 128 << 20;
constexpr int64_t kZeroBytes = 1 << 18;        // bytes zeroed by a work-group

// ---- one lane's vector of a row: elements col .. col + EPC - 1, the row's last
// one short where TAIL (its elements then move one by one)

template <typename T, bool TAIL>
__device__ __forceinline__ u32x4_t load_vec(const T* row, int col, int H) {
  constexpr int EPC = Elem<T>::kPer16B;
  if (!TAIL || col + EPC <= H) return *reinterpret_cast<const u32x4_any_t*>(row + col);
  float v[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) v[e] = col + e < H ? Elem<T>::to_f(row[col + e]) : 0.f;
  return pack16(v, T());
}
template <typename T, bool TAIL>
__device__ __forceinline__ void store_vec(T* row, int col, int H, const float* v) {
  constexpr int EPC = Elem<T>::kPer16B;
  if (!TAIL || col + EPC <= H) {
    *reinterpret_cast<u32x4_any_t*>(row + col) = pack16(v, T());
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e)
      if (col + e < H) row[col + e] = Elem<T>::from_f(v[e]);
  }
}
// The same of fp32 rows, EPC elements (4 or 8).
template <int EPC, bool TAIL>
__device__ __forceinline__ void load_sum(const float* row, int col, int H, float* v) {
#pragma unroll
  for (int e = 0; e < EPC; e += 4) {
    f32x4_t q{0.f, 0.f, 0.f, 0.f};
    if (!TAIL || col + e + 4 <= H) {
      q = *reinterpret_cast<const f32x4_any_t*>(row + col + e);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (col + e + f < H) q[f] = row[col + e + f];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) v[e + f] = q[f];
  }
}
template <int EPC, bool TAIL>
__device__ __forceinline__ void store_sum(float* row, int col, int H, const float* v) {
#pragma unroll
  for (int e = 0; e < EPC; e += 4) {
    if (!TAIL || col + e + 4 <= H) {
      *reinterpret_cast<f32x4_any_t*>(row + col + e) = f32x4_t{v[e], v[e + 1], v[e + 2], v[e + 3]};
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (col + e + f < H) row[col + e + f] = v[e + f];
    }
  }
}
// Zeroes n values from p on by `threads` threads, this one the `tid`-th.
__device__ __forceinline__ void zero_values(float* p, int n, int tid, int threads) {
  for (int q = tid; q < n / 4; q += threads)
    *reinterpret_cast<u32x4_any_t*>(p + 4 * q) = u32x4_t{0u, 0u, 0u, 0u};
  if (tid < n % 4) p[n - 1 - tid] = 0.f;
}

// ---- forward

template <typename T, bool TAIL>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(const T* __restrict__ W,
                                                                 const int32_t* __restrict__ ids,
                                                                 T* __restrict__ Y, int64_t N,
                                                                 int64_t V, int H, float scale) {
  constexpr int EPC = Elem<T>::kPer16B;
  const int cpr = (H + EPC - 1) / EPC;
  const int64_t total = N * cpr;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < total;
       q += (int64_t)gridDim.x * kThreads) {
    const int64_t t = q / cpr;
    const int col = (int)(q - t * cpr) * EPC;
    const int64_t id = ids[t];
    float v[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e) v[e] = 0.f;
    if (id >= 0 && id < V) {
      unpack16(load_vec<T, TAIL>(W + id * H, col, H), v, T());
#pragma unroll
      for (int e = 0; e < EPC; ++e) v[e] *= scale;
    }
    store_vec<T, TAIL>(Y + t * H, col, H, v);
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
  // work-groups from `groups` on zero [zero, zero_end)
  int groups;
  float* zero;
  float* zero_end;
};

// Zeroes kZeroBytes of [p, end) from piece i on, by the whole work-group.
__device__ __forceinline__ void zero_piece(float* p, float* end, int64_t i) {
  p += i * (kZeroBytes / 4);
  zero_values(p, (int)min((int64_t)(end - p), kZeroBytes / 4), (int)threadIdx.x, (int)blockDim.x);
}
__device__ __forceinline__ bool zeroes(const SortPass& a) {
  if ((int)blockIdx.x < a.groups) return false;
  zero_piece(a.zero, a.zero_end, (int)blockIdx.x - a.groups);
  return true;
}

__device__ __forceinline__ uint32_t sort_key(const SortPass& a, int64_t i) {
  if (!a.ids) return a.key[i];
  const int64_t id = a.ids[i];
  return id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

__global__ __launch_bounds__(kThreads) void sort_count_kernel(const SortPass a) {
  __shared__ int32_t cnt[1 << kMaxDigit];
  if (zeroes(a)) return;
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

// Exclusive scan of the n counts in place by one work-group: each wave sums a
// contiguous share (256 counts at a time), the shares are scanned, and each
// wave scans its share again from its start.
__global__ __launch_bounds__(kScanThreads) void sort_scan_kernel(const SortPass a, int n) {
  constexpr int W = kScanThreads / 64;
  __shared__ int32_t sums[W];
  if (zeroes(a)) return;
  int32_t* v = a.hist;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int share = (n + W * 256 - 1) / (W * 256) * 256;
  const int lo = min(n, w * share), hi = min(n, lo + share);
  auto load = [&](int i) {  // counts i .. i + 3; the array is padded to whole 256
    return *reinterpret_cast<const int4*>(v + i + 4 * lane);
  };
  int s = 0;
#pragma unroll 4
  for (int i = lo; i < hi; i += 256) {
    const int4 c = load(i);
    s += c.x + c.y + c.z + c.w;
  }
  s = run_sumi<64>(s);
  if (lane == 0) sums[w] = s;
  __syncthreads();
  int run = 0;
  for (int x = 0; x < w; ++x) run += sums[x];
#pragma unroll 4
  for (int i = lo; i < hi; i += 256) {
    int4 c = load(i);
    const int own = c.x + c.y + c.z + c.w;
    int inc = own;
    inc += row_shr<1>(inc);
    inc += row_shr<2>(inc);
    inc += row_shr<4>(inc);
    inc += row_shr<8>(inc);
    const int r0 = __builtin_amdgcn_readlane(inc, 15), r1 = __builtin_amdgcn_readlane(inc, 31),
              r2 = __builtin_amdgcn_readlane(inc, 47), r3 = __builtin_amdgcn_readlane(inc, 63);
    inc += (lane >= 16 ? r0 : 0) + (lane >= 32 ? r1 : 0) + (lane >= 48 ? r2 : 0);
    int at = run + inc - own;
    const int4 o = make_int4(at, at + c.x, at + c.x + c.y, at + c.x + c.y + c.z);
    *reinterpret_cast<int4*>(v + i + 4 * lane) = o;
    run += r0 + r1 + r2 + r3;
  }
}

// The output place of each lane's digit d: equal digits of a wave rank by lane
// (one ballot per digit bit); next[d], the wave's own, moves past them.
__device__ __forceinline__ int place_equal(int32_t* next, uint32_t d, int bits, bool in) {
  const int lane = threadIdx.x & 63;
  uint64_t same = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    same &= (d >> b) & 1 ? m : ~m;
  }
  const int at = in ? next[d] + __popcll(same & ((1ull << lane) - 1)) : 0;
  wave_lds_order();  // every lane has read its start
  if (in && (same >> lane) == 1) next[d] = at + 1;  // the digit's last lane
  wave_lds_order();
  return at;
}

// Each wave places its kSortTile / kWaves consecutive keys in order.
__global__ __launch_bounds__(kThreads) void sort_place_kernel(const SortPass a) {
  __shared__ int32_t next[kWaves][1 << kMaxDigit];
  if (zeroes(a)) return;
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
    const int at = place_equal(next[w], (key[r] >> a.shift) & (bins - 1), a.bits, in);
    if (in) {
      a.key_out[at] = key[r];
      a.pos_out[at] = a.ids ? (uint32_t)i : a.pos[i];
    }
  }
}

// All passes for N <= kSmallSort positions in one work-group, which saves
// launches: a gradient of 4096 x 512 into 20,000 rows takes 35.9 us so and 40.6
// by the passes above, of 2048 positions 30.4 and 38.7.  Each wave holds
// consecutive ones in registers, places them in LDS by digits of 8 bits, and
// takes them up again in order.
constexpr int kSmallSort = 4096, kSmallThreads = 1024, kSmallBits = 8;
__global__ __launch_bounds__(kSmallThreads) void sort_small_kernel(const SortPass a) {
  constexpr int W = kSmallThreads / 64, R = kSmallSort / kSmallThreads, BINS = 1 << kSmallBits;
  __shared__ uint32_t keys[kSmallSort], poss[kSmallSort];
  __shared__ int32_t next[W][BINS];
  __shared__ int32_t sums[BINS / 64];
  if (zeroes(a)) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int N = (int)a.N;
  const int per = (N + W * 64 - 1) / (W * 64);  // rounds of 64 a wave
  uint32_t key[R], pos[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (w * per + r) * 64 + lane;
    key[r] = 0u;
    pos[r] = (uint32_t)i;
    if (r < per && i < N) key[r] = sort_key(a, i);
  }
  for (int shift = 0; shift < a.bits; shift += kSmallBits) {
    for (int b = threadIdx.x; b < W * BINS; b += kSmallThreads) (&next[0][0])[b] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < per && (w * per + r) * 64 + lane < N) atomicAdd(&next[w][(key[r] >> shift) & (BINS - 1)], 1);
    __syncthreads();
    // first places: bins in order, a bin's waves in order
    int total = 0, inc = 0;
    if (threadIdx.x < BINS) {
      for (int v = 0; v < W; ++v) total += next[v][threadIdx.x];
      inc = total;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 63) sums[w] = inc;
    }
    __syncthreads();
    if (threadIdx.x < BINS) {
      int run = inc - total;
      for (int v = 0; v < w; ++v) run += sums[v];
      for (int v = 0; v < W; ++v) {
        const int c = next[v][threadIdx.x];
        next[v][threadIdx.x] = run;
        run += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r < per) {
        const bool in = (w * per + r) * 64 + lane < N;
        const int at = place_equal(next[w], (key[r] >> shift) & (BINS - 1), kSmallBits, in);
        if (in) {
          keys[at] = key[r];
          poss[at] = pos[r];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = (w * per + r) * 64 + lane;
      if (r < per && i < N) {
        key[r] = keys[i];
        pos[r] = poss[i];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (w * per + r) * 64 + lane;
    if (r < per && i < N) {
      a.key_out[i] = key[r];
      a.pos_out[i] = pos[r];
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
  int rows;     // positions per tile
  // embed_sum_kernel's work-groups: `groups` for tiles, `blocks` of columns
  // each; the others zero zero_step rows each, from zero_from on
  int blocks;
  int64_t groups, zero_from, zero_step;
};
constexpr int kMaxZeroRows = 4096;

template <int EPC, bool TAIL>
__device__ __forceinline__ void write_dw(const SumArgs& a, uint32_t id, int col, const float* acc) {
  float* row = a.dW + (int64_t)id * a.H;
  float v[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) v[e] = a.scale * acc[e];
  if (a.accumulate) {
    float old[EPC];
    load_sum<EPC, TAIL>(row, col, a.H, old);
#pragma unroll
    for (int e = 0; e < EPC; ++e) v[e] += old[e];
  }
  store_sum<EPC, TAIL>(row, col, a.H, v);
}

// First sorted position with key >= id, by the whole wave: 64 probes a step.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t N, uint32_t id) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = N;  // key[lo - 1] < id <= key[hi]
  while (hi - lo > 0) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t at = lo + lane * step;
    const int below = __popcll(__ballot(at < hi && key[min(at, N - 1)] < id));
    if (below == 0) return lo;
    lo += (below - 1) * step + 1;
    hi = min(hi, lo - 1 + step);
  }
  return lo;
}

// Zeroes rows [r0, r1) of dW but those whose ids occur.
__device__ __forceinline__ void zero_rows(const SumArgs& a, int64_t r0, int64_t r1, uint8_t* occurs) {
  const int rows = (int)(r1 - r0);
  for (int r = threadIdx.x; r < rows; r += kThreads) occurs[r] = 0;
  __syncthreads();
  for (int64_t i = lower_bound(a.key, a.N, (uint32_t)r0) + threadIdx.x; i < a.N; i += kThreads) {
    const uint32_t k = a.key[i];
    if (k >= r1) break;
    occurs[k - r0] = 1;
  }
  __syncthreads();
  // a narrow row takes a part of the work-group, a power of two of four threads up
  // (rows one by one: 34 MB of 128 columns in 60 us, with the pieces' rule 7.4)
  int part = kThreads;
  while (part >= 8 && part / 2 * 4 >= a.H) part /= 2;
  const int tid = threadIdx.x % part;
  for (int r = threadIdx.x / part; r < rows; r += kThreads / part)
    if (!occurs[r]) zero_values(a.dW + (r0 + r) * a.H, a.H, tid, part);
}

// Work-groups [0, tiles * blocks): one tile of sorted positions by a block of
// columns, kAhead rows in flight.  The others zero `zero_rows` rows each.
template <typename T, bool TAIL>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(const SumArgs a) {
  constexpr int EPC = Elem<T>::kPer16B;
  constexpr int kAhead = 16;
  __shared__ uint8_t occurs[kMaxZeroRows];
  if ((int64_t)blockIdx.x >= a.groups) {
    const int64_t r0 = a.zero_from + ((int64_t)blockIdx.x - a.groups) * a.zero_step;
    zero_rows(a, r0, min(a.V, r0 + a.zero_step), occurs);
    return;
  }
  const int64_t tile = blockIdx.x / a.blocks;
  const int64_t i0 = tile * a.rows;
  const int n = (int)min((int64_t)a.rows, a.N - i0);
  const int col = ((int)(blockIdx.x - tile * a.blocks) * kThreads + (int)threadIdx.x) * EPC;
  // lane l holds position i0 + l; lanes n and up repeat the last
  const int lane = threadIdx.x & 63;
  const uint32_t my_key = a.key[i0 + min(lane, n - 1)], my_pos = a.pos[i0 + min(lane, n - 1)];
  uint32_t cur = __builtin_amdgcn_readfirstlane(my_key);
  const bool starts = i0 == 0 || a.key[i0 - 1] != cur;
  const uint32_t last = __builtin_amdgcn_readlane(my_key, n - 1);
  const bool goes_on = i0 + n < a.N && a.key[min(i0 + n, a.N - 1)] == last;
  const bool in = col < a.H;  // the other lanes stay: their keys are read
  bool head = !starts;
  float acc[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) acc[e] = 0.f;
  auto flush = [&](bool on) {
    if (cur >= a.V || !in) return;
    if (head || on)
      store_sum<EPC, TAIL>(a.part + (tile * 2 + (head ? 0 : 1)) * (int64_t)a.H, col, a.H, acc);
    else
      write_dw<EPC, TAIL>(a, cur, col, acc);
  };
  // The rows of a batch are requested together, without a branch: a store in
  // between would make the next row's wait cover it.  Padded positions are read
  // for nothing; lanes past the row read its start.
  const T* dY = static_cast<const T*>(a.dY);
  const int from = in ? col : 0;
  for (int b0 = 0; b0 < n; b0 += kAhead) {
    u32x4_t raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t p = __builtin_amdgcn_readlane(my_pos, min(b0 + u, n - 1));
      raw[u] = load_vec<T, TAIL>(dY + (int64_t)p * a.H, from, a.H);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (b0 + u < n) {
        const uint32_t k = __builtin_amdgcn_readlane(my_key, b0 + u);
        if (k != cur) {
          flush(false);
          cur = k;
          head = false;
#pragma unroll
          for (int e = 0; e < EPC; ++e) acc[e] = 0.f;
        }
        float v[EPC];
        unpack16(raw[u], v, T());
#pragma unroll
        for (int e = 0; e < EPC; ++e) acc[e] += v[e];
      }
    }
  }
  flush(goes_on);
}

// Joins the run that starts in tile blockIdx.x and goes on past it: a wave adds
// a quarter of the tiles' sums, in order, and the waves' sums are added in
// order.  64 lanes' columns per work-group.
template <int EPC, bool TAIL>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const SumArgs a) {
  __shared__ float sums[kWaves][64 * EPC];
  const int64_t tile = blockIdx.x, i0 = tile * a.rows, i1 = i0 + a.rows;
  if (i1 >= a.N) return;
  const uint32_t cur = a.key[i1];
  if (cur >= a.V || a.key[i1 - 1] != cur) return;  // nothing goes on
  if (i0 > 0 && a.key[i0 - 1] == cur) return;      // it started earlier
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  // tiles that the run reaches after its first
  int64_t more = 0;
  for (bool full = true; full;) {
    const int64_t at = (tile + 1 + more + lane) * a.rows;
    const int c = __popcll(__ballot(at < a.N && a.key[min(at, a.N - 1)] == cur));
    more += c;
    full = c == 64;
  }
  const int col = ((int)blockIdx.y * 64 + lane) * EPC;
  const bool in = col < a.H;
  const int64_t share = (more + 1 + kWaves - 1) / kWaves;
  const int64_t lo = min(more + 1, w * share), hi = min(more + 1, lo + share);
  float acc[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) acc[e] = 0.f;
  if (in) {
    // sum 0 is the first tile's second row, the others the tiles' first rows
    const float* p = a.part + tile * 2 * (int64_t)a.H;
#pragma unroll 8
    for (int64_t c = lo; c < hi; ++c) {
      float v[EPC];
      load_sum<EPC, TAIL>(p + (2 * c + (c == 0 ? 1 : 0)) * (int64_t)a.H, col, a.H, v);
#pragma unroll
      for (int e = 0; e < EPC; ++e) acc[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < EPC; ++e) sums[w][lane * EPC + e] = acc[e];
  __syncthreads();
  if (w != 0 || !in) return;
#pragma unroll
  for (int v = 1; v < kWaves; ++v)
#pragma unroll
    for (int e = 0; e < EPC; ++e) acc[e] += sums[v][lane * EPC + e];
  write_dw<EPC, TAIL>(a, cur, col, acc);
}

struct EmbedLayout {
  size_t key[2], pos[2], hist, part, total;
  int tiles, passes, bits, key_bits;
};

// Short tiles while 64 positions a tile make fewer than four work-groups a CU.
int tile_rows(int64_t N, int H, int dtype) {
  const int64_t groups = ceil_div(N, kTileRows) * ceil_div(H, kThreads * 16 / elem_bytes(dtype));
  return groups < 1024 ? kFewRows : kTileRows;
}

EmbedLayout embed_layout(int64_t N, int64_t V, int H, int dtype) {
  EmbedLayout L{};
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) & ~(size_t)255;
    return o;
  };
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V
  L.key_bits = bits;
  L.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  L.bits = (bits + L.passes - 1) / L.passes;
  L.tiles = (int)ceil_div(N, kSortTile);
  for (int i = 0; i < 2; ++i) L.key[i] = take((size_t)N * 4);
  for (int i = 0; i < 2; ++i) L.pos[i] = take((size_t)N * 4);
  L.hist = take((((size_t)L.tiles << L.bits) + 255) / 256 * 256 * 4);  // whole 256 for the scan
  L.part = take((size_t)ceil_div(N, tile_rows(N, H, dtype)) * 2 * H * 4);
  L.total = cur;
  return L;
}

template <typename T, bool TAIL>
hipError_t sum_and_join(SumArgs a, hipStream_t st) {
  constexpr int EPC = Elem<T>::kPer16B;
  const int64_t tiles = ceil_div(a.N, a.rows);
  a.blocks = (int)ceil_div(a.H, kThreads * EPC);
  a.groups = tiles * a.blocks;
  // four pieces for each of the 256 CUs at least, of 16 KB at least
  const int64_t rest = (a.V - a.zero_from) * a.H * 4;
  const int64_t piece = std::clamp<int64_t>(rest / 1024, 1 << 14, kZeroBytes);
  a.zero_step = std::min<int64_t>(std::max<int64_t>(piece / 4 / a.H, 1), kMaxZeroRows);
  const unsigned grid = (unsigned)(a.groups + ceil_div(a.V - a.zero_from, a.zero_step));
  embed_sum_kernel<T, TAIL><<<grid, kThreads, 0, st>>>(a);
  const dim3 join((unsigned)tiles, (unsigned)ceil_div(a.H, 64 * EPC));
  if (a.N > a.rows) embed_join_kernel<EPC, TAIL><<<join, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

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
  p.bwd_workspace_bytes = N == 0 ? 0 : (int64_t)embed_layout(N, V, H, dtype).total;
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
  const bool tail = P.H % epc != 0;
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(P.N * ceil_div(P.H, epc), kThreads), 1 << 20);
  auto run = [&](auto kern, auto* w, auto* y) { kern<<<grid, kThreads, 0, st>>>(w, ids, y, P.N, P.V, P.H, P.scale); };
  if (P.dtype == MOE_BF16)
    run(tail ? embed_forward_kernel<bf16_t, true> : embed_forward_kernel<bf16_t, false>, (const bf16_t*)W, (bf16_t*)Y);
  else
    run(tail ? embed_forward_kernel<float, true> : embed_forward_kernel<float, false>, (const float*)W, (float*)Y);
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
  const int64_t values = P.V * P.H;
  if (P.N == 0) {
    if (!accumulate && launch_fill_zero(dW, (size_t)values * sizeof(float), st) != hipSuccess)
      return MOE_EHIP;
    return MOE_OK;
  }
  const EmbedLayout L = embed_layout(P.N, P.V, P.H, P.dtype);
  char* ws = (char*)workspace;
  // rows [0, zeroed) of dW are zeroed beside the sort
  int64_t zeroed = accumulate ? P.V : 0;
  SortPass s{};
  s.ids = ids;
  s.hist = (int32_t*)(ws + L.hist);
  s.N = P.N;
  s.V = P.V;
  s.tiles = L.tiles;
  s.bits = L.bits;
  // takes the next slice; the launch's work-groups
  auto grid = [&](int groups, int64_t slice) {
    const int64_t rows = std::min(P.V - zeroed, ceil_div(slice / 4, P.H));
    s.groups = groups;
    s.zero = dW + zeroed * P.H;
    s.zero_end = s.zero + rows * P.H;
    zeroed += rows;
    return (unsigned)(groups + ceil_div(rows * P.H, kZeroBytes / 4));
  };
  if (P.N <= kSmallSort) {
    s.bits = L.key_bits;
    s.key_out = (uint32_t*)(ws + L.key[0]);
    s.pos_out = (uint32_t*)(ws + L.pos[0]);
    const unsigned g = grid(1, kSmallSlice);
    sort_small_kernel<<<g, kSmallThreads, 0, st>>>(s);
    s.key = s.key_out;
    s.pos = s.pos_out;
  }
  for (int i = 0; P.N > kSmallSort && i < L.passes; ++i) {
    s.shift = i * L.bits;
    s.key_out = (uint32_t*)(ws + L.key[i & 1]);
    s.pos_out = (uint32_t*)(ws + L.pos[i & 1]);
    unsigned g = grid(L.tiles, kSliceBytes);
    sort_count_kernel<<<g, kThreads, 0, st>>>(s);
    g = grid(1, kSliceBytes);
    sort_scan_kernel<<<g, kScanThreads, 0, st>>>(s, L.tiles << L.bits);
    g = grid(L.tiles, kSliceBytes);
    sort_place_kernel<<<g, kThreads, 0, st>>>(s);
    s.ids = nullptr;
    s.key = s.key_out;
    s.pos = s.pos_out;
  }
  if (hipGetLastError() != hipSuccess) return MOE_EHIP;
  const SumArgs a{s.key, s.pos, dY, dW, (float*)(ws + L.part), P.N, P.V, P.H, accumulate != 0, P.scale,
                  tile_rows(P.N, P.H, P.dtype), 0, 0, zeroed, 0};
  const bool tail = P.H % (16 / elem_bytes(P.dtype)) != 0;
  const hipError_t err = P.dtype == MOE_BF16
                             ? (tail ? sum_and_join<bf16_t, true>(a, st) : sum_and_join<bf16_t, false>(a, st))
                             : (tail ? sum_and_join<float, true>(a, st) : sum_and_join<float, false>(a, st));
  return err == hipSuccess ? MOE_OK : MOE_EHIP;
}
