// Rows in 8 bits, and SwiGLU with activation checkpoints in 8 bits (include/q8.h).
//
// All of it moves a few bytes per operation and is bound by HBM.  A block of 128
// columns is eight lanes with 16 columns each: 16 bytes of e4m3 a lane, and a scale by
// three reductions in DPP operands.  Every value is read once.
#include <algorithm>

#include "device_common.hpp"
#include "moe_internal.h"
#include "q8.h"
#include "q8_ops.hpp"
#include "q8_shapes.hpp"
#include "wave_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kQ8Magic = 0x51385031u;  // "Q8P1"

constexpr int kCols = 16, kLanes = kQBlock / kCols;  // columns of a lane, lanes of a block

// The column of vector c (16 bytes) of a lane in its block.  Either a lane's vectors
// are neighbours, and its 16 numbers of e4m3, or (TURN) the lanes' vectors lie in turn,
// so that a store fills whole lines of memory, and the numbers of e4m3 in pieces.
//  * fp32: in turn (131,072 x 1536 SwiGLU backward 496 us, neighbours 700; unpacked 167,
//    292; 98,304 x 1000 281, 393).
//  * bf16, where 8-bit rows are read and rows are whole lines (LINES): in turn (131,072
//    x 1536 backward 288, 301; unpacked 101, 111); on other widths neighbours (98,304 x
//    1000 167, 153; 65, 57).
//  * bf16, where 8-bit rows are written: neighbours (98,304 x 1000 forward 136, 127; on
//    131,072 x 1536 the same).
// Stores of whole lines, which no kernel here reads again, go past L2 (131,072 x 1536
// bf16 unpacked 101 us, 85 so; backward 288, 280; of 8-bit rows, forward 252, 240), parts
// of lines through it (98,304 x 1000 fp32 backward 285, past L2 405).
template <typename T>
constexpr bool kTurn = Elem<T>::kPer16B == 4;
template <typename T, bool TURN>
__device__ __forceinline__ int column(int lane, int c) {
  constexpr int EPC = Elem<T>::kPer16B;
  return TURN ? (c * kLanes + lane) * EPC : lane * kCols + c * EPC;
}
// The EPC values of a vector at p, of which n (maybe none) are there; the rest 0.
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, int n, float* v) {
  constexpr int EPC = Elem<T>::kPer16B;
  if (n >= EPC) {
    const u32x4_t w = *reinterpret_cast<const u32x4_any_t*>(p);
    unpack16(w, v, T());
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e) v[e] = e < n ? Elem<T>::to_f(p[e]) : 0.f;
  }
}
// A lane's values of a block at p, of which n columns are there; the rest 0.
template <typename T, bool TURN>
__device__ __forceinline__ void load_some(const T* p, int lane, int n, float* v) {
  constexpr int EPC = Elem<T>::kPer16B;
#pragma unroll
  for (int c = 0; c < kCols / EPC; ++c) {
    const int at = column<T, TURN>(lane, c);
    load_vec(p + at, n - at, v + c * EPC);
  }
}
template <typename T, bool LINES>
__device__ __forceinline__ void store_some(T* p, int lane, int n, const float* v) {
  constexpr int EPC = Elem<T>::kPer16B;
#pragma unroll
  for (int c = 0; c < kCols / EPC; ++c) {
    const int at = column<T, LINES || kTurn<T>>(lane, c);
    if (n >= at + EPC) {
      const u32x4_any_t w = pack16(v + c * EPC, T());
      if constexpr (LINES)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any_t*>(p + at));
      else
        *reinterpret_cast<u32x4_any_t*>(p + at) = w;
    } else {
#pragma unroll
      for (int e = 0; e < EPC; ++e)
        if (at + e < n) p[at + e] = Elem<T>::from_f(v[c * EPC + e]);
    }
  }
}

// Where blocks go.
struct Packed {
  uint8_t *q, *s;
};
// A launch's blocks: `units` of them from row `first` on.  u / blocks is a product by
// `magic` and a shift (q8_shapes.hpp).
struct Shape8 {
  int64_t first;
  uint32_t units, magic, shift;
  int H, blocks, row_pitch, scale_pitch;
};
// Writes a lane's values of block b of row r, with the block's scale; the row's last
// block writes the scales' padding too.
template <typename T>
__device__ __forceinline__ void put(const Packed& to, const Shape8& sh, int64_t r, int b, int lane, const float* v) {
  const uint32_t byte = q8_scale_byte(q8_amax<kCols>(v, [](float m) { return run8_maxf(m); }));
  const float inv = q8_inverse(byte);
  uint8_t* q = to.q + r * sh.row_pitch + b * kQBlock;
  if constexpr (!kTurn<T>) {
    const u32x4_t w{q8_round4(v, inv), q8_round4(v + 4, inv), q8_round4(v + 8, inv), q8_round4(v + 12, inv)};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(q + lane * kCols));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      __builtin_nontemporal_store(q8_round4(v + 4 * c, inv), reinterpret_cast<uint32_t*>(q + column<T, true>(lane, c)));
  }
  uint8_t* s = to.s + r * sh.scale_pitch;
  if (lane == 0) s[b] = (uint8_t)byte;
  if (b == sh.blocks - 1 && lane < sh.scale_pitch - sh.blocks) s[sh.blocks + lane] = kQOne;
}
template <typename T, bool TURN>
__device__ __forceinline__ void get(const uint8_t* q, const uint8_t* s, const Shape8& sh, int64_t r, int b, int lane,
                                    float* v) {
  constexpr int WORDS = Elem<T>::kPer16B / 4;  // of a vector's numbers
  const float scale = q8_scale(s[r * sh.scale_pitch + b]);
  q += r * sh.row_pitch + b * kQBlock;
  u32x4_t w;
  if constexpr (!TURN) {
    w = *reinterpret_cast<const u32x4_t*>(q + lane * kCols);
  } else if constexpr (WORDS == 2) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint2 x = *reinterpret_cast<const uint2*>(q + column<T, true>(lane, c));
      w[2 * c] = x.x;
      w[2 * c + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint32_t*>(q + column<T, true>(lane, c));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) q8_values4(w[e], scale, v + 4 * e);
}

// Calls f(row, block, lane of the block, the block's place in a matrix, columns there
// from it on) for this thread's block.
template <typename F>
__device__ __forceinline__ void my_block(const Shape8& sh, F f) {
  const int lane = threadIdx.x % kLanes;
  const uint32_t u = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (u >= sh.units) return;
  const uint32_t row = (uint32_t)(((uint64_t)u * sh.magic) >> sh.shift);
  const int b = (int)(u - row * sh.blocks), col = b * kQBlock;
  const int64_t r = sh.first + row;
  f(r, b, lane, r * sh.H + col, sh.H - col);
}

// 65,536 x 2048 bf16: 69 us, 5.9 TB/s; fp32 113 us, 5.9 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_kernel(const T* __restrict__ X, const Packed to, const Shape8 sh) {
  my_block(sh, [&](int64_t r, int b, int lane, int64_t at, int n) {
    float v[kCols];
    load_some<T, kTurn<T>>(X + at, lane, n, v);
    put<T>(to, sh, r, b, lane, v);
  });
}

// 131,072 x 1536 to bf16 85 us, 7.1 TB/s; to fp32 143 us, 7.1 TB/s.
template <typename T, bool LINES>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                          T* __restrict__ X, const Shape8 sh) {
  constexpr bool TURN = LINES || kTurn<T>;
  my_block(sh, [&](int64_t r, int b, int lane, int64_t at, int n) {
    float v[kCols];
    get<T, TURN>(q, s, sh, r, b, lane, v);
    store_some<T, LINES>(X + at, lane, n, v);
  });
}

// 1 / (1 + e^-a): in bf16 through the hardware's exponential and reciprocal, as the
// layer's own SwiGLU does (an IEEE exponential and quotient take longer than the
// bytes), in fp32 exactly rounded steps.
__device__ __forceinline__ float gate(float a, bf16_t) { return logistic(a); }
__device__ __forceinline__ float gate(float a, float) { return 1.f / (1.f + expf(-a)); }

// Below this e^-a, or its reciprocal in bf16's form, leaves fp32's range; what is formed
// from it there takes 64 bits.
constexpr float kLeastGate = -87.f;

// a u / (1 + e^-a) in 32 bits, and whether they may be off by enough to leave open on
// which side of a border of e4m3 or of a scale it lies: in fp32 by five last places at
// most; in bf16 the hardware exponential's argument, a log2(e), is rounded twice, by 1.25
// |a| last places of h, and the rest is another seven.
__device__ __forceinline__ float activated(float a, float u, bf16_t) { return swiglu_h(a, u); }
__device__ __forceinline__ float activated(float a, float u, float) { return a / (1.f + expf(-a)) * u; }
__device__ __forceinline__ bool unsure(float h, float a, bf16_t) {
  return q8_border(h, (uint32_t)fmaf(2.f, fminf(fabsf(a), 96.f), 8.f));  // past 96 no exponential is left
}
__device__ __forceinline__ bool unsure(float h, float, float) { return q8_border(h); }
// h for 8 bits.  (32,768 x 1536 fp32: all numbers are those of 64 bits; all in 32 bits 29 to
// 41 are not.  Of the 491,520 pairs of bf16 mantissas with 2^-9 <= |a| < 2^6 11 are not.
// 131,072 x 1536 bf16 take as long either way, 779 x 1000 5.1 us for 4.3.)
template <typename T>
__device__ __forceinline__ void swiglu_for8(const float* a, const float* u, float* h) {
  bool again = false;
  float least = 0.f;
#pragma unroll
  for (int e = 0; e < kCols; ++e) {
    h[e] = activated(a[e], u[e], T());
    again |= unsure(h[e], a[e], T());
    least = fminf(least, a[e]);
  }
  if (!again && !(least < kLeastGate)) return;
#pragma unroll
  for (int e = 0; e < kCols; ++e)
    if (a[e] < kLeastGate || unsure(h[e], a[e], T()))
      h[e] = q8_to_odd((double)a[e] / (1.0 + exp(-(double)a[e])) * (double)u[e]);
}

// 131,072 x 1536 bf16 with the checkpoint: 240 us, 5.9 TB/s; fp32 414 us, 5.3 TB/s.
template <typename T, bool KEEP>
__global__ __launch_bounds__(kThreads) void swiglu_forward_kernel(const T* __restrict__ A, const T* __restrict__ U,
                                                                  const Packed h, const Packed ka,
                                                                  const Packed ku, const Shape8 sh) {
  my_block(sh, [&](int64_t r, int b, int lane, int64_t at, int n) {
    float a[kCols], u[kCols], v[kCols];
    load_some<T, kTurn<T>>(A + at, lane, n, a);
    load_some<T, kTurn<T>>(U + at, lane, n, u);
    swiglu_for8<T>(a, u, v);
    put<T>(h, sh, r, b, lane, v);
    if constexpr (KEEP) {
      put<T>(ka, sh, r, b, lane, a);
      put<T>(ku, sh, r, b, lane, u);
    }
  });
}

// 131,072 x 1536 bf16: 261 us, 6.2 TB/s; fp32 470 us, 6.0 TB/s.  (Each gate's own look at
// kLeastGate, in place of one a lane: fp32 496.)
template <typename T, bool LINES>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    const uint8_t* __restrict__ Aq, const uint8_t* __restrict__ As, const uint8_t* __restrict__ Uq,
    const uint8_t* __restrict__ Us, const T* dH, T* dA, T* __restrict__ dU, const Shape8 sh) {
  constexpr bool TURN = LINES || kTurn<T>;
  my_block(sh, [&](int64_t r, int b, int lane, int64_t at, int n) {
    float a[kCols], u[kCols], d[kCols];
    get<T, TURN>(Aq, As, sh, r, b, lane, a);
    get<T, TURN>(Uq, Us, sh, r, b, lane, u);
    load_some<T, TURN>(dH + at, lane, n, d);
    float least = 0.f;
#pragma unroll
    for (int e = 0; e < kCols; ++e) least = fminf(least, a[e]);
    auto one = [&](int e) __attribute__((always_inline)) {
      const float g = gate(a[e], T()), dg = d[e] * g;
      u[e] = dg * u[e] * fmaf(a[e], 1.f - g, 1.f);
      d[e] = dg * a[e];
    };
    if (least < kLeastGate) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        if (a[e] < kLeastGate) {
          const double g = 1.0 / (1.0 + exp(-(double)a[e])), dg = (double)d[e] * g;
          u[e] = (float)(dg * (double)u[e] * fma((double)a[e], 1.0 - g, 1.0));
          d[e] = (float)(dg * (double)a[e]);
        } else {
          one(e);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kCols; ++e) one(e);
    }
    store_some<T, LINES>(dA + at, lane, n, u);
    store_some<T, LINES>(dU + at, lane, n, d);
  });
}

// A 128 x 128 block of one matrix per work-group: read once into registers, its
// scale by a reduction over the work-group, written along both axes (the second
// through LDS).  64 x 2048 x 1408 both ways bf16 163 us, 4.5 TB/s; fp32 218 us, 5.1 TB/s.
constexpr int kTrPitch = kQBlock + 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_weights_kernel(
    const T* __restrict__ W, int K, int N, uint8_t* __restrict__ q, uint8_t* __restrict__ s,
    uint8_t* __restrict__ qt, uint8_t* __restrict__ st) {
  __shared__ float red[kThreads / 64];
  __shared__ __attribute__((aligned(16))) uint8_t tile[kQBlock * kTrPitch];
  const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int lane = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int kblocks = q8_blocks(K), nblocks = q8_blocks(N);
  const T* w = W + (int64_t)e * K * N;
  const int col = nb * kQBlock + lane * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = kb * kQBlock + i * 16 + row;
    const T* from = w + (int64_t)min(k, K - 1) * N + min(col, N);
    const int there = k < K ? N - col : 0;
#pragma unroll
    for (int c = 0; c < 8; c += Elem<T>::kPer16B) load_vec(from + c, there - c, v[i] + c);
  }
  const uint32_t byte = q8_scale_byte(q8_amax<64>(&v[0][0], [&](float m) {
    m = run_maxf<64>(m);
    __syncthreads();  // the reads of a first reduction are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  }));
  const float inv = q8_inverse(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = kb * kQBlock + i * 16 + row;
    const uint2 p = make_uint2(q8_round4(v[i], inv), q8_round4(v[i] + 4, inv));
    if (q && k < K)
      *reinterpret_cast<uint2*>(q + ((int64_t)e * K + k) * (nblocks * kQBlock) + col) = p;
    *reinterpret_cast<uint32_t*>(tile + (i * 16 + row) * kTrPitch + lane * 8) = p.x;
    *reinterpret_cast<uint32_t*>(tile + (i * 16 + row) * kTrPitch + lane * 8 + 4) = p.y;
  }
  if (s && threadIdx.x == 0) {
    uint8_t* to = s + ((int64_t)e * kblocks + kb) * q8_scale_pitch(N);
    to[nb] = (uint8_t)byte;
    if (nb == nblocks - 1)
      for (int b = nblocks; b < q8_scale_pitch(N); ++b) to[b] = kQOne;
  }
  if (st && threadIdx.x == 0) {
    uint8_t* to = st + ((int64_t)e * nblocks + nb) * q8_scale_pitch(K);
    to[kb] = (uint8_t)byte;
    if (kb == kblocks - 1)
      for (int b = kblocks; b < q8_scale_pitch(K); ++b) to[b] = kQOne;
  }
  if (!qt) return;
  __syncthreads();
  // thread t: column t / 2 of the block, one half of its 128 rows
  const int n = threadIdx.x >> 1, k0 = (threadIdx.x & 1) * 64;
  if (nb * kQBlock + n >= N) return;
  uint8_t* to = qt + ((int64_t)e * N + nb * kQBlock + n) * (kblocks * kQBlock) + kb * kQBlock + k0;
#pragma unroll
  for (int c = 0; c < 64; c += 16) {
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* from = tile + (k0 + c + i * 4) * kTrPitch + n;
      word[i] = (uint32_t)from[0] | (uint32_t)from[kTrPitch] << 8 | (uint32_t)from[2 * kTrPitch] << 16 |
                (uint32_t)from[3 * kTrPitch] << 24;
    }
    *reinterpret_cast<u32x4_t*>(to + c) = u32x4_t{word[0], word[1], word[2], word[3]};
  }
}

// Whether the rows of a matrix are whole lines of memory.
template <typename T>
bool whole_lines(const q8_plan_t& P, const void* a, const void* b) {
  return P.H * sizeof(T) % 128 == 0 && ((uintptr_t)a | (uintptr_t)b) % 128 == 0;
}

// Calls f(shape, work-groups) for the launches that cover all rows.
template <typename F>
int in_launches(const q8_plan_t& P, F f) {
  static_assert(kThreads == kQ8GroupThreads && kThreads / kLanes == kQ8GroupBlocks, "a work-group's blocks");
  const int blocks = q8_blocks(P.H);
  (void)hipGetLastError();
  for (int64_t first = 0; first < P.N;) {
    const Q8Launch l = q8_launch(P.N - first, blocks);
    f(Shape8{first, l.units, l.magic, l.shift, P.H, blocks, P.row_pitch, P.scale_pitch}, l.groups);
    if (hipGetLastError() != hipSuccess) return MOE_EHIP;
    first += l.rows;
  }
  return MOE_OK;
}
bool plan_ok(const q8_plan_t* p) { return p != nullptr && p->magic == kQ8Magic; }
template <typename T>
int unpack(const q8_plan_t& P, const void* q, const void* s, void* X, void* stream) {
  return in_launches(P, [&](const Shape8& sh, unsigned groups) {
    auto kern = whole_lines<T>(P, X, X) ? unpack_kernel<T, true> : unpack_kernel<T, false>;
    kern<<<groups, kThreads, 0, (hipStream_t)stream>>>((const uint8_t*)q, (const uint8_t*)s, (T*)X, sh);
  });
}

// q on a 16-byte step, s on a 4-byte step, both there
bool pair_ok(const void* q, const void* s) {
  return q && s && (uintptr_t)q % 16 == 0 && (uintptr_t)s % 4 == 0;
}
bool elem_ok(const q8_plan_t& P, const void* p) { return p && (uintptr_t)p % elem_bytes(P.dtype) == 0; }
Packed packed(void* q, void* s) { return Packed{(uint8_t*)q, (uint8_t*)s}; }
int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int q8_plan(int64_t N, int32_t H, int32_t dtype, q8_plan_t* out) {
  if (!out || N < 0 || H < 1) return MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (H > 65536 || N >= ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
  q8_plan_t p{};
  p.magic = kQ8Magic;
  p.dtype = dtype;
  p.N = N;
  p.H = H;
  p.row_pitch = q8_row_pitch(H);
  p.scale_pitch = q8_scale_pitch(H);
  *out = p;
  return MOE_OK;
}

MOE_API int q8_pack(const q8_plan_t* plan, const void* X, void* q, void* s, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  if (plan->N == 0) return MOE_OK;
  if (!elem_ok(*plan, X) || !pair_ok(q, s)) return MOE_EINVAL;
  return in_launches(*plan, [&](const Shape8& sh, unsigned groups) {
    if (plan->dtype == MOE_BF16)
      pack_kernel<bf16_t><<<groups, kThreads, 0, (hipStream_t)stream>>>((const bf16_t*)X, packed(q, s), sh);
    else
      pack_kernel<float><<<groups, kThreads, 0, (hipStream_t)stream>>>((const float*)X, packed(q, s), sh);
  });
}

MOE_API int q8_unpack(const q8_plan_t* plan, const void* q, const void* s, void* X, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  if (plan->N == 0) return MOE_OK;
  if (!elem_ok(*plan, X) || !pair_ok(q, s)) return MOE_EINVAL;
  return plan->dtype == MOE_BF16 ? unpack<bf16_t>(*plan, q, s, X, stream) : unpack<float>(*plan, q, s, X, stream);
}

MOE_API int q8_pack_weights(int32_t E, int32_t K, int32_t N, int32_t dtype, const void* W, void* q,
                            void* s, void* qt, void* st, void* stream) {
  if (E < 0 || K < 1 || N < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_EINVAL;
  if (K > 65536 || N > 65536 || E > 65535) return MOE_EUNSUPPORTED;
  if (E == 0) return MOE_OK;
  if (!W || (uintptr_t)W % elem_bytes(dtype) || (!q && !qt)) return MOE_EINVAL;
  if ((q || s) && !pair_ok(q, s)) return MOE_EINVAL;
  if ((qt || st) && !pair_ok(qt, st)) return MOE_EINVAL;
  const dim3 grid(q8_blocks(K), q8_blocks(N), E);
  (void)hipGetLastError();
  if (dtype == MOE_BF16)
    pack_weights_kernel<bf16_t><<<grid, kThreads, 0, (hipStream_t)stream>>>(
        (const bf16_t*)W, K, N, (uint8_t*)q, (uint8_t*)s, (uint8_t*)qt, (uint8_t*)st);
  else
    pack_weights_kernel<float><<<grid, kThreads, 0, (hipStream_t)stream>>>(
        (const float*)W, K, N, (uint8_t*)q, (uint8_t*)s, (uint8_t*)qt, (uint8_t*)st);
  return launched();
}

namespace {
template <typename T>
int swiglu_forward(const q8_plan_t& P, const void* A, const void* U, const Packed& h, const Packed& ka,
                   const Packed& ku, void* stream) {
  return in_launches(P, [&](const Shape8& sh, unsigned groups) {
    if (ka.q)
      swiglu_forward_kernel<T, true><<<groups, kThreads, 0, (hipStream_t)stream>>>((const T*)A, (const T*)U, h, ka, ku, sh);
    else
      swiglu_forward_kernel<T, false><<<groups, kThreads, 0, (hipStream_t)stream>>>((const T*)A, (const T*)U, h, ka, ku, sh);
  });
}
template <typename T>
int swiglu_backward(const q8_plan_t& P, const void* Aq, const void* As, const void* Uq, const void* Us,
                    const void* dH, void* dA, void* dU, void* stream) {
  return in_launches(P, [&](const Shape8& sh, unsigned groups) {
    auto kern = whole_lines<T>(P, dA, dU) ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>;
    kern<<<groups, kThreads, 0, (hipStream_t)stream>>>((const uint8_t*)Aq, (const uint8_t*)As, (const uint8_t*)Uq,
                                                       (const uint8_t*)Us, (const T*)dH, (T*)dA, (T*)dU, sh);
  });
}
}  // namespace

MOE_API int q8_swiglu_forward(const q8_plan_t* plan, const void* A, const void* U, void* Hq, void* Hs,
                              void* Aq, void* As, void* Uq, void* Us, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const q8_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!elem_ok(P, A) || !elem_ok(P, U) || !pair_ok(Hq, Hs)) return MOE_EINVAL;
  if ((Aq || As || Uq || Us) && (!pair_ok(Aq, As) || !pair_ok(Uq, Us))) return MOE_EINVAL;
  const Packed h = packed(Hq, Hs), ka = packed(Aq, As), ku = packed(Uq, Us);
  return P.dtype == MOE_BF16 ? swiglu_forward<bf16_t>(P, A, U, h, ka, ku, stream)
                             : swiglu_forward<float>(P, A, U, h, ka, ku, stream);
}

MOE_API int q8_swiglu_backward(const q8_plan_t* plan, const void* Aq, const void* As, const void* Uq,
                               const void* Us, const void* dH, void* dA, void* dU, void* stream) {
  if (!plan_ok(plan)) return MOE_EINVAL;
  const q8_plan_t& P = *plan;
  if (P.N == 0) return MOE_OK;
  if (!pair_ok(Aq, As) || !pair_ok(Uq, Us) || !elem_ok(P, dH) || !elem_ok(P, dA) || !elem_ok(P, dU))
    return MOE_EINVAL;
  return P.dtype == MOE_BF16 ? swiglu_backward<bf16_t>(P, Aq, As, Uq, Us, dH, dA, dU, stream)
                             : swiglu_backward<float>(P, Aq, As, Uq, Us, dH, dA, dU, stream);
}
