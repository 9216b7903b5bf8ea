// Matrix products grouped by expert, with ragged sizes (include/gmm.h).
#include <algorithm>

#include "device_common.hpp"
#include "gmm.h"
#include "moe_internal.h"
#include "q8_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr uint32_t kGmmMagic = 0x474d4d31u;  // "GMM1"

// Rows of expert e, kept inside the matrix whatever the offsets say.
struct Segment {
  int lo, hi;
};
__device__ __forceinline__ Segment segment(const int32_t* offsets, int e, int R) {
  if (!offsets) return Segment{0, R};
  const int lo = min(max(offsets[e], 0), R);
  return Segment{lo, min(max(offsets[e + 1], lo), R)};
}

__device__ __forceinline__ int xcd_contiguous(int L, int total) {
  const int xcd = L & 7, slot = L >> 3;
  const int q = total >> 3, r = total & 7;
  return xcd < r ? xcd * (q + 1) + slot : r * (q + 1) + (xcd - r) * q + slot;
}

struct Tile {
  int e, m0, row_end, nt;
};

// The tile of work-group bid: row tiles of bm rows never cross an expert's end;
// an expert's tiles run column tile by column tile, so that the row tiles that
// read one part of its weights start together, on one XCD (ids go to the eight
// XCDs in turn, the tiles to each in one piece).  Every wave finds it for itself:
// 64 experts at a time, one a lane, whose tile counts are added up over the lanes.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int R, int bm, int ntiles, int bid,
                                          Tile& t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, tiles = 0, cum = 0, total = 0;  // of the chunk last read; cum: including this lane's
  auto chunk = [&](int e0) {
    lo = tiles = 0;
    if (e0 + lane < E) {
      const Segment s = segment(offsets, e0 + lane, R);
      lo = s.lo;
      tiles = (s.hi - s.lo + bm - 1) / bm;
    }
    cum = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(cum, o);
      if (lane >= o) cum += v;
    }
  };
  const int chunks = (E + 63) / 64;
  for (int c = 0; c < chunks; ++c) {
    chunk(c * 64);
    total += __builtin_amdgcn_readlane(cum, 63);
  }
  if (bid >= total * ntiles) return false;
  const int lid = xcd_contiguous(bid, total * ntiles);
  int base = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) chunk(c * 64);
    const int all = __builtin_amdgcn_readlane(cum, 63);
    if (lid < (base + all) * ntiles) {
      const unsigned long long past = __ballot(lid < (base + cum) * ntiles);
      const int l = __ffsll((long long)past) - 1;
      const int me = __builtin_amdgcn_readlane(tiles, l);
      const int first = base + __builtin_amdgcn_readlane(cum, l) - me;
      const int local = lid - first * ntiles;
      if (me <= 0 || local < 0) return false;
      t.e = c * 64 + l;
      t.nt = local / me;
      const int seg0 = __builtin_amdgcn_readlane(lo, l);
      t.m0 = seg0 + (local - t.nt * me) * bm;
      t.row_end = segment(offsets, t.e, R).hi;
      t.row_end = __builtin_amdgcn_readfirstlane(t.row_end);
      return t.nt < ntiles && t.m0 < t.row_end;
    }
    base += all;
  }
  return false;
}

// What a product reads and writes.  Forward and dX: C[row][j] = sum_k A[row][k]
// B(k, j); dW: C[e][i][j] = sum over rows of A[row][i] B[row][j].
struct Args {
  const void *A, *As, *B, *Bs;
  void* C;
  const int32_t* offsets;
  int R, E;
  int K, N;  // columns of A, columns of C
  int accumulate;
};

enum class Form {
  NN,  // B [E][K][N], bf16
  NT,  // B [E][N][K], bf16
  Q8   // A and B [E][N][K] in 8 bits
};

constexpr int kTile = 64, kStep = 32, kPitch = kStep + 8;

// 64 x 64 of the sum over 32 values of k, from bf16 tiles [64][kPitch] in LDS.
__device__ __forceinline__ void multiply(const bf16_t* a, const bf16_t* b, f32x4_t (&acc)[4]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto frag = [&](const bf16_t* t, int row) {
    return __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(t + (row + (lane & 15)) * kPitch + (lane >> 4) * 8));
  };
  const bf16x8_t fa = frag(a, wave * 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, frag(b, j * 16), acc[j], 0, 0, 0);
}

template <Form F>
__global__ __launch_bounds__(kThreads) void rows_kernel(const Args p, int ntiles) {
  __shared__ __attribute__((aligned(16))) bf16_t a[kTile * kPitch], b[kTile * kPitch];
  Tile t;
  if (!find_tile(p.offsets, p.E, p.R, kTile, ntiles, blockIdx.x, t)) return;
  const int K = p.K, N = p.N, n0 = t.nt * kTile;
  const int kp = q8_row_pitch(K), sp = q8_scale_pitch(K);
  f32x4_t acc[4] = {};
  for (int k0 = 0; k0 < K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int r = i / kStep, k = k0 + i % kStep;
      const int64_t row = t.m0 + r;
      bf16_t v = 0, w = 0;
      if (row < t.row_end && k < K) {
        if constexpr (F == Form::Q8) {
          float x[4];
          q8_values4(((const uint8_t*)p.A)[row * kp + k], q8_scale(((const uint8_t*)p.As)[row * sp + k / kQBlock]), x);
          v = f2bf(x[0]);
        } else {
          v = ((const bf16_t*)p.A)[row * K + k];
        }
      }
      const int64_t n = n0 + r;
      if (n < N && k < K) {
        if constexpr (F == Form::Q8) {
          float x[4];
          const int64_t blocks = q8_blocks(N);
          q8_values4(((const uint8_t*)p.B)[(t.e * (int64_t)N + n) * kp + k],
                     q8_scale(((const uint8_t*)p.Bs)[(t.e * blocks + n / kQBlock) * sp + k / kQBlock]), x);
          w = f2bf(x[0]);
        } else if constexpr (F == Form::NT) {
          w = ((const bf16_t*)p.B)[(t.e * (int64_t)N + n) * K + k];
        } else {
          w = ((const bf16_t*)p.B)[(t.e * (int64_t)K + k) * N + n];
        }
      }
      a[r * kPitch + i % kStep] = v;
      b[r * kPitch + i % kStep] = w;
    }
    __syncthreads();
    multiply(a, b, acc);
    __syncthreads();
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = t.m0 + wave * 16 + (lane >> 4) * 4 + q;
      const int n = n0 + j * 16 + (lane & 15);
      if (row < t.row_end && n < N) ((bf16_t*)p.C)[row * N + n] = f2bf(acc[j][q]);
    }
}

template <bool Q8>
__global__ __launch_bounds__(kThreads) void weights_kernel(const Args p) {
  __shared__ __attribute__((aligned(16))) bf16_t a[kTile * kPitch], b[kTile * kPitch];
  const int K = p.K, N = p.N, e = blockIdx.z;
  const int i0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  const int kp = q8_row_pitch(K), sp = q8_scale_pitch(K);
  const Segment s = segment(p.offsets, e, p.R);
  f32x4_t acc[4] = {};
  for (int r0 = s.lo; r0 < s.hi; r0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
      const int c = i % kTile;
      const int64_t row = r0 + i / kTile;
      bf16_t v = 0, w = 0;
      if (row < s.hi && i0 + c < K) {
        if constexpr (Q8) {
          float x[4];
          q8_values4(((const uint8_t*)p.A)[row * kp + i0 + c],
                     q8_scale(((const uint8_t*)p.As)[row * sp + (i0 + c) / kQBlock]), x);
          v = f2bf(x[0]);
        } else {
          v = ((const bf16_t*)p.A)[row * K + i0 + c];
        }
      }
      if (row < s.hi && n0 + c < N) w = ((const bf16_t*)p.B)[row * N + n0 + c];
      a[c * kPitch + i / kTile] = v;
      b[c * kPitch + i / kTile] = w;
    }
    __syncthreads();
    multiply(a, b, acc);
    __syncthreads();
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + wave * 16 + (lane >> 4) * 4 + q, n = n0 + j * 16 + (lane & 15);
      if (i < K && n < N) {
        float* c = (float*)p.C + ((int64_t)e * K + i) * N + n;
        *c = p.accumulate ? *c + acc[j][q] : acc[j][q];
      }
    }
}

bool plan_ok(const gmm_plan_t* p, int operands) {
  return p != nullptr && p->magic == kGmmMagic && p->operands == operands;
}
bool aligned(const void* p, int to) { return p && (uintptr_t)p % to == 0; }
// 0: go on
int check_call(const gmm_plan_t& P, const int32_t* offsets, const void* workspace, size_t bytes,
               int64_t needed) {
  if (offsets ? (uintptr_t)offsets % 4 != 0 : P.E != 1) return MOE_EINVAL;
  if (needed > 0 && !aligned(workspace, 256)) return MOE_EINVAL;
  return bytes < (size_t)needed ? MOE_EWORKSPACE : MOE_OK;
}
int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }

// Row tiles of all experts at most.
int64_t row_tiles(int64_t R, int E, int bm) { return R / bm + std::min<int64_t>(E, R); }

template <Form F>
int rows_product(const Args& a, hipStream_t st) {
  const int ntiles = (int)ceil_div(a.N, kTile);
  (void)hipGetLastError();
  rows_kernel<F><<<(unsigned)(row_tiles(a.R, a.E, kTile) * ntiles), kThreads, 0, st>>>(a, ntiles);
  return launched();
}

template <bool Q8>
int weights_product(const Args& a, hipStream_t st) {
  (void)hipGetLastError();
  weights_kernel<Q8><<<dim3(ceil_div(a.K, kTile), ceil_div(a.N, kTile), a.E), kThreads, 0, st>>>(a);
  return launched();
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API int gmm_plan(int64_t R, int32_t K, int32_t N, int32_t E, int32_t operands, gmm_plan_t* out) {
  if (!out || R < 0 || K < 1 || N < 1 || E < 0 || (E == 0 && R > 0)) return MOE_EINVAL;
  if (operands != GMM_BF16 && operands != GMM_Q8) return MOE_EINVAL;
  if (N % 8 || (operands == GMM_BF16 && K % 8)) return MOE_EINVAL;
  if (K > 65536 || N > 65536 || E > 1024 || R >= ((int64_t)1 << 31) - 65536) return MOE_EUNSUPPORTED;
  if (2 * (int64_t)K * N >= ((int64_t)1 << 31) || R * std::max(K, N) >= ((int64_t)1 << 40)) return MOE_EUNSUPPORTED;
  gmm_plan_t p{};
  p.magic = kGmmMagic;
  p.operands = operands;
  p.R = R;
  p.K = K;
  p.N = N;
  p.E = E;
  p.row_pitch = operands == GMM_BF16 ? 2 * K : q8_row_pitch(K);
  *out = p;
  return MOE_OK;
}

MOE_API int gmm_forward(const gmm_plan_t* plan, const void* X, const void* W, const int32_t* offsets,
                        void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::NN>(Args{X, nullptr, W, nullptr, Y, offsets, (int)P.R, P.E, P.K, P.N, 0}, (hipStream_t)stream);
}

MOE_API int gmm_backward_dx(const gmm_plan_t* plan, const void* dY, const void* W, const int32_t* offsets,
                            void* dX, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(dY, 16) || !aligned(W, 16) || !aligned(dX, 16)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::NT>(Args{dY, nullptr, W, nullptr, dX, offsets, (int)P.R, P.E, P.N, P.K, 0}, (hipStream_t)stream);
}

MOE_API int gmm_backward_dw(const gmm_plan_t* plan, const void* X, const void* dY, const int32_t* offsets,
                            float* dW, int32_t accumulate, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!plan_ok(plan, GMM_BF16)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.E == 0) return MOE_OK;
  if (!aligned(dW, 16) || (P.R > 0 && (!aligned(X, 16) || !aligned(dY, 16)))) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.bwd_workspace_bytes)) return bad;
  return weights_product<false>(Args{X, nullptr, dY, nullptr, dW, offsets, (int)P.R, P.E, P.K, P.N, accumulate != 0}, (hipStream_t)stream);
}

MOE_API int gmm8_forward(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* Wq,
                         const void* Ws, const int32_t* offsets, void* Y, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_Q8)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.R == 0) return MOE_OK;
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(Xs, 4) || !aligned(Ws, 4)) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.fwd_workspace_bytes)) return bad;
  return rows_product<Form::Q8>(Args{Xq, Xs, Wq, Ws, Y, offsets, (int)P.R, P.E, P.K, P.N, 0}, (hipStream_t)stream);
}

MOE_API int gmm8_backward_dw(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* dY,
                             const int32_t* offsets, float* dW, int32_t accumulate, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!plan_ok(plan, GMM_Q8)) return MOE_EINVAL;
  const gmm_plan_t& P = *plan;
  if (P.E == 0) return MOE_OK;
  if (!aligned(dW, 16) || (P.R > 0 && (!aligned(Xq, 16) || !aligned(Xs, 4) || !aligned(dY, 16)))) return MOE_EINVAL;
  if (const int bad = check_call(P, offsets, workspace, workspace_bytes, P.bwd_workspace_bytes)) return bad;
  return weights_product<true>(Args{Xq, Xs, dY, nullptr, dW, offsets, (int)P.R, P.E, P.K, P.N, accumulate != 0}, (hipStream_t)stream);
}
