// What the grouped products (gmm_rows.hpp, gmm_weights.hpp) share: the rows of an
// expert, loads of operands into LDS.
#pragma once

#include "device_common.hpp"
#include "gemm_lds.hpp"  // loads into LDS, waits, renumbering of work-groups
#include "q8_ops.hpp"

namespace moe {
namespace gmm {

using namespace gemm;

enum class Form {
  NN,  // rows of A by B [E][K][N], bf16
  NT,  // rows of A by B [E][N][K], bf16
  Q8,  // rows of A by B [E][N][K to 128], both e4m3 with scales
  TN,  // A^T B over an expert's rows, bf16
  TN8  // the same with A e4m3 with scales
};

// What a product reads and writes.  Forward and dX: C[row][j] = sum_k A[row][k]
// B(k, j); dW: C[e][i][j] = sum over rows of A[row][i] B[row][j].
struct Args {
  const void *A, *As, *B, *Bs;
  void* C;
  const int32_t* offsets;
  int R, E;
  int K, N;  // columns of A, columns of C
  int accumulate;
  float* part;  // partial sums, where k is split
};

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// A work-group's tile, its waves and its stages of operands in LDS.
template <int BM_, int BN_, int WGM_, int WGN_, int NS_>
struct GShape {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, WAVES = WGM_ * WGN_, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WN = BN / WGN, NS = NS_;
  // Where wave w's part of the tile lies.  Waves w and w + 4 share a SIMD: of eight,
  // the second four are placed so that each half of the tile, upper or left, has one
  // wave on every SIMD, and a tile of which the other half lies past the matrix takes
  // half the multiplications' time.
  static __device__ __forceinline__ int row(int w) {
    return WGM == 4 && WGN == 2 ? (w >> 2) * 2 + (w & 1) : w / WGN;
  }
  static __device__ __forceinline__ int col(int w) {
    if (WGM == 4 && WGN == 2) return ((w >> 1) & 1) ^ (w >> 2);
    return WGM == 2 && WGN == 4 ? (w & 3) ^ ((w >> 2) * 2) : w % WGN;
  }
};

// Rows of expert e, kept inside the matrix whatever the offsets say.
struct Segment {
  int lo, hi;
};
__device__ __forceinline__ Segment segment(const int32_t* offsets, int e, int R) {
  if (!offsets) return Segment{0, R};
  const int lo = min(max(offsets[e], 0), R);
  return Segment{lo, min(max(offsets[e + 1], lo), R)};
}

// 4 bytes a lane from a buffer into LDS at an LDS address
__device__ __forceinline__ void lds_load4_at(const i32x4_t& srd, uint32_t lds_addr, uint32_t voff) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(m0v), "v"(voff), "s"(srd)
               : "memory", "m0");
}

// lds_barrier, with ordinary LDS accesses kept on their side of it
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  lds_barrier();
  asm volatile("" ::: "memory");
}

// A resource over whatever lies from base on: every offset used with it is inside
// its tensor, or kOob.  Not there: its loads give zeros and touch no memory.
__device__ __forceinline__ i32x4_t open_srd(const void* base, bool there = true) { return make_srd(base, there ? 0x7FFFFFF0 : 0); }

// One wave's share of an operand's loads of a step: 1 KiB per instruction, the
// waves in turn.
template <int BYTES, int WAVES>
struct Loader {
  static constexpr int INSTR = BYTES / 1024, PW = (INSTR + WAVES - 1) / WAVES;
  static constexpr bool EVEN = INSTR % WAVES == 0;
  uint32_t off[PW];
  uint32_t tail;  // bit u: load u of the last step lies inside k

  // rows of 128 bytes along k: `rows` of them there, ld bytes apart; `left`: bytes
  // of k in the last step
  __device__ __forceinline__ void along_k(int wave, int lane, int rows, uint32_t ld, int left) {
    tail = 0;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      const int r = (u * WAVES + wave) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
      off[u] = r < rows ? (uint32_t)r * ld + (uint32_t)c * 16 : kOob;
      if (c * 16 < left) tail |= 1u << u;
    }
  }
  // rows of k with COLS bf16 columns, of which `cols` are there; `left`: rows in the
  // last step
  template <int COLS>
  __device__ __forceinline__ void across_k(int wave, int lane, int cols, uint32_t ld, int left) {
    constexpr int RC = COLS / 8, RPI = 64 / RC;
    tail = 0;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      const int k = (u * WAVES + wave) * RPI + lane / RC, c = (lane % RC) ^ trswz<RC>(k);
      off[u] = c * 8 < cols ? (uint32_t)k * ld + (uint32_t)c * 16 : kOob;
      if (k < left) tail |= 1u << u;
    }
  }
  // load u of a step
  __device__ __forceinline__ void issue(int u, const i32x4_t& srd, uint32_t lds, int wave, bool last) const {
    if (EVEN || u * WAVES + wave < INSTR)
      lds_load16_at(srd, lds + (uint32_t)(u * WAVES + wave) * 1024, last && !(tail >> u & 1) ? kOob : off[u]);
  }
};

// Fragments out of LDS: 16 bytes a lane, or eight values of k of a column through
// the transposing loads (rows k to k + 3, and four rows on).
__device__ __forceinline__ u32x4_t ld128(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>((uintptr_t)addr);
}
__device__ __forceinline__ int ld32(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) int*>((uintptr_t)addr);
}
__device__ __forceinline__ u32x4_t ldtr(uint32_t lo_addr, uint32_t hi_off) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_p)(uintptr_t)lo_addr);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_p)(uintptr_t)(lo_addr + hi_off));
  return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// Byte of a lane's first transposing read of the 16 columns from col, in rows of rc
// chunks.
__device__ __forceinline__ uint32_t tr_base(int lane, int rc, int col) {
  const int k = (lane >> 4) * 8 + ((lane & 15) >> 2), at = col + (lane & 3) * 4;
  const int sw = rc >= 16 ? trswz<16>(k) : trswz<8>(k);
  return (uint32_t)(k * rc * 16 + (((at >> 3) ^ sw) << 4) + (((at >> 2) & 1) << 3));
}

}  // namespace gmm
}  // namespace moe
