// Matrix products grouped by expert, with ragged sizes (include/gmm.h).
//
// One kernel body for all products.  A work-group of W waves computes a BM x BN
// tile of one expert's output.  Both operands go from HBM straight into LDS
// (buffer loads that write LDS, 16 bytes a lane), in steps of 128 bytes of k for
// operands whose rows run along k, of 64 rows of k for the others: 64 bf16 or 128
// e4m3 numbers of k.  Two such stages alternate.  A step's fragments are read in
// two halves of k, the second while the first is multiplied, the first of the next
// step while the second is, so that half a step lies in registers and the stage
// can be filled again from the middle of the step on: a load has one step's
// multiplications (2,048 cycles of a SIMD and more in the large tiles) to arrive.
//
//  * Operands along k (X, dY; W in dX; all of the 8-bit product) lie in LDS as rows
//    of 128 bytes; 16-byte chunk c of row r sits at c ^ (r / 2 % 8), so that 16
//    rows' reads of one chunk cover all 64 banks.
//  * The others (W [K][N] in the forward product; X and dY in dW) stay as they are
//    and are read with the transposing LDS loads, as in gemm_lds.hpp.
//  * e4m3 goes through v_mfma_scale_f32_32x32x64_f8f6f4, which takes the scales'
//    bytes itself: a lane's operand is a row's word of four bytes, one for each of
//    four steps, loaded into LDS once per four steps.  No instruction is spent on
//    scales otherwise, and the sum stays in the accumulators.
//  * W's fragments are the instruction's first operand, X's the second, so that a
//    lane's accumulators hold four neighbours of one output row.
#include <algorithm>

#include "device_common.hpp"
#include "gemm_lds.hpp"  // loads into LDS, waits, renumbering of work-groups
#include "gmm.h"
#include "moe_internal.h"
#include "q8_ops.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

using namespace gemm;

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
  NN,  // rows of A by B [E][K][N], bf16
  NT,  // rows of A by B [E][N][K], bf16
  Q8,  // rows of A by B [E][N][K to 128], both e4m3 with scales
  TN,  // A^T B over an expert's rows, bf16
  TN8  // the same with A e4m3 with scales
};
constexpr bool over_rows(Form f) { return f == Form::TN || f == Form::TN8; }

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

template <int BM_, int BN_, int WGM_, int WGN_>
struct GShape {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, WAVES = WGM_ * WGN_, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WN = BN / WGN;
};

// LDS of a work-group: two stages of A and B, two slots of scales' words (a word
// per row of A and, for each 128 columns of B, one in 64 copies); the finished
// tile takes the stages over.
template <Form F, class S>
struct GCfg {
  static constexpr int STEP = 128;  // bytes of k; rows of k: 64
  static constexpr int A_BYTES = S::BM * STEP, B_BYTES = S::BN * STEP, STAGE = A_BYTES + B_BYTES;
  static constexpr int A_SLOTS = (S::BM + 63) / 64, B_SLOTS = (S::BN + 127) / 128;  // 256 bytes each
  static constexpr int SCALES = F == Form::Q8 ? (A_SLOTS + B_SLOTS) * 256 : 0;
  static constexpr int OUT = over_rows(F) ? 0 : S::WAVES * S::WM * (S::WN + 8) * 2;
  static constexpr int LDS = std::max(2 * STAGE + 2 * SCALES, OUT);
  static_assert(LDS <= kLdsBytes, "LDS");
};

// One wave's share of an operand's loads of a step: 1 KiB per instruction.
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
      const int r = (wave * PW + u) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
      off[u] = r < rows ? (uint32_t)r * ld + (uint32_t)c * 16 : kOob;
      if (c * 16 < left) tail |= 1u << u;
    }
  }
  // 64 rows of k with COLS bf16 columns, of which `cols` are there; `left`: rows in
  // the last step
  template <int COLS>
  __device__ __forceinline__ void across_k(int wave, int lane, int cols, uint32_t ld, int left) {
    constexpr int RC = COLS / 8, RPI = 64 / RC;
    tail = 0;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      const int k = (wave * PW + u) * RPI + lane / RC, c = (lane % RC) ^ trswz<RC>(k);
      off[u] = c * 8 < cols ? (uint32_t)k * ld + (uint32_t)c * 16 : kOob;
      if (k < left) tail |= 1u << u;
    }
  }
  __device__ __forceinline__ void issue(const i32x4_t& srd, uint32_t lds, int wave, bool last) const {
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      if (EVEN || wave * PW + u < INSTR)
        lds_load16_at(srd, lds + (uint32_t)(wave * PW + u) * 1024, last && !(tail >> u & 1) ? kOob : off[u]);
    }
  }
};

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
// its tensor, or kOob.
__device__ __forceinline__ i32x4_t open_srd(const void* base) { return make_srd(base, 0x7FFFFFF0); }

template <Form F, class S>
__global__ __launch_bounds__(S::THREADS) void gmm_kernel(const Args p, int mtiles, int ntiles) {
  using C = GCfg<F, S>;
  constexpr bool Q8 = F == Form::Q8, ROWS = over_rows(F);
  constexpr int FR = Q8 ? 32 : 16;  // rows and columns of a fragment
  constexpr int FM = S::WM / FR, FN = S::WN / FR;
  static_assert(FM >= 1 && FN >= 1, "wave tile");
  constexpr bool A_K = !ROWS, B_K = F == Form::NT || Q8;
  constexpr int RCA = S::BM / 8, RCB = S::BN / 8;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WGN, wn = wave % S::WGN;

  // ---- the tile
  int e, m0, n0, m_end, k_len;  // rows of C up to m_end; k_len in numbers
  int64_t k0 = 0;               // first row of k
  if constexpr (ROWS) {
    const int total = gridDim.x, per = mtiles * ntiles;
    const int lid = xcd_contiguous(blockIdx.x, total);
    e = lid / per;
    const int rem = lid - e * per;
    n0 = rem / mtiles;
    m0 = (rem - n0 * mtiles) * S::BM;
    n0 *= S::BN;
    const Segment s = segment(p.offsets, e, p.R);
    k0 = __builtin_amdgcn_readfirstlane(s.lo);
    k_len = __builtin_amdgcn_readfirstlane(s.hi - s.lo);
    m_end = p.K;
  } else {
    Tile t;
    if (!find_tile(p.offsets, p.E, p.R, S::BM, ntiles, blockIdx.x, t)) return;
    e = t.e;
    m0 = t.m0;
    m_end = t.row_end;
    n0 = t.nt * S::BN;
    k_len = p.K;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  n0 = __builtin_amdgcn_readfirstlane(n0);
  m_end = __builtin_amdgcn_readfirstlane(m_end);
  constexpr int KT = Q8 ? 128 : 64;  // numbers of k in a step
  const int nk = (k_len + KT - 1) / KT, last = nk - 1;
  const int kp = Q8 || F == Form::TN8 ? q8_row_pitch(p.K) : 0, sp = Q8 || F == Form::TN8 ? q8_scale_pitch(p.K) : 0;

  // ---- loads
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_void_p)smem));
  Loader<C::A_BYTES, S::WAVES> la;
  Loader<C::B_BYTES, S::WAVES> lb;
  const unsigned char *ap, *bp;  // where step 0 of the tile's operand starts
  int64_t a_step, b_step;        // bytes from a step to the next
  const int left = k_len - last * KT;
  if constexpr (A_K) {
    const int64_t ld = Q8 ? kp : 2 * (int64_t)p.K;
    ap = (const unsigned char*)p.A + m0 * ld;
    a_step = C::STEP;
    la.along_k(wave, lane, m_end - m0, (uint32_t)ld, Q8 ? C::STEP : left * 2);
  } else if constexpr (F == Form::TN) {
    const int64_t ld = 2 * (int64_t)p.K;
    ap = (const unsigned char*)p.A + k0 * ld + (int64_t)m0 * 2;
    a_step = 64 * ld;
    la.template across_k<S::BM>(wave, lane, p.K - m0, (uint32_t)ld, left);
  } else {
    ap = nullptr;
    a_step = 0;
  }
  if constexpr (B_K) {
    const int64_t ld = Q8 ? kp : 2 * (int64_t)p.K;
    bp = (const unsigned char*)p.B + ((int64_t)e * p.N + n0) * ld;
    b_step = C::STEP;
    lb.along_k(wave, lane, p.N - n0, (uint32_t)ld, Q8 ? C::STEP : left * 2);
  } else {
    const int64_t ld = 2 * (int64_t)p.N;
    bp = (const unsigned char*)p.B + (ROWS ? k0 : (int64_t)e * p.K) * ld + (int64_t)n0 * 2;
    b_step = 64 * ld;
    lb.template across_k<S::BN>(wave, lane, p.N - n0, (uint32_t)ld, left);
  }
  // scales: rows of A in A_SLOTS instructions, 128 columns of B in one each
  const unsigned char *as = nullptr, *bs = nullptr;
  if constexpr (Q8) {
    as = (const unsigned char*)p.As + (int64_t)m0 * sp;
    bs = (const unsigned char*)p.Bs + ((int64_t)e * q8_blocks(p.N) + n0 / kQBlock) * sp;
  }
  auto issue_scales = [&](int group) __attribute__((always_inline)) {
    const uint32_t slot = lds0 + 2 * C::STAGE + (uint32_t)(group & 1) * C::SCALES;
#pragma unroll
    for (int i = 0; i < (C::A_SLOTS + C::B_SLOTS + S::WAVES - 1) / S::WAVES; ++i) {
      const int ins = i * S::WAVES + wave;
      if (ins < C::A_SLOTS) {
        const int r = ins * 64 + lane;
        const uint32_t off = r < m_end - m0 ? (uint32_t)(r * sp + group * 4) : kOob;
        lds_load4_at(open_srd(as), slot + (uint32_t)ins * 256, off);
      } else if (ins < C::A_SLOTS + C::B_SLOTS) {
        const int b = ins - C::A_SLOTS;
        const uint32_t off = n0 + b * kQBlock < p.N ? (uint32_t)(b * sp + group * 4) : kOob;
        lds_load4_at(open_srd(bs), slot + (uint32_t)ins * 256, off);
      }
    }
  };
  // A in 8 bits with columns along its rows: through registers, where it becomes
  // bf16.  16 numbers of one row (one scale) a thread and turn.
  constexpr int TURNS = F == Form::TN8 ? S::BM * 64 / 16 / S::THREADS : 1;
  static_assert(F != Form::TN8 || TURNS * S::THREADS * 16 == S::BM * 64, "A's step must split over the threads");
  u32x4_t a8[TURNS];
  uint32_t a8s[TURNS];
  auto fetch8 = [&](int kt) __attribute__((always_inline)) {
    if constexpr (F == Form::TN8) {
#pragma unroll
      for (int i = 0; i < TURNS; ++i) {
        const int at = i * S::THREADS + threadIdx.x, r = at / (S::BM / 16), c = at % (S::BM / 16) * 16;
        const int64_t row = k0 + (int64_t)kt * 64 + r;
        a8[i] = u32x4_t{0u, 0u, 0u, 0u};
        a8s[i] = kQOne;
        if (kt * 64 + r < k_len && m0 + c < kp) {
          a8[i] = *reinterpret_cast<const u32x4_t*>((const unsigned char*)p.A + row * kp + m0 + c);
          a8s[i] = ((const unsigned char*)p.As)[row * sp + (m0 + c) / kQBlock];
        }
      }
    }
  };
  auto place8 = [&](int stage) __attribute__((always_inline)) {
    if constexpr (F == Form::TN8) {
#pragma unroll
      for (int i = 0; i < TURNS; ++i) {
        const int at = i * S::THREADS + threadIdx.x, r = at / (S::BM / 16), c = at % (S::BM / 16) * 2;
        const float scale = a8s[i] == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(a8s[i] << 23);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a8[i][j], scale, false));
          w[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a8[i][j], scale, true));
        }
        unsigned char* row = smem + stage * C::STAGE + r * (RCA * 16);
        *reinterpret_cast<u32x4_t*>(row + ((c ^ trswz<RCA>(r)) << 4)) = u32x4_t{w[0], w[1], w[2], w[3]};
        *reinterpret_cast<u32x4_t*>(row + (((c + 1) ^ trswz<RCA>(r)) << 4)) = u32x4_t{w[4], w[5], w[6], w[7]};
      }
    }
  };
  auto issue = [&](int kt, int stage) __attribute__((always_inline)) {
    const uint32_t at = lds0 + (uint32_t)stage * C::STAGE;
    if constexpr (F != Form::TN8) la.issue(open_srd(ap + kt * a_step), at, wave, kt == last);
    lb.issue(open_srd(bp + kt * b_step), at + C::A_BYTES, wave, kt == last);
    if constexpr (Q8)
      if (kt % 4 == 0) issue_scales(kt / 4);
    fetch8(kt);
  };

  // ---- fragments
  const int l16 = lane & 15, lg = lane >> 4, l32 = lane & 31, lh = lane >> 5;
  constexpr int NA = A_K ? (Q8 ? 4 : 2) : FM, NB = B_K ? (Q8 ? 4 : 2) : FN;
  uint32_t base_a[NA], base_b[NB];
  {
    const uint32_t smem0 = (uint32_t)reinterpret_cast<uintptr_t>((lds_void_p)smem);
    const int trj = l16 >> 2, trq = l16 & 3;
    // along k: half ks of the step, chunk 4 ks + lg (bf16) or 4 ks + 2 lh + {0, 1};
    // any order of k serves, as both operands have the same
    auto along = [&](int w0, int b) -> uint32_t {
      const int r = w0 + (Q8 ? l32 : l16), c = Q8 ? (b >> 1) * 4 + lh * 2 + (b & 1) : b * 4 + lg;
      return (uint32_t)(r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
    };
    auto across = [&](int rc, int col) -> uint32_t {
      const int k = lg * 8 + trj, sw = rc >= 16 ? trswz<16>(k) : trswz<8>(k);
      return (uint32_t)(k * rc * 16 + (((col >> 3) ^ sw) << 4) + (((col >> 2) & 1) << 3));
    };
#pragma unroll
    for (int b = 0; b < NA; ++b) base_a[b] = smem0 + (A_K ? along(wm * S::WM, b) : across(RCA, wm * S::WM + b * 16 + trq * 4));
#pragma unroll
    for (int b = 0; b < NB; ++b)
      base_b[b] = smem0 + C::A_BYTES + (B_K ? along(wn * S::WN, b) : across(RCB, wn * S::WN + b * 16 + trq * 4));
  }
  auto launder = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NA; ++b) asm volatile("" : "+v"(base_a[b]));
#pragma unroll
    for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(base_b[b]));
  };
  auto ld128 = [](uint32_t addr) __attribute__((always_inline)) -> u32x4_t {
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t*>((uintptr_t)addr);
  };
  auto ldtr = [](uint32_t lo_addr, uint32_t hi_off) __attribute__((always_inline)) -> u32x4_t {
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_p)(uintptr_t)lo_addr);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_p)(uintptr_t)(lo_addr + hi_off));
    return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  constexpr int PARTS = Q8 ? 2 : 1;  // registers of a fragment, in fours
  u32x4_t fa[2][FM][PARTS], fb[2][FN][PARTS];
  auto read_half = [&](int stage, int ks) __attribute__((always_inline)) {
    const uint32_t so = (uint32_t)(stage * C::STAGE);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
        fa[ks][i][q] = A_K ? ld128(base_a[ks * PARTS + q] + so + (uint32_t)(i * FR * 128))
                           : ldtr(base_a[A_K ? 0 : i] + so + (uint32_t)(ks * 32 * RCA * 16), 4 * RCA * 16);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
        fb[ks][j][q] = B_K ? ld128(base_b[ks * PARTS + q] + so + (uint32_t)(j * FR * 128))
                           : ldtr(base_b[B_K ? 0 : j] + so + (uint32_t)(ks * 32 * RCB * 16), 4 * RCB * 16);
  };
  // the scales' words of a group of four steps: this lane's rows of A, its columns of B
  int sa[FM], sb = 0, sa_next[FM], sb_next = 0;
  auto read_scales = [&](int group) __attribute__((always_inline)) {
    if constexpr (Q8) {
      const uint32_t slot = lds0 + 2 * C::STAGE + (uint32_t)(group & 1) * C::SCALES;
      auto ld32 = [](uint32_t addr) { return *reinterpret_cast<const __attribute__((address_space(3))) int*>((uintptr_t)addr); };
#pragma unroll
      for (int i = 0; i < FM; ++i) sa_next[i] = ld32(slot + (uint32_t)(wm * S::WM + i * 32 + l32) * 4);
      sb_next = ld32(slot + (uint32_t)(C::A_SLOTS + wn * S::WN / kQBlock) * 256 + (uint32_t)lane * 4);
    }
  };
  auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = sa_next[i];
    sb = sb_next;
  };
  using Acc = std::conditional_t<Q8, f32x16_t, f32x4_t>;
  Acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = Acc{};
  auto multiply = [&](int ks, auto byte) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (Q8) {
          struct Pair { u32x4_t lo, hi; };
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              __builtin_bit_cast(i32x8_t, (Pair{fb[ks][j][0], fb[ks][j][1]})),
              __builtin_bit_cast(i32x8_t, (Pair{fa[ks][i][0], fa[ks][i][1]})), acc[i][j], 0, 0, byte.value, sb,
              byte.value, sa[i]);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fb[ks][j][0]),
                                                              __builtin_bit_cast(bf16x8_t, fa[ks][i][0]), acc[i][j], 0, 0, 0);
        }
      }
  };
  // LDS reads spread over the multiplications
  auto mix = [&]() __attribute__((always_inline)) {
    constexpr int NMF = FM * FN;
    constexpr int NRD = FM * (A_K ? PARTS : 2) + FN * (B_K ? PARTS : 2);
    constexpr int EACH = (NRD + NMF - 1) / NMF;
    constexpr int TURNS_ = NRD / EACH < NMF ? NRD / EACH : NMF;
#pragma unroll
    for (int q = 0; q < TURNS_; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // one multiplication
      __builtin_amdgcn_sched_group_barrier(0x100, EACH, 0);  // LDS reads
    }
    if constexpr (NMF > TURNS_) __builtin_amdgcn_sched_group_barrier(0x008, NMF - TURNS_, 0);
    if constexpr (NRD > TURNS_ * EACH) __builtin_amdgcn_sched_group_barrier(0x100, NRD - TURNS_ * EACH, 0);
  };

  // ---- the sum.  Steps past the last are loads of the last one again, never used.
  const bool active = m0 + wm * S::WM < m_end;  // a wave without rows only helps with the loads
  if (nk > 0) {
    issue(0, 0);
    wait_vmcnt<0>();
    place8(0);
    step_barrier();
    issue(min(1, last), 1);
    if (active) {
      read_half(0, 0);
      read_scales(0);
      take_scales();
    }
    constexpr int UNROLL = Q8 ? 4 : 2;
    for (int kt0 = 0; kt0 < nk; kt0 += UNROLL) {
      auto step = [&](auto u) __attribute__((always_inline)) {
        const int kt = kt0 + u.value;
        constexpr int stage = u.value & 1;
        launder();
        if (active) {
          read_half(stage, 1);
          multiply(0, u);
          mix();
        }
        wait_vmcnt<0>();  // this wave's loads of step kt + 1
        place8(stage ^ 1);
        step_barrier();
        issue(min(kt + 2, last), stage);
        launder();
        if (active) {
          read_half(stage ^ 1, 0);
          if constexpr (Q8 && u.value == 3) read_scales((kt0 >> 2) + 1);
          multiply(1, u);
          mix();
          if constexpr (Q8 && u.value == 3) take_scales();
        }
      };
      step(std::integral_constant<int, 0>());
      if (kt0 + 1 >= nk) break;
      step(std::integral_constant<int, 1>());
      if constexpr (UNROLL == 4) {
        if (kt0 + 2 >= nk) break;
        step(std::integral_constant<int, 2>());
        if (kt0 + 3 >= nk) break;
        step(std::integral_constant<int, 3>());
      }
    }
    wait_vmcnt<0>();
    step_barrier();  // the stages are free
  }

  // ---- the tile's output.  Element q of a fragment: row of C along the lanes, four
  // neighbouring columns in a lane.
  constexpr int QUADS = FR == 32 ? 4 : 1;
  auto column = [&](int j, int quad) { return j * FR + (FR == 32 ? quad * 8 + lh * 4 : lg * 4); };
  auto row_of = [&](int i) { return i * FR + (FR == 32 ? l32 : l16); };
  if constexpr (ROWS) {
    float* c = (float*)p.C + ((int64_t)e * p.K + m0 + wm * S::WM) * p.N + n0 + wn * S::WN;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = row_of(i);
      if (m0 + wm * S::WM + r >= m_end) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = column(j, 0);
        if (n0 + wn * S::WN + n >= p.N) continue;
        f32x4_t* to = reinterpret_cast<f32x4_t*>(c + (int64_t)r * p.N + n);
        f32x4_t v = acc[i][j];
        if (p.accumulate) v += *to;
        *to = v;
      }
    }
  } else {
    // through this wave's part of LDS as bf16, then 16 bytes a lane, rows in a piece
    if (!active) return;
    constexpr int PITCH = S::WN + 8;
    bf16_t* own = reinterpret_cast<bf16_t*>(smem) + wave * S::WM * PITCH;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int quad = 0; quad < QUADS; ++quad) {
          uint2 v;
          v.x = (uint32_t)f2bf(acc[i][j][quad * 4]) | (uint32_t)f2bf(acc[i][j][quad * 4 + 1]) << 16;
          v.y = (uint32_t)f2bf(acc[i][j][quad * 4 + 2]) | (uint32_t)f2bf(acc[i][j][quad * 4 + 3]) << 16;
          *reinterpret_cast<uint2*>(own + row_of(i) * PITCH + column(j, quad)) = v;
        }
    wave_lds_sync();
    constexpr int CH = S::WN / 8;
    bf16_t* c = (bf16_t*)p.C + (int64_t)(m0 + wm * S::WM) * p.N + n0 + wn * S::WN;
#pragma unroll
    for (int u = 0; u < S::WM * CH / 64; ++u) {
      const int at = u * 64 + lane, r = at / CH, n = at % CH * 8;
      if (m0 + wm * S::WM + r < m_end && n0 + wn * S::WN + n < p.N)
        *reinterpret_cast<u32x4_t*>(c + (int64_t)r * p.N + n) = *reinterpret_cast<const u32x4_t*>(own + r * PITCH + n);
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

template <Form F, class S>
int launch(const Args& a, unsigned grid, int mtiles, int ntiles, hipStream_t st) {
  auto kern = gmm_kernel<F, S>;
  constexpr int lds = GCfg<F, S>::LDS;
  static uint64_t attr_set = 0;
  (void)hipGetLastError();
  if (set_lds_attr(kern, lds, attr_set) != hipSuccess) return MOE_EHIP;
  kern<<<grid, S::THREADS, lds, st>>>(a, mtiles, ntiles);
  return launched();
}

template <Form F, class S>
int rows_launch(const Args& a, hipStream_t st) {
  const int ntiles = (int)ceil_div(a.N, S::BN);
  return launch<F, S>(a, (unsigned)(row_tiles(a.R, a.E, S::BM) * ntiles), 0, ntiles, st);
}
template <Form F, class S>
int weights_launch(const Args& a, hipStream_t st) {
  const int mtiles = (int)ceil_div(a.K, S::BM), ntiles = (int)ceil_div(a.N, S::BN);
  return launch<F, S>(a, (unsigned)((int64_t)a.E * mtiles * ntiles), mtiles, ntiles, st);
}

template <Form F>
int rows_product(const Args& a, hipStream_t st) {
  return rows_launch<F, GShape<256, 256, 4, 2>>(a, st);
}

template <bool Q8>
int weights_product(const Args& a, hipStream_t st) {
  return weights_launch<Q8 ? Form::TN8 : Form::TN, GShape<256, 256, 4, 2>>(a, st);
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
