// Grouped weight gradients dW[e] = X_e^T dY_e over an expert's rows, with X in bf16
// or e4m3.
//
// A work-group computes a BM x BN tile of one expert's matrix, over the expert's
// rows in steps of 32.  Both operands stay as they are in memory (columns along the
// rows), go straight into LDS and are read with the transposing LDS loads; a step is
// 64 bytes of every column, NS of them take turns, and while step t is multiplied
// out of registers, step t + 1's fragments are read and steps t + 2 to t + NS fly.
// (Two stages of 64 rows: 388 us where these take 358 for 64 experts of 512 rows,
// 2048 x 1408, whose 738 MB of dW alone take 110 us to fill.)
//
// What bounds it: with few rows an expert, HBM.  Those 64 experts with operands out of
// HBM take 281 us for 964 MB, 1.17 GB with what XCDs read twice, near what a copy of as
// much takes; 16,384 rows and one matrix of 4096 x 4096 421 us, 1.31 PFLOP/s.
//
// X in 8 bits lands in LDS as it is, each lane's 16 numbers of one row with the word
// of their scale; one step before they are read, the lane makes them bf16, which
// holds them, and writes them to the stage.  That stands between a step's wait and its
// barrier, with no multiplication beside it: the same experts take 290 us so for 1.04 GB.
#pragma once

#include "gmm_common.hpp"

namespace moe {
namespace gmm {

// LDS of a work-group: NS stages of A and B.  For X in 8 bits: two stages of A as
// bf16, NS of B, NS of A as it is with its scales' words.
template <Form F, class S>
struct WeightsCfg {
  static constexpr int KT = 32;  // rows of k of a step
  static constexpr bool RAW = F == Form::TN8;
  static constexpr int A_BYTES = S::BM * 2 * KT, B_BYTES = S::BN * 2 * KT, STAGE = A_BYTES + B_BYTES;
  static constexpr int RAW_PW = RAW ? S::BM * KT / 1024 / S::WAVES : 0;  // loads of 1 KiB a wave
  static constexpr int RAW_WAVE = 1280, RAW_BYTES = RAW_WAVE * S::WAVES;
  static constexpr int PITCH = S::WN + 4;  // of a finished row, in fp32
  static constexpr int IN = RAW ? 2 * A_BYTES + S::NS * (B_BYTES + RAW_BYTES) : S::NS * STAGE;
  static constexpr int LDS = std::max(IN, S::WAVES * 16 * PITCH * 4);
  // loads a wave has of a step at least
  static constexpr int PER_STEP = (RAW ? 2 * RAW_PW : A_BYTES / 1024 / S::WAVES) + B_BYTES / 1024 / S::WAVES;
  static_assert(LDS <= kLdsBytes, "LDS");
  static_assert(!RAW || (RAW_PW == 1 && S::WAVES * 1024 == S::BM * KT), "A's step is one load of every wave");
  static_assert(S::NS == 4, "stages by the unrolled step; A's two stages go by its parity");
  static __device__ __forceinline__ uint32_t a_at(int s) { return (uint32_t)(RAW ? (s & 1) * A_BYTES : s * STAGE); }
  static __device__ __forceinline__ uint32_t b_at(int s) {
    return (uint32_t)(RAW ? 2 * A_BYTES + s * B_BYTES : s * STAGE + A_BYTES);
  }
  static __device__ __forceinline__ uint32_t raw_at(int s, int wave) {
    return (uint32_t)(2 * A_BYTES + S::NS * B_BYTES + s * RAW_BYTES + wave * RAW_WAVE);
  }
};

// An expert's tiles run in blocks of 4 x 4, whose work-groups share row panels in an
// XCD's L2; the tiles go to the XCDs in turn, sixteen at a time, so that every XCD has
// its part of each expert's rows, however they are spread.  With an expert's tiles on
// one XCD instead (each pass on other operands): 32,768 rows, 2048 x 1408, over 64
// experts whose shares fall by r^-0.2 302 us where these take 281, by r^-1 487 and
// 309; 65,536 rows, 4096 x 1536, 32 experts, r^-0.5 1020 and 766.  (Eight at a time in
// blocks of 4 x 2 283, 301, 771, but one matrix of 4096 x 4096 from 16,384 rows 455 us
// where these take 421.)
// Experts of more than twice the mean rows come first: their tiles take longest.
// (128 experts, 1024 x 1024, r^-1, the same operands every pass: 214 us in the
// experts' order, 139.)
constexpr int kBlockM = 4, kBlockN = 4, kDeal = 16;
inline int64_t weights_groups(int64_t tiles) { return ceil_div(tiles, 8 * kDeal) * 8 * kDeal; }
struct WeightsTile {
  int e, mt, nt;
  Segment rows;
};
template <int C>  // sets of 64 experts, one a lane
__device__ __forceinline__ bool find_weights_tile_in(const int32_t* offsets, int E, int R, int place, WeightsTile& t) {
  const int lane = threadIdx.x & 63;
  Segment s[C];
  unsigned long long large[C];
  int first = 0;  // large experts
#pragma unroll
  for (int c = 0; c < C; ++c) s[c] = segment(offsets, min(c * 64 + lane, E - 1), R);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    large[c] = __ballot(c * 64 + lane < E && (int64_t)(s[c].hi - s[c].lo) * E > 2 * (int64_t)R);
    first += __popcll(large[c]);
  }
  int at = place < first ? place : place - first;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const unsigned long long there = __ballot(c * 64 + lane < E), of = place < first ? large[c] : there & ~large[c];
    const int here = __popcll(of);
    if (at < here) {
      const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(of >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)of, 0));
      const int l = __ffsll((long long)__ballot((of >> lane & 1) && before == at)) - 1;
      t.e = c * 64 + l;
      t.rows = Segment{__builtin_amdgcn_readlane(s[c].lo, l), __builtin_amdgcn_readlane(s[c].hi, l)};
      return true;
    }
    at -= here;
  }
  return false;
}
__device__ __forceinline__ bool find_weights_tile(const int32_t* offsets, int E, int R, int mtiles, int ntiles, int bid,
                                                  WeightsTile& t) {
  const int slot = bid >> 3, lid = (slot / kDeal * 8 + (bid & 7)) * kDeal + slot % kDeal;
  const int per = mtiles * ntiles, place = lid / per;
  if (place >= E) return false;
  const int local = lid - place * per, pair = local / (kBlockN * mtiles), wide = min(kBlockN, ntiles - pair * kBlockN);
  const int r = local - pair * kBlockN * mtiles, block = r / (kBlockM * wide), in_block = r - block * kBlockM * wide;
  const int high = min(kBlockM, mtiles - block * kBlockM);
  t.nt = pair * kBlockN + in_block / high;
  t.mt = block * kBlockM + in_block % high;
  if (E <= 64) return find_weights_tile_in<1>(offsets, E, R, place, t);
  if (E <= 256) return find_weights_tile_in<4>(offsets, E, R, place, t);
  return find_weights_tile_in<16>(offsets, E, R, place, t);
}

// Split over the rows (PART): work-group (x, y) sums part y of its expert's steps
// of gridDim.y, into p.part [y][E][K][N].
template <Form F, class S, bool PART>
__global__ __launch_bounds__(S::THREADS) void gmm_weights_kernel(const Args p, int mtiles, int ntiles) {
  using C = WeightsCfg<F, S>;
  constexpr int FM = S::WM / 16, FN = S::WN / 16, NS = S::NS, KT = C::KT;
  constexpr int RCA = S::BM / 8, RCB = S::BN / 8;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = S::row(wave), wn = S::col(wave);

  WeightsTile t;
  if (!find_weights_tile(p.offsets, p.E, p.R, mtiles, ntiles, blockIdx.x, t)) return;
  const int e = __builtin_amdgcn_readfirstlane(t.e);
  const int m0 = __builtin_amdgcn_readfirstlane(t.mt) * S::BM, n0 = __builtin_amdgcn_readfirstlane(t.nt) * S::BN;
  int64_t k0 = __builtin_amdgcn_readfirstlane(t.rows.lo);
  int k_len = __builtin_amdgcn_readfirstlane(t.rows.hi - t.rows.lo);
  if constexpr (PART) {
    const int each = ((k_len + KT - 1) / KT + gridDim.y - 1) / gridDim.y * KT;
    const int from = min(k_len, each * (int)blockIdx.y);
    k_len = min(k_len - from, each);
    k0 += from;
  }
  const int nk = (k_len + KT - 1) / KT, last = nk - 1, left = k_len - last * KT;

  // ---- loads
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_void_p)smem));
  Loader<C::A_BYTES, S::WAVES> la;
  Loader<C::B_BYTES, S::WAVES> lb;
  const int64_t lda = C::RAW ? q8_row_pitch(p.K) : 2 * (int64_t)p.K, ldb = 2 * (int64_t)p.N;
  const int kp = C::RAW ? (int)lda : 0, sp = C::RAW ? q8_scale_pitch(p.K) : 0;
  const unsigned char* ap = (const unsigned char*)p.A + k0 * lda + (int64_t)m0 * (C::RAW ? 1 : 2);
  const unsigned char* bp = (const unsigned char*)p.B + k0 * ldb + (int64_t)n0 * 2;
  if constexpr (!C::RAW) la.template across_k<S::BM>(wave, lane, p.K - m0, (uint32_t)lda, left);
  lb.template across_k<S::BN>(wave, lane, p.N - n0, (uint32_t)ldb, left);
  // A in 8 bits: in each of a wave's loads a lane has 16 numbers of one row and, in a
  // load of its own, the word of four scales that theirs is in
  constexpr int LR = S::BM / 16;  // lanes of a row
  const int raw_col = lane % LR * 16, raw_block = (m0 + raw_col) / kQBlock;
  uint32_t raw_off = 0, raw_soff = 0, raw_to = 0;
  if constexpr (C::RAW) {
    const int r = wave * (64 / LR) + lane / LR;
    const bool there = m0 + raw_col < kp;
    raw_off = there ? (uint32_t)(r * kp + raw_col) : kOob;
    raw_soff = there ? (uint32_t)(r * sp + (raw_block & ~3)) : kOob;
    raw_to = lds0 + (uint32_t)(r * (RCA * 16) + (((lane % LR * 2) ^ trswz<RCA>(r)) << 4));
  }
  auto issue_raw = [&](int kt, int stage) __attribute__((always_inline)) {
    if constexpr (C::RAW) {
      const i32x4_t rq = open_srd(ap + (int64_t)kt * KT * kp, kt <= last);
      const i32x4_t rs = open_srd((const unsigned char*)p.As + (k0 + (int64_t)kt * KT) * sp, kt <= last);
      const bool in = kt * KT + wave * (64 / LR) + lane / LR < k_len;
      const uint32_t at = lds0 + C::raw_at(stage, wave);
      lds_load16_at(rq, at, in ? raw_off : kOob);
      lds_load4_at(rs, at + 1024, in ? raw_soff : kOob);
    }
  };
  // Each lane takes back what it loaded itself, so this wave's own wait is enough.
  auto place_raw = [&](int kt, int stage) __attribute__((always_inline)) {
    if constexpr (C::RAW) {
      const uint32_t from = lds0 + C::raw_at(stage, wave);
      const u32x4_t q = ld128(from + (uint32_t)lane * 16);
      const uint32_t byte = (uint32_t)ld32(from + 1024 + (uint32_t)lane * 4) >> (raw_block & 3) * 8 & 255u;
      const float scale = byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h + j], scale, false));
          w[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h + j], scale, true));
        }
        // (an even chunk's neighbour is its address with bit 4 turned)
        *reinterpret_cast<__attribute__((address_space(3))) u32x4_t*>((uintptr_t)((raw_to ^ (uint32_t)h * 16) + C::a_at(kt))) = w;
      }
    }
  };
  auto issue = [&](int kt, int stage) __attribute__((always_inline)) {
    if constexpr (C::RAW) {
      issue_raw(kt, stage);
    } else {
      const i32x4_t ra = open_srd(ap + (int64_t)kt * KT * lda, kt <= last);
#pragma unroll
      for (int u = 0; u < decltype(la)::PW; ++u) la.issue(u, ra, lds0 + C::a_at(stage), wave, kt == last);
    }
    const i32x4_t rb = open_srd(bp + (int64_t)kt * KT * ldb, kt <= last);
#pragma unroll
    for (int u = 0; u < decltype(lb)::PW; ++u) lb.issue(u, rb, lds0 + C::b_at(stage), wave, kt == last);
  };

  // ---- fragments
  const int l16 = lane & 15, lg = lane >> 4;
  // X in 8 bits needs the registers: there fragment b's address is fragment 0's with
  // the column's bits turned (its chunk is 2 b of the wave's, under the swizzle's
  // exclusive or)
  constexpr int NA = C::RAW ? 1 : FM, NB = C::RAW ? 1 : FN;
  static_assert((FM & (FM - 1)) == 0 && (FN & (FN - 1)) == 0, "a wave's columns are an aligned power of two");
  uint32_t base_a[NA], base_b[NB];
#pragma unroll
  for (int b = 0; b < NA; ++b) base_a[b] = lds0 + tr_base(lane, RCA, wm * S::WM + b * 16);
#pragma unroll
  for (int b = 0; b < NB; ++b) base_b[b] = lds0 + tr_base(lane, RCB, wn * S::WN + b * 16);
  auto launder = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NA; ++b) asm volatile("" : "+v"(base_a[b]));
#pragma unroll
    for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(base_b[b]));
  };
  u32x4_t fa[2][FM], fb[2][FN];
  auto read = [&](int stage, int set) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[set][i] = ldtr((C::RAW ? base_a[0] ^ (uint32_t)i * 32 : base_a[C::RAW ? 0 : i]) + C::a_at(stage), 4 * RCA * 16);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[set][j] = ldtr((C::RAW ? base_b[0] ^ (uint32_t)j * 32 : base_b[C::RAW ? 0 : j]) + C::b_at(stage), 4 * RCB * 16);
  };
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int set) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fb[set][j]),
                                                            __builtin_bit_cast(bf16x8_t, fa[set][i]), acc[i][j], 0, 0, 0);
  };

  // ---- the sum, as in gmm_rows.hpp: step t in stage t % NS, steps past the last load
  // nothing
  const bool active = m0 + wm * S::WM < p.K && n0 + wn * S::WN < p.N;
  if (nk > 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s, s);
    wait_vmcnt<(NS - 1) * C::PER_STEP>();
    place_raw(0, 0);
    step_barrier();
    if (active) read(0, 0);
    auto step = [&](int kt, auto u) __attribute__((always_inline)) {
      wait_vmcnt<(NS - 2) * C::PER_STEP>();  // this wave's loads of step kt + 1
      place_raw(u.value + 1, (u.value + 1) % NS);
      step_barrier();
      launder();
      issue(kt + NS, u.value);
      if (active) {
        read((u.value + 1) % NS, (u.value + 1) & 1);
        multiply(u.value & 1);
        constexpr int NMF = FM * FN, NRD = 2 * (FM + FN), TURNS = NRD < NMF ? NRD : NMF;
#pragma unroll
        for (int q = 0; q < TURNS; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one multiplication
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
        }
        if constexpr (NMF > TURNS) __builtin_amdgcn_sched_group_barrier(0x008, NMF - TURNS, 0);
        if constexpr (NRD > TURNS) __builtin_amdgcn_sched_group_barrier(0x100, NRD - TURNS, 0);
      }
    };
    for (int kt = 0; kt < nk; kt += NS) {
      step(kt, std::integral_constant<int, 0>());
      if (kt + 1 >= nk) break;
      step(kt + 1, std::integral_constant<int, 1>());
      if (kt + 2 >= nk) break;
      step(kt + 2, std::integral_constant<int, 2>());
      if (kt + 3 >= nk) break;
      step(kt + 3, std::integral_constant<int, 3>());
    }
    wait_vmcnt<0>();
    step_barrier();  // the stages are free
  }
  if (!active) return;

  // ---- the tile: a lane has four neighbours of a row in each fragment; 16 rows at a
  // time go through this wave's part of LDS, so that memory sees rows in a piece.
  // dW is read and written once: its accesses leave the operands in L2.
  const int64_t at = ((int64_t)e * p.K + m0 + wm * S::WM) * p.N + n0 + wn * S::WN;
  float* c = PART ? p.part + (int64_t)blockIdx.y * p.E * p.K * p.N + at : (float*)p.C + at;
  float* own = reinterpret_cast<float*>(smem) + wave * 16 * C::PITCH;
  constexpr int VR = S::WN / 4;  // vectors of a row
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i > 0) wave_lds_sync();  // the last rows' reads are done
#pragma unroll
    for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4_t*>(own + l16 * C::PITCH + j * 16 + lg * 4) = acc[i][j];
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < 16 * VR / 64; ++u) {
      const int r = (u * 64 + lane) / VR, n = (u * 64 + lane) % VR * 4;
      if (m0 + wm * S::WM + i * 16 + r >= p.K || n0 + wn * S::WN + n >= p.N) continue;
      f32x4_t* to = reinterpret_cast<f32x4_t*>(c + (int64_t)(i * 16 + r) * p.N + n);
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(own + r * C::PITCH + n);
      if (!PART && p.accumulate) v += __builtin_nontemporal_load(to);
      __builtin_nontemporal_store(v, to);
    }
  }
}

// dW = the sum of the splits' partial sums, in order, onto dW's own with accumulate.
__global__ __launch_bounds__(kThreads) void gmm_join_weights_kernel(const float* __restrict__ part, float* __restrict__ C,
                                                                    int64_t vecs, int splits, int accumulate) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * kThreads) {
    f32x4_t s{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int y = 0; y < splits; ++y) s += reinterpret_cast<const f32x4_t*>(part)[(int64_t)y * vecs + i];
    f32x4_t* to = reinterpret_cast<f32x4_t*>(C) + i;
    if (accumulate) s += *to;
    *to = s;
  }
}

}  // namespace gmm
}  // namespace moe
