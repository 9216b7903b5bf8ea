// Rows in 8 bits on the device (include/q8.h): the scale of a block, rounding to
// e4m3 and back.
#pragma once

#include "device_common.hpp"
#include "wave_ops.hpp"

namespace moe {

constexpr int kQBlock = 128;  // columns that share a scale
constexpr uint32_t kQOne = 127;  // the scale byte of 2^0, which the padding holds
// bytes of a row of H numbers, and of its scales
constexpr int q8_row_pitch(int H) { return (H + kQBlock - 1) / kQBlock * kQBlock; }
constexpr int q8_blocks(int H) { return (H + kQBlock - 1) / kQBlock; }
constexpr int q8_scale_pitch(int H) { return (q8_blocks(H) + 3) / 4 * 4; }

// The byte of the smallest power of two 2^e, e >= -110, with amax / 2^e <= 448 =
// 1.75 * 2^8: with amax = 1.f * 2^x, e = x - 8, and one more where 1.f > 1.75.
__device__ __forceinline__ uint32_t q8_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int byte = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(byte, 17);
}
// 1 / scale, of a byte that q8_scale_byte gave (17 to 247: a normal number)
__device__ __forceinline__ float q8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// the scale of any byte: 2^-127 is subnormal in fp32, 255 is NaN
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// The largest finite magnitude among n values of each of a run of lanes, by reduce().
// A maximum passes NaN over; where it finds an infinity the values are gone through
// again without it.
template <int n, typename R>
__device__ __forceinline__ float q8_amax(const float* v, R reduce) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < n; ++e) m = fmaxf(m, fabsf(v[e]));
  m = reduce(m);
  if (__builtin_isinf(m)) {  // the same in all lanes of the run
    m = 0.f;
#pragma unroll
    for (int e = 0; e < n; ++e) m = fmaxf(m, __builtin_isinf(v[e]) ? 0.f : fabsf(v[e]));
    m = reduce(m);
  }
  return m;
}

// Whether v is within `off` of its last places of where e4m3 or a scale turn, under any
// power of two: a value with at most four bits after its first.  There 32 bits do not say
// which side a computed value is on, and it is formed again in 64.
__device__ __forceinline__ bool q8_border(float v, uint32_t off = 8) {
  return ((__float_as_uint(v) + off) & 0x7ffffu) <= 2 * off && v != 0.f;
}
// x in 32 bits to odd (a value between two numbers becomes the one whose last bit is 1),
// so that rounding it once more gives what rounding x would.
__device__ __forceinline__ float q8_to_odd(double x) {
  const float f = (float)x;
  const uint32_t b = __float_as_uint(f);
  if (!(fabsf(f) < __builtin_inff()) || (double)f == x || (b & 1)) return f;
  return __uint_as_float(fabs(x) > fabs((double)f) ? b + 1 : b - 1);
}

// Four values as e4m3 (v_cvt_pk_fp8_f32: to nearest, ties to even; infinities and NaN
// to NaN).  The scale leaves no finite quotient above 448.
__device__ __forceinline__ uint32_t q8_round4(const float* v, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
  return (uint32_t)w;
}
// Four numbers of a word times the scale
__device__ __forceinline__ void q8_values4(uint32_t w, float scale, float* v) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0] * scale;
  v[1] = lo[1] * scale;
  v[2] = hi[0] * scale;
  v[3] = hi[1] * scale;
}

}  // namespace moe
