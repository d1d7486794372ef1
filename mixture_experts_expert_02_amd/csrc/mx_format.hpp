// Microscaled blocks (OCP Microscaling v1.0 reading): 32 consecutive values
// share one e8m0 scale 2^(code - 127); the elements are e2m1 (MXFP4) or e4m3
// (MXFP8). For a block whose largest magnitude lies in [2^e, 2^(e+1)) the
// scale is 2^(e - emax), emax the element type's largest exponent (2 or 8),
// its code clamped to [0, 254]; elements are value / scale rounded to nearest
// (ties to even) and saturated at the largest element (6 or 448). This is the
// rule by which the experts step quantizes its MXFP8 rows. A block that holds an
// infinity or NaN has no such form: it gets the format's NaN scale (255) and
// zero codes, so every value read from it is NaN.
#pragma once

#include "common.hpp"

namespace moe {
namespace mxf {

enum Fmt { MXFP4 = 1, MXFP8 = 2 };  // moe_mxfmt (0: none)

constexpr int kNanCode = 255;

__host__ __device__ constexpr int emax(int fmt) { return fmt == MXFP4 ? 2 : 8; }
// bytes of n values' codes
__host__ __device__ constexpr int64_t code_bytes(int fmt, int64_t n) { return fmt == MXFP4 ? n / 2 : n; }

// Scale code of a block from the bits of its largest magnitude.
template <int FMT>
__device__ __forceinline__ int scale_code(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kNanCode;
  return max((int)(amax_bits >> 23) - emax(FMT), 0);
}

// 1 / scale, 2^(127 - code); 0 for the NaN code. Codes of finite blocks are
// at most 252, so the result is a normal number.
__device__ __forceinline__ float inv_scale(int code) {
  return code == kNanCode ? 0.f : __uint_as_float((uint32_t)(254 - code) << 23);
}

// scale, 2^(code - 127) (code 0: the subnormal 2^-127); NaN for the NaN code
__device__ __forceinline__ float scale_value(uint32_t code) {
  if (code == (uint32_t)kNanCode) return __uint_as_float(0x7fc00000u);
  return code == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23);
}

// Largest magnitude (as bits) of the block that this lane's quad (4 lanes,
// 8 values each) holds. Integer maxima, so a NaN wins over everything.
__device__ __forceinline__ uint32_t quad_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));  // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // lane ^ 2
  return m;
}

// Codes of 8 values times inv: MXFP4 one 32-bit word (value 2i in the low half
// of byte i), MXFP8 two. A value of a NaN block becomes 0 (code 0).
template <int FMT>
__device__ __forceinline__ void encode8(const float (&v)[8], int code, uint32_t (&w)[2]) {
  constexpr float top = FMT == MXFP4 ? 6.f : 448.f;
  const float inv = inv_scale(code);
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = fminf(fmaxf(v[j] * inv, -top), top);
    if (code == kNanCode) s[j] = 0.f;
  }
  if constexpr (FMT == MXFP4) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, s[0], s[1], 1.f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, s[2], s[3], 1.f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, s[4], s[5], 1.f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, s[6], s[7], 1.f, 3);
    w[0] = r;
    w[1] = 0;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int r = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * h], s[4 * h + 1], 0, false);
      r = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * h + 2], s[4 * h + 3], r, true);
      w[h] = (uint32_t)r;
    }
  }
}

// The 8 values that codes w stand for, scale included.
template <int FMT>
__device__ __forceinline__ void decode8(const uint32_t (&w)[2], float scale, float (&v)[8]) {
  if constexpr (FMT == MXFP4) {
#define MOE_FP4_PAIR(i)                                                                    \
  {                                                                                        \
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.f, i);                \
    v[2 * (i)] = p[0] * scale;                                                             \
    v[2 * (i) + 1] = p[1] * scale;                                                         \
  }
    MOE_FP4_PAIR(0)
    MOE_FP4_PAIR(1)
    MOE_FP4_PAIR(2)
    MOE_FP4_PAIR(3)
#undef MOE_FP4_PAIR
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
      const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
      v[4 * h] = a[0] * scale;
      v[4 * h + 1] = a[1] * scale;
      v[4 * h + 2] = b[0] * scale;
      v[4 * h + 3] = b[1] * scale;
    }
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 8 values of chunk c (values 8c..8c+7) of a row's codes
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c, const uint32_t (&w)[2]) {
  if constexpr (FMT == MXFP4) *(uint32_t*)(row + 4 * c) = w[0];
  else *(u32x2*)(row + 8 * c) = u32x2{w[0], w[1]};
}
template <int FMT>
__device__ __forceinline__ void load_codes(const uint8_t* row, int64_t c, uint32_t (&w)[2]) {
  if constexpr (FMT == MXFP4) {
    w[0] = *(const uint32_t*)(row + 4 * c);
    w[1] = 0;
  } else {
    const u32x2 t = *(const u32x2*)(row + 8 * c);
    w[0] = t[0];
    w[1] = t[1];
  }
}

}  // namespace mxf
}  // namespace moe
