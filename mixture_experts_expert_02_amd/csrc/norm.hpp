// Residual addition and root-mean-square norm of hidden rows, with outputs in
// the rows' type and / or as microscaled blocks (moe_add_rmsnorm).
//
//   h = round(x + residual)   (the stored stream; h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * w
//
// One workgroup per row, the row kept in registers between the sum and the
// scaling (one read of x and residual). Squares, their sum and the root are
// doubles, where the square of every float32 is in range (sums in fp32 lost rows above 2^64 and below
// 2^-75, and half the bits of r). The root is split into 2^k m, m in [1, 2): h 2^k is at most sqrt(H), so the
// products with w and m pass float32 only if y does (and an h 2^k below 2^-126 rounds as float32 does there).
// The microscaled output and a float32 y carry the roundings of both products and of m along (e below); the
// former is quantized from y rounded to odd, so that its elements are the nearest ones to h * w * r, not to a
// y rounded before.
// A 16-bit y takes the plain products. A thread
// holds C chunks of 8 values, NT chunks apart; a block of 32 values is one
// quad of lanes, as in the quantizer. Bound by HBM where rows are many: 8192 x 7168 bf16 with
// residual and MXFP8 output 83 us, 413 MB at 5.0 TB/s; few rows by the chain load, sum, scale, store:
// 1 x 7168 4.1 us, where an empty kernel in a graph takes 2. Squares and products in fp32, the carried bits without
// w's, took 82.5 and 3.9 us; every product in double 92 and 4.3.
#pragma once

#include "elem.hpp"
#include "mx_format.hpp"

namespace moe {

struct NormParams {
  const void* x;
  const void* res;    // or nullptr
  const void* w;
  void* res_out;      // written when res is given
  void* y;            // or nullptr
  uint8_t* codes;     // or nullptr (FMT 0)
  uint8_t* scales;
  int64_t ldx, ld_res, ld_res_out, ldy, ld_codes, ld_scales;
  int32_t H, w_type;
  float eps;
  double inv_h;       // 1 / H
};

template <int NT>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[NT / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if (NT == 64) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) s[i & 1] += part[i];
  return s[0] + s[1];
}

// 1 / sqrt(v): the hardware's estimate y, off by 2^-23 or less, times (1 - e)^(-1/2) with e = 1 - v y^2,
// by the series to e^2 (the next term is below 2^-66); 0 and infinity keep theirs.
__device__ __forceinline__ double rsqrt_f64(double v) {
  const double y = __builtin_amdgcn_rsq(v);
  const double e = fma(-v * y, y, 1.0);
  const double z = fma(y * e, fma(0.375, e, 0.5), y);
  return v > 0.0 && v < (double)INFINITY ? z : y;
}

// v + e, |e| at most half a step of v, cut toward zero with the last bit set if
// anything was cut off: rounding that to fewer bits gives what rounding v + e would.
// An infinity or NaN stays (e is an infinity or NaN then, by v's own subtraction): its block becomes a NaN block.
__device__ __forceinline__ float to_odd(float v, float e) {
  constexpr int kFiniteNotZero = 0x198;  // normal and subnormal numbers of either sign
  const int b = __float_as_int(v);
  return __builtin_amdgcn_classf(e, kFiniteNotZero) ? __int_as_float((b + ((b ^ __float_as_int(e)) >> 31)) | 1) : v;
}

template <int DT, int FMT, int NT, int C>
__global__ __launch_bounds__(NT) void k_add_rmsnorm(const NormParams p) {
  const size_t t = blockIdx.x;
  const int n8 = p.H / 8;
  float h[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (int)threadIdx.x + c * NT;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] = 0.f;
    if (i < n8) load8<DT>(p.x, t * p.ldx + 8 * (size_t)i, h[c]);
  }
  if (p.res) {
    float r[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (int)threadIdx.x + c * NT;
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] = 0.f;
      if (i < n8) load8<DT>(p.res, t * p.ld_res + 8 * (size_t)i, r[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (int)threadIdx.x + c * NT;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = round_to<DT>(h[c][j] + r[c][j]);
      if (i < n8) store8<DT>(p.res_out, t * p.ld_res_out + 8 * (size_t)i, h[c]);
    }
  }
  double sq[2] = {0.0, 0.0};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[j & 1] = fma((double)h[c][j], (double)h[c][j], sq[j & 1]);
  const double rd = rsqrt_f64(fma(block_sum<NT>(sq[0] + sq[1]), p.inv_h, (double)p.eps));
  const int k = __builtin_amdgcn_frexp_exp(rd) - 1;  // rd = 2^k m, m in [1, 2) (0, infinity and NaN: themselves)
  const double m = __builtin_amdgcn_ldexp(rd, -k);
  const float r = (float)m, r_lo = (float)(m - (double)r);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (int)threadIdx.x + c * NT;
    if (i >= n8) break;
    float w[8], y[8], odd[8];
    load8_as(p.w_type, p.w, 8 * (size_t)i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = __builtin_amdgcn_ldexpf(h[c][j], k);
      const float hw = u * w[j];
      y[j] = hw * r;
      if constexpr (FMT != 0 || DT == T_FP32) {
        const float e = fmaf(hw, r_lo, fmaf(u, w[j], -hw) * r);
        const float v = fmaf(hw, r, e);
        if (FMT != 0) odd[j] = to_odd(v, fmaf(hw, r, -v) + e);
        if (DT == T_FP32) y[j] = fabsf(y[j]) < INFINITY ? v : y[j];  // e is NaN beside an infinite hw
      }
    }
    if (p.y) store8<DT>(p.y, t * p.ldy + 8 * (size_t)i, y);
    if constexpr (FMT != 0) {  // H is a multiple of 32: quads are whole
      const int code = mxf::scale_code<FMT>(mxf::quad_amax(odd));
      uint32_t q[2];
      mxf::encode8<FMT>(odd, code, q);
      mxf::store_codes<FMT>(p.codes + t * p.ld_codes, i, q);
      if ((threadIdx.x & 3) == 0) p.scales[t * p.ld_scales + i / 4] = (uint8_t)code;
    }
  }
}

}  // namespace moe
