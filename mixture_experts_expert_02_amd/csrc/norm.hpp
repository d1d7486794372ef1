// Residual addition and root-mean-square norm of hidden rows, with outputs in
// the rows' type and / or as microscaled blocks (moe_add_rmsnorm).
//
//   h = round(x + residual)   (the stored stream; h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * w
//
// One workgroup per row, the row kept in registers between the sum and the
// scaling (one read of x and residual). Squares are added in fp32 by eights and
// in double from there, the root is taken in double; h * w is exact for 16-bit
// types, so y is off by the rounding of its last product and of r alone. The microscaled
// output is quantized from the fp32 y rounded to odd (below), so that its elements are
// the nearest ones to h * w * r, not to a y rounded before. A thread
// holds C chunks of 8 values, NT chunks apart; a block of 32 values is one
// quad of lanes, as in the quantizer. Bound by HBM where rows are many: 8192 x 7168 bf16 with
// residual and MXFP8 output 84 us, 413 MB at 4.9 TB/s; few rows by the chain load, sum, scale, store:
// 1 x 7168 3.9 us, where an empty kernel in a graph takes 2. The sums and the root in fp32 and y rounded
// to nearest took 3.5 and 82.5 us and put four times as many elements on the other side of a tie.
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
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) s += part[i];
  return s;
}

// 1 / sqrt(v): one Newton step on the hardware's estimate; 0 and infinity keep theirs.
__device__ __forceinline__ double rsqrt_f64(double v) {
  const double y = __builtin_amdgcn_rsq(v);
  const double z = fma(0.5 * fma(-v * y, y, 1.0), y, y);
  return v > 0.0 && v < (double)INFINITY ? z : y;
}

// v + e, |e| at most half a step of v, cut toward zero with the last bit set if
// anything was cut off: rounding that to fewer bits gives what rounding v + e would.
// An infinity or NaN stays (e is the other infinity or NaN then): its block becomes a NaN block.
__device__ __forceinline__ float to_odd(float v, float e) {
  const int b = __float_as_int(v);
  const bool cut = e != 0.f && (b & 0x7f800000) != 0x7f800000;
  return cut ? __int_as_float((b + ((b ^ __float_as_int(e)) >> 31)) | 1) : v;
}

template <int DT, int FMT, int NT, int C>
__global__ __launch_bounds__(NT) void k_add_rmsnorm(const NormParams p) {
  const size_t t = blockIdx.x;
  const int n8 = p.H / 8;
  float h[C][8];
  double sq = 0.0;
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
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) q += h[c][j] * h[c][j];
    sq += (double)q;
  }
  const double rd = rsqrt_f64(fma(block_sum<NT>(sq), p.inv_h, (double)p.eps));
  const float r = (float)rd, r_lo = (float)(rd - (double)r);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (int)threadIdx.x + c * NT;
    if (i >= n8) break;
    float w[8], y[8];
    load8_as(p.w_type, p.w, 8 * (size_t)i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[c][j] *= w[j];
      y[j] = h[c][j] * r;
    }
    if (p.y) store8<DT>(p.y, t * p.ldy + 8 * (size_t)i, y);
    if constexpr (FMT != 0) {  // H is a multiple of 32: quads are whole
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = to_odd(y[j], fmaf(h[c][j], r_lo, fmaf(h[c][j], r, -y[j])));
      const int code = mxf::scale_code<FMT>(mxf::quad_amax(y));
      uint32_t q[2];
      mxf::encode8<FMT>(y, code, q);
      mxf::store_codes<FMT>(p.codes + t * p.ld_codes, i, q);
      if ((threadIdx.x & 3) == 0) p.scales[t * p.ld_scales + i / 4] = (uint8_t)code;
    }
  }
}

}  // namespace moe
