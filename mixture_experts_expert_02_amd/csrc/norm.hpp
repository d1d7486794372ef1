// Residual addition and root-mean-square norm of hidden rows, with outputs in
// the rows' type and / or as microscaled blocks (moe_add_rmsnorm).
//
//   h = round(x + residual)   (the stored stream; h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * w
//
// One workgroup per row, the row kept in registers between the sum and the
// scaling (one read of x and residual), sums in fp32. The microscaled output
// is quantized from the fp32 y, so its elements are rounded once. A thread
// holds C chunks of 8 values, NT chunks apart; a block of 32 values is one
// quad of lanes, as in the quantizer. Bound by HBM where rows are many: 8192 x 7168 bf16 with
// residual and MXFP8 output 80 us, 413 MB at 5.2 TB/s; few rows by the chain load, sum, scale, store:
// 1 x 7168 3.4 us, where an empty kernel in a graph takes 2.
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
};

template <int NT>
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[NT / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if (NT == 64) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) s += part[i];
  return s;
}

template <int DT, int FMT, int NT, int C>
__global__ __launch_bounds__(NT) void k_add_rmsnorm(const NormParams p) {
  const size_t t = blockIdx.x;
  const int n8 = p.H / 8;
  float h[C][8];
  float sq = 0.f;
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
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq += h[c][j] * h[c][j];
  const float r = 1.f / sqrtf(block_sum<NT>(sq) / (float)p.H + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (int)threadIdx.x + c * NT;
    if (i >= n8) break;
    float w[8], y[8];
    load8_as(p.w_type, p.w, 8 * (size_t)i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[c][j] * r * w[j];
    if (p.y) store8<DT>(p.y, t * p.ldy + 8 * (size_t)i, y);
    if constexpr (FMT != 0) {  // H is a multiple of 32: quads are whole
      const int code = mxf::scale_code<FMT>(mxf::quad_amax(y));
      uint32_t q[2];
      mxf::encode8<FMT>(y, code, q);
      mxf::store_codes<FMT>(p.codes + t * p.ld_codes, i, q);
      if ((threadIdx.x & 3) == 0) p.scales[t * p.ld_scales + i / 4] = (uint8_t)code;
    }
  }
}

}  // namespace moe
