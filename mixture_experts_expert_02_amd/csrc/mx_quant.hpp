// Rows to microscaled blocks and back (moe_mx_quantize, moe_mx_dequantize).
//
// A thread takes 8 consecutive values (16 or 32 bytes), so a quad of lanes
// holds one block of 32: its largest magnitude is two DPP maxima away, no LDS,
// and a wave reads and writes whole contiguous lines. Each thread does kUnroll
// chunks, 256 chunks apart, with all loads issued first. Both kernels are bound by HBM:
// bf16 14336 x 16384 to MXFP4 98 us (6.1 TB/s read and written), to MXFP8 118 us (6.0), a copy
// of 1 GiB runs at 5.1. Chunks per thread 1 / 2 / 4 / 8: 99 / 98 / 104 / 110 us, 64 x 7168 2.3 / 2.4 / 2.6 / 3.5.
#pragma once

#include "elem.hpp"
#include "mx_format.hpp"

namespace moe {
namespace mxf {

constexpr int kUnroll = 2;

struct RowsParams {
  const void* x;      // quantize: values in; dequantize: unused
  void* out;          // dequantize: values out
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld;         // elements between rows of the values
  int64_t ld_codes;   // bytes
  int64_t ld_scales;  // bytes
  uint32_t per_row;   // chunks of 8 values per row (a multiple of 4)
  uint32_t n;         // chunks in all
};

// row and chunk within the row of flat chunk i; FLAT (all rows contiguous):
// one row
template <bool FLAT>
__device__ __forceinline__ void place(const RowsParams& p, uint32_t i, uint32_t& row, uint32_t& c) {
  row = FLAT ? 0u : i / p.per_row;
  c = FLAT ? i : i - row * p.per_row;
}

template <int DT, int FMT, bool FLAT>
__global__ __launch_bounds__(256) void k_quantize(const RowsParams p) {
  const uint32_t i0 = blockIdx.x * (256u * kUnroll) + threadIdx.x;
  float v[kUnroll][8];
  uint32_t row[kUnroll], c[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = i0 + 256u * u;
    place<FLAT>(p, min(i, p.n - 1), row[u], c[u]);
    load8<DT>(p.x, (size_t)row[u] * p.ld + 8 * (size_t)c[u], v[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (i0 + 256u * u >= p.n) break;  // n is a multiple of 4: whole quads
    const int code = scale_code<FMT>(quad_amax(v[u]));
    uint32_t w[2];
    encode8<FMT>(v[u], code, w);
    store_codes<FMT>(p.codes + (size_t)row[u] * p.ld_codes, c[u], w);
    if ((threadIdx.x & 3) == 0) p.scales[(size_t)row[u] * p.ld_scales + c[u] / 4] = (uint8_t)code;
  }
}

template <int DT, int FMT, bool FLAT>
__global__ __launch_bounds__(256) void k_dequantize(const RowsParams p) {
  const uint32_t i0 = blockIdx.x * (256u * kUnroll) + threadIdx.x;
  uint32_t w[kUnroll][2], code[kUnroll], row[kUnroll], c[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    place<FLAT>(p, min(i0 + 256u * u, p.n - 1), row[u], c[u]);
    load_codes<FMT>(p.codes + (size_t)row[u] * p.ld_codes, c[u], w[u]);
    code[u] = p.scales[(size_t)row[u] * p.ld_scales + c[u] / 4];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (i0 + 256u * u >= p.n) break;
    float v[8];
    decode8<FMT>(w[u], scale_value(code[u]), v);
    store8<DT>(p.out, (size_t)row[u] * p.ld + 8 * (size_t)c[u], v);
  }
}

}  // namespace mxf
}  // namespace moe
