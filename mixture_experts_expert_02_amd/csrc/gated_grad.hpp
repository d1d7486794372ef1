// Row-wise steps of the gated block's backward pass: gradients of its
// pre-activations and sums of columns.
#pragma once

#include "dense16.hpp"

namespace moe {
namespace d16 {

// dg = dout f_g(g, u), du = dout f_u(g, u), rounded to the type: the matrix
// instruction takes 16-bit operands, and each rounding is off by half a step of its own value, so a sum of
// many carries an error of the size of its own last rounding (together 1.41 times as much; of 1500 sizes beyond kPartValues 1.52 in
// one output of a hundred, 1.86 at most, where heavy rows or columns rule the sums). A few values always are ruled by the largest (one row of
// 88 columns: 1.8 times, of 256: 1.7), so up to kPartValues, in however many rows, their lower parts go along, and the gradients are as exact as from unrounded
// values. Others get them on request (64 x 7168 x 2048 44 -> 54 us, 77 x 2880 x 2880 40 -> 58, 1023 x 7168 x 2048 145 -> 242,
// 4096 x 4096 x 14336 1554 -> 3006; root mean square errors of bf16 results 0.00234 and 0.00166). With sums != nullptr the columns'
// sums over this workgroup's rows as well, from the unrounded values: to their place where one workgroup
// has all rows, else for k_column_sums.
// Memory-bound: three reads and two writes of 16 bits a value. 64 columns to a workgroup, whole lines of 32 rows at a time.
struct GradParams {
  const void *dout, *gate, *up;
  void *dg, *du;      // [M or, in two parts, 2 M, I] contiguous
  float* sums;        // [row blocks][2][I] or nullptr
  float* dbias[2];    // [I]
  int64_t ld_dout, ld_gate, ld_up;
  int32_t M, I;
  int32_t rows;       // of a workgroup, a multiple of 32
  int32_t accumulate;
  int32_t parts;      // lower parts too, M rows further on
  ActParams act;
};

// Stores v rounded to the type and leaves in v what that left of it; 0 of what it made an infinity, so that the products
// stay infinite. The rest is taken from the bits that are stored, which the asm makes the compiler use: it would round
// again, by an instruction that multiplies and rounds to 16 bits at once, and near a tie that is another value.
template <int DT>
__device__ __forceinline__ void store_upper(uint16_t* to, float (&v)[8]) {
  u32x4 bits;
  store8<DT>(&bits, 0, v);
  asm("" : "+v"(bits));
  *(u32x4*)to = bits;
  float up[8];
  load8<DT>(&bits, 0, up);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fabsf(up[j]) < INFINITY ? v[j] - up[j] : 0.f;
}

template <int DT>
__global__ __launch_bounds__(256) void k_gated_grad(const GradParams p) {
  __shared__ float part[2][32][64 + 1];
  const int c8 = (threadIdx.x & 7) * 8, r0 = threadIdx.x >> 3;
  const int col = blockIdx.y * 64 + c8;
  float sg[8], su[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.f;
  if (col < p.I) {
    with_act(p.act, [&](auto k) {
#pragma unroll 2
      for (int r = r0; r < p.rows; r += 32) {
        const int64_t row = (int64_t)blockIdx.x * p.rows + r;
        if (row >= p.M) break;
        float d[8], g[8], u[8];
        load8<DT>(p.dout, (size_t)(row * p.ld_dout + col), d);
        load8<DT>(p.gate, (size_t)(row * p.ld_gate + col), g);
        load8<DT>(p.up, (size_t)(row * p.ld_up + col), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float fg, fu;
          act_df<decltype(k)::value>(p.act, g[j], u[j], fg, fu);
          g[j] = d[j] * fg;
          u[j] = d[j] * fu;
          sg[j] += g[j];
          su[j] += u[j];
        }
        store_upper<DT>((uint16_t*)p.dg + row * p.I + col, g);
        store_upper<DT>((uint16_t*)p.du + row * p.I + col, u);
        if (p.parts) {
          store8<DT>(p.dg, (size_t)((row + p.M) * p.I + col), g);
          store8<DT>(p.du, (size_t)((row + p.M) * p.I + col), u);
        }
      }
    });
  }
  if (!p.sums) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    part[0][r0][c8 + j] = sg[j];
    part[1][r0][c8 + j] = su[j];
  }
  __syncthreads();
  const int which = threadIdx.x >> 6, c = threadIdx.x & 63, at = blockIdx.y * 64 + c;
  if (which > 1 || at >= p.I) return;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) s += part[which][q][c];
  if (gridDim.x == 1) p.dbias[which][at] = p.accumulate ? p.dbias[which][at] + s : s;
  else p.sums[((size_t)blockIdx.x * 2 + which) * p.I + at] = s;
}

// dst[which][c] (+)= sum over blocks of sums[block][which][c], in the blocks' order
__global__ __launch_bounds__(256) void k_column_sums(const float* sums, int blocks, int I, float* dg, float* du, int accumulate) {
  const int c = blockIdx.x * 256 + threadIdx.x, which = blockIdx.y;
  if (c >= I) return;
  double s = 0;
  for (int b = 0; b < blocks; ++b) s += sums[((size_t)b * 2 + which) * I + c];
  float* dst = (which ? du : dg) + c;
  *dst = (float)(accumulate ? s + *dst : s);
}

// Gradients of weights where there are no rows: zeros, eight columns to a thread.
template <int DT>
__global__ __launch_bounds__(256) void k_zero_rows(void* a, void* b, int64_t ld_a, int64_t ld_b, int rows, int cols) {
  const int cpr = cols / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)rows * cpr) return;
  const int64_t row = i / cpr, col = (i - row * cpr) * 8;
  const float zero[8] = {};
  if (blockIdx.y) store8<DT>(b, (size_t)(row * ld_b + col), zero);
  else store8<DT>(a, (size_t)(row * ld_a + col), zero);
}

}  // namespace d16
}  // namespace moe
