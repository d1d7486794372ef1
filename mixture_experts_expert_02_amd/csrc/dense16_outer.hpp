// Gradients of weights from few rows (K <= kOuterRows): dWg = dg^T x, dWu = du^T x are little more than their output written once.
//
// 128 x 128 of the output to a workgroup of four waves, all of K in LDS at once (rows of 256 bytes of either
// operand, read transposed), no pipeline: several workgroups share a compute unit, one's loads and products under
// another's stores. 128 rows take 64 KB, which leaves two workgroups to a unit. us of the weights' gradients
// with k_gated_grad before them, k_big second: 65 x 7168 x 2048 25.3 and 27.3, 96 x 2880 x 2880 19.7 and 26.5, 128 x 7168 x 2048 28.5 and 29.4.
#pragma once

#include "dense16.hpp"

namespace moe {
namespace d16 {

constexpr int kOuterRows = 128;
inline int outer_lds(int K) { return (K + 15) / 16 * 16 * 512; }

template <int DT>
__global__ __launch_bounds__(256, 4) void k_outer(const Params p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_arr[];  // outer_lds(K) bytes
  lds_u8* smem = (lds_u8*)smem_arr;
  Item it;
  if (!item_of(p, 2, it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, lr = lane & 31, lk = lane >> 5, tr = (lane >> 2) & 3;
  const int m0 = it.mt * 128, n0 = it.nt * 128, z = it.z;
  const int ksteps = (p.K + 15) / 16;
  {
    const int64_t ldm = p.ldm[z], ldn = p.ldn[0];
    const auto rm = rsrc(p.m[z] + m0, ((p.K - 1) * ldm + p.M - m0) * 2), rn = rsrc(p.n[0] + n0, ((p.fold ? p.fold - 1 : p.K - 1) * ldn + p.N - n0) * 2);
    for (int i = wave; i < ksteps * 4; i += 4) {  // 4 K rows of either operand
      int k, chunk;
      major_src<128>(i, lane, k, chunk);
      // rows past K read as zero: past the descriptor's end, or beyond it by offset
      const bool in = k < p.K;
      dma(rm, smem + i * 1024, in ? (uint32_t)(k * ldm * 2 + chunk * 16) : kNoLoad, 0);
      dma(rn, smem + ksteps * 4096 + i * 1024, in ? (uint32_t)((p.fold && k >= p.fold ? k - p.fold : k) * ldn * 2 + chunk * 16) : kNoLoad, 0);
    }
  }
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto at = [&](int col) {
    const int cb = 2 * (col + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
    return (uint32_t)((8 * lk + tr) * 256 + (((cb >> 6) ^ tr) << 6) + (cb & 63));
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  uint32_t ma[2], na[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ma[j] = lds0 + at(wm * 64 + j * 32);
    na[j] = lds0 + ksteps * 4096 + at(wn * 64 + j * 32);
  }
  wait_loads<0>();
  barrier();
  for (int ks = 0; ks < ksteps; ++ks) {
    Frag<true> fm[2], fn[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      fm[j].read(ma[j] + ks * 4096, 1024);
      fn[j].read(na[j] + ks * 4096, 1024);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      fm[j].tie();
      fn[j].tie();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma<DT>(fn[i].get(), fm[j].get(), acc[i][j]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = m0 + wm * 64 + j * 32 + lr;
      float v[4][4];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r >> 2][r & 3] = acc[i][j][r];
      finish_dw<DT>(p, z, row, n0 + wn * 64 + i * 32, v, lk, row < p.M);
    }
}

}  // namespace d16
}  // namespace moe
