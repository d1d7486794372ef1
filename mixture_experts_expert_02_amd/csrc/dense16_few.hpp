// Few rows (decode) of the dense 16-bit products: the weights stream from HBM once.
//
// A workgroup owns 16 FN weight rows (GATED: 8 FN gate and the same up rows, eight by
// eight) and up to 8 XI rows of x; its S waves split K and work each for itself:
// a wave's slice goes memory -> LDS in units of 64 K values, whole 128-byte lines of each row,
// through a ring of D units of its own, so that it waits for nothing but its own oldest
// unit; MFMA 16x16x32, and the partial sums meet in LDS in wave order.
#pragma once

#include "dense16.hpp"

namespace moe {
namespace d16 {

constexpr int kMaxRank = 256;

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == T_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Four neighbouring ranks' products of a row with its adapter's first factor, by one wave: sums of all lanes.
template <int DT>
__device__ __forceinline__ void first_products(const uint16_t* x, const uint16_t* a, int K, int lane, float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = 0.f;
#pragma unroll 4
  for (int k = lane * 8; k < K; k += 512) {
    float xv[8], av[4][8];
    load8<DT>(x, k, xv);
#pragma unroll
    for (int i = 0; i < 4; ++i) load8<DT>(a, (size_t)i * K + k, av[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i] = fmaf(xv[j], av[i][j], s[i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += __shfl_xor(s[i], d);
}

// LORA here: p.sid holds the ids; the scaled x A^T, in float32, come from p.tf, [M, R] in the rows' own order, or (OWN) every
// workgroup finds them for itself while its first units are on their way, which saves a launch where they are few.
template <int DT, int MODE, int S, int FN, int XI, int D, bool OWN>
__global__ __launch_bounds__(64 * S) void k_few(const Params p) {
  constexpr int FM = (XI + 1) / 2, NI = 2 * FN;  // 16-row fragments of x; load instructions of a unit's weights
  constexpr int UNIT = (NI + XI) * 1024;
  constexpr int COLS = MODE == GATED ? 8 * FN : 16 * FN;
  constexpr int PART = FN * FM * 256;  // floats of a wave's partial sums
  static_assert(S * D * UNIT <= 160 * 1024 && S * PART * 4 <= S * D * UNIT, "LDS");
  __shared__ __attribute__((aligned(16))) uint8_t smem_arr[S * D * UNIT];
  lds_u8* smem = (lds_u8*)smem_arr;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = blockIdx.x % p.nt, mt = blockIdx.x / p.nt;
  const int n0 = nt * COLS, m0 = mt * 8 * XI;
  const int units = (p.K + 63) / 64;
  const int lo = wave * units / S, cnt = (wave + 1) * units / S - lo;
  lds_u8* ring = smem + wave * (D * UNIT);

  // lane's row in an instruction's eight, and the chunk it fetches for the slot it fills
  const int r8 = lane >> 3;
  int chunk[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) chunk[q] = (lane & 7) ^ (((q * 8 + r8) >> 1) & 7);
  auto load = [&](int u, int slot) {
    const bool live = u < cnt;
    const int k0 = (lo + u) * 64;
    lds_u8* dst = ring + slot * UNIT;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int w = MODE == GATED ? i & 1 : 0;
      const int first = n0 + (MODE == GATED ? (i >> 1) * 8 : i * 8);
      const int64_t ld = p.ldn[w];
      const auto rs = rsrc(p.n[w] + (int64_t)first * ld, live && first < p.N ? ((min(8, p.N - first) - 1) * ld + p.K) * 2 : 0);
      uint32_t off = (uint32_t)r8 * (uint32_t)(ld * 2) + chunk[i & 1] * 16;
      if (k0 + chunk[i & 1] * 8 >= p.K) off = kNoLoad;
      dma(rs, dst + i * 1024, off, k0 * 2);
    }
    const int64_t ld = p.ldm[0];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int first = m0 + i * 8;
      const auto rs = rsrc(p.m[0] + (int64_t)first * ld, live && first < p.M ? ((min(8, p.M - first) - 1) * ld + p.K) * 2 : 0);
      uint32_t off = (uint32_t)r8 * (uint32_t)(ld * 2) + chunk[i & 1] * 16;
      if (k0 + chunk[i & 1] * 8 >= p.K) off = kNoLoad;
      dma(rs, dst + (NI + i) * 1024, off, k0 * 2);
    }
  };

  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t at[2];  // K halves of a unit
  const int c = lane & 15;
  // with eight rows of x the upper half of the fragment repeats the lower (its results are never used)
  const int cx = XI == 1 ? c & 7 : c;
  uint32_t at_x[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    at[h] = (uint32_t)(uintptr_t)ring + 16 * row_slot(c, 4 * h + (lane >> 4));
    at_x[h] = (uint32_t)(uintptr_t)ring + NI * 1024 + 16 * row_slot(cx, 4 * h + (lane >> 4));
  }
#pragma unroll
  for (int u = 0; u < D - 1; ++u) load(u, u);
  // LORA: what a thread's outputs get besides the projection, loaded and multiplied while the first units are on their way
  // (64 x 2880 x 2895 with rank 32 behind the main loop 13.5 us, here 12.9)
  constexpr int OUT = MODE == LORA ? (8 * XI * COLS + 64 * S - 1) / (64 * S) : 1;
  float lora[OUT], bias[OUT], add[OUT];
  __shared__ float own[OWN ? 8 * XI * kMaxRank : 1];
  if constexpr (OWN) {
    const int per = p.R / 4;
    for (int i = wave; i < min(p.M, 8 * XI) * per; i += S) {
      const int m = i / per, r = (i - m * per) * 4, a = __builtin_amdgcn_readfirstlane(p.sid[m]);
      if (a < 0 || a >= p.L) continue;
      float s[4];
      first_products<DT>(p.m[0] + m * p.ldm[0], p.a + ((int64_t)a * p.R + r) * p.K, p.K, lane, s);
      if (lane < 4) own[m * p.R + r + lane] = (lane < 2 ? lane ? s[1] : s[0] : lane == 2 ? s[2] : s[3]) * p.scales[a];
    }
    __syncthreads();
  }
  if constexpr (MODE == LORA) {
    int64_t b[OUT], t[OUT];
    bool has[OUT];
#pragma unroll
    for (int o = 0; o < OUT; ++o) {
      const int x = tid + o * 64 * S, row = min(m0 + x / COLS, p.M - 1), col = min(n0 + x % COLS, p.N - 1);
      const int a = p.sid[row];
      has[o] = a >= 0 && a < p.L;
      b[o] = ((int64_t)(has[o] ? a : 0) * p.N + col) * p.R;
      t[o] = (int64_t)row * p.R;
      lora[o] = 0.f;
      bias[o] = p.bias[0] ? p.bias[0][col] : 0.f;
      add[o] = p.add ? load1<DT>(p.add, (size_t)(row * p.ld_add + col)) : 0.f;
    }
#pragma unroll 2
    for (int r = 0; r < p.R; r += 8) {
#pragma unroll
      for (int o = 0; o < OUT; ++o) {
        float bv[8], tv[8];
        load8<DT>(p.b, (size_t)(b[o] + r), bv);
        load8<T_FP32>(OWN ? own : p.tf, (size_t)(t[o] + r), tv);
#pragma unroll
        for (int q = 0; q < 8; ++q) lora[o] = fmaf(tv[q], bv[q], lora[o]);
      }
    }
    // a row without an adapter has no first product either: what was read there is left out
#pragma unroll
    for (int o = 0; o < OUT; ++o) lora[o] = has[o] ? lora[o] : 0.f;
  }
  int slot = 0;
  for (int u = 0; u < cnt; ++u) {
    load(u + D - 1, slot == 0 ? D - 1 : slot - 1);  // the slot read in the last turn
    wait_loads<(D - 1) * (NI + XI)>();
    Frag<false> fw[2][FN], fx[2][FM];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FN; ++i) fw[h][i].read(at[h] + slot * UNIT + i * 2048, 0);
#pragma unroll
      for (int j = 0; j < FM; ++j) fx[h][j].read(at_x[h] + slot * UNIT + j * 2048, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FN; ++i) fw[h][i].tie();
#pragma unroll
      for (int j = 0; j < FM; ++j) fx[h][j].tie();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = mfma16<DT>(fw[h][i].get(), fx[h][j].get(), acc[i][j]);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  wait_loads<0>();
  __syncthreads();

  // partial sums [wave][fragment][row of x][weight row]
  float* part = (float*)smem_arr;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) *(f32x4*)(part + wave * PART + (i * FM + j) * 256 + c * 16 + 4 * (lane >> 4)) = acc[i][j];
  __syncthreads();
  auto sum = [&](int i, int m, int r) {
    const float* q = part + (i * FM + (m >> 4)) * 256 + (m & 15) * 16 + r;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < S; ++w) s += q[w * PART];
    return s;
  };
  const int rows = min(8 * XI, p.M - m0);
  constexpr int TURNS = (8 * XI * COLS + 64 * S - 1) / (64 * S);
#pragma unroll
  for (int o = 0; o < TURNS; ++o) {
    const int x = tid + o * 64 * S;
    if (x >= rows * COLS) break;
    const int m = x / COLS, n = x % COLS, col = n0 + n;
    const int64_t row = m0 + m;
    if (col >= p.N) continue;
    if constexpr (MODE == GATED) {
      float g = sum(n >> 3, m, n & 7), u = sum(n >> 3, m, 8 + (n & 7));
      if (p.bias[0]) {
        g += p.bias[0][col];
        u += p.bias[1][col];
      }
      if (p.keep[0]) {
        store1<DT>(p.keep[0], (size_t)(row * p.ld_keep[0] + col), g);
        store1<DT>(p.keep[1], (size_t)(row * p.ld_keep[1] + col), u);
      }
      float v = 0.f;
      with_act(p.act, [&](auto k) { v = act_f<decltype(k)::value>(p.act, g, u); });
      store1<DT>(p.out[0], (size_t)(row * p.ldo[0] + col), v);
    } else {
      const float v = sum(n >> 4, m, n & 15) + lora[o] + bias[o] + add[o];
      store1<DT>(p.out[0], (size_t)(row * p.ldo[0] + col), v);
    }
  }
}

}  // namespace d16
}  // namespace moe
