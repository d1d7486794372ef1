// Low-rank adapters of many requests: rows sorted by adapter, and their products
// with the first factors, t_m = s_a x_m A_a^T for row m of adapter a.
// The second factors join the projection's tiles (dense16.hpp, LORA).
#pragma once

#include "dense16.hpp"

namespace moe {
namespace d16 {

constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 256;

struct SortParams {
  const int32_t* ids;  // [M]; outside [0, L): no adapter
  int32_t *perm, *sid; // [M]
  int32_t* ends;       // [L]
  int32_t M, L;
};

// One workgroup: counts, their running sum, places. Rows of one adapter may come in any order among
// themselves: nothing that is computed from a row depends on its place.
__global__ __launch_bounds__(1024) void k_lora_sort(const SortParams p) {
  __shared__ int32_t at[kMaxAdapters + 1];  // counts, then next places
  __shared__ int32_t wave_sum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i <= p.L; i += 1024) at[i] = 0;
  __syncthreads();
  auto key = [&](int m) {
    const int a = p.ids[m];
    return a >= 0 && a < p.L ? a : p.L;
  };
  // a wave whose rows share one adapter counts them at once
  auto take = [&](int m, bool in) {
    const int a = in ? key(m) : -1;
    const uint64_t live = __ballot(in);
    const int first = __builtin_amdgcn_readfirstlane(a);
    const uint64_t same = __ballot(in && a == first);
    int place = 0;
    if (first >= 0 && same == live) {
      if (lane == 0) place = atomicAdd(&at[first], __popcll(live));
      place = __builtin_amdgcn_readfirstlane(place) + __popcll(live & lanemask_lt());
    } else if (in) {
      place = atomicAdd(&at[a], 1);
    }
    return place;
  };
  const int steps = (p.M + 1023) / 1024;
  for (int i = 0; i < steps; ++i) take(i * 1024 + tid, i * 1024 + tid < p.M);
  __syncthreads();
  // exclusive running sum, five counters to a thread
  constexpr int PER = (kMaxAdapters + 1 + 1023) / 1024;
  int c[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = tid * PER + j;
    c[j] = i <= p.L ? at[i] : 0;
    sum += c[j];
  }
  int run = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) wave_sum[wave] = run;
  __syncthreads();
  int base = run - sum;
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = tid * PER + j;
    if (i <= p.L) at[i] = base;
    base += c[j];
    if (i < p.L) p.ends[i] = base;
  }
  __syncthreads();
  for (int i = 0; i < steps; ++i) {
    const int m = i * 1024 + tid;
    const int place = take(m, m < p.M);
    if (m < p.M) {
      p.perm[place] = m;
      p.sid[place] = key(m);
    }
  }
}

struct ShrinkParams {
  const uint16_t* x;
  const uint16_t* a;      // [L, R, K]
  const float* scales;    // [L]
  const int32_t *perm, *sid, *ends;
  uint16_t* t;            // [M, 2R]
  float* tf;              // [M]
  int64_t ldx;
  int32_t M, K, R, L;
};

// 16 sorted rows to a workgroup; its eight waves split K and join in LDS in wave
// order. The results (float32) get their adapter's scale and leave as two
// 16-bit parts over the row's own power of two, 16 significand bits or more of
// each: what the second product loses by its 16-bit operands is far below the
// output's own rounding, and float16 keeps results of any size.
// RF: fragments of 16 ranks.
template <int DT, int RF>
__global__ __launch_bounds__(512) void k_lora_shrink(const ShrinkParams p) {
  constexpr int RC = RF < 4 ? RF : 4;  // fragments joined at a time
  __shared__ float part[8][RC][16][17];
  __shared__ float sum[RF * 16][17];
  __shared__ float top[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, kq = (lane >> 4) * 8;
  const int m0 = blockIdx.x * 16, last = min(m0 + 16, p.M);
  const int row = min(m0 + c, p.M - 1);
  const int id = m0 + c < p.M ? p.sid[row] : p.L;
  const uint16_t* xr = p.x + (int64_t)p.perm[row] * p.ldx;
  const int steps = (p.K + 31) / 32, lo = wave * steps / 8, hi = (wave + 1) * steps / 8;
  f32x4 acc[RF];
#pragma unroll
  for (int i = 0; i < RF; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  int pos = m0;
  while (pos < last) {
    const int a = __builtin_amdgcn_readfirstlane(p.sid[pos]);
    if (a >= p.L) break;
    pos = max(pos + 1, __builtin_amdgcn_readfirstlane(p.ends[a]));
    f32x4 tmp[RF];
#pragma unroll
    for (int i = 0; i < RF; ++i) tmp[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* ar = p.a + (int64_t)a * p.R * p.K;
#pragma unroll 4
    for (int s = lo; s < hi; ++s) {
      const int k = s * 32 + kq;
      const bool in = k < p.K;
      const u32x4 zero = {0, 0, 0, 0};
      const u32x4 xv = in ? *(const u32x4*)(xr + k) : zero;
#pragma unroll
      for (int i = 0; i < RF; ++i) {
        const int r = min(i * 16 + c, p.R - 1);
        const u32x4 av = in ? *(const u32x4*)(ar + (int64_t)r * p.K + k) : zero;
        if constexpr (DT == T_BF16)
          tmp[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, xv), tmp[i], 0, 0, 0);
        else
          tmp[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, av), __builtin_bit_cast(f16x8, xv), tmp[i], 0, 0, 0);
      }
    }
    if (id == a) {
#pragma unroll
      for (int i = 0; i < RF; ++i) acc[i] = tmp[i];
    }
  }
  // rank 16 i + 4 (lane / 16) + q of row c
#pragma unroll
  for (int i0 = 0; i0 < RF; i0 += RC) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RC; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[wave][i][4 * (lane >> 4) + q][c] = acc[i0 + i][q];
    __syncthreads();
    for (int x = tid; x < RC * 256; x += 512) {
      const int i = x >> 8, r = (x >> 4) & 15, m = x & 15;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += part[w][i][r][m];
      sum[(i0 + i) * 16 + r][m] = s;
    }
  }
  __syncthreads();
  if (tid < 16) {
    const int a = m0 + tid < p.M ? p.sid[m0 + tid] : p.L;
    const float sc = a < p.L ? p.scales[a] : 0.f;
    float most = 0.f;
    for (int r = 0; r < p.R; ++r) {
      const float v = a < p.L ? sum[r][tid] * sc : 0.f;
      sum[r][tid] = v;
      most = fmaxf(most, fabsf(v));
    }
    // 2^e above the largest finite magnitude; float32's ends keep both it and its inverse normal
    int e = most > 0.f && most < INFINITY ? ilogbf(most) + 1 : 0;
    e = min(max(e, -120), 120);
    top[tid] = ldexpf(1.f, -e);
    if (m0 + tid < p.M) p.tf[m0 + tid] = ldexpf(1.f, e);
  }
  __syncthreads();
  for (int x = tid; x < 16 * p.R; x += 512) {
    const int m = x / p.R, r = x - m * p.R;
    if (m0 + m >= p.M) break;
    const float v = sum[r][m] * top[m];
    const float h = round_to<DT>(v);
    const float l = fabsf(h) < INFINITY ? v - h : 0.f;
    uint16_t* t = p.t + (int64_t)(m0 + m) * 2 * p.R + r;
    if constexpr (DT == T_BF16) {
      *(__bf16*)t = (__bf16)h;
      *(__bf16*)(t + p.R) = (__bf16)l;
    } else {
      *(_Float16*)t = (_Float16)h;
      *(_Float16*)(t + p.R) = (_Float16)l;
    }
  }
}

}  // namespace d16
}  // namespace moe
