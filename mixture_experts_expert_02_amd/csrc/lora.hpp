// Low-rank adapters of many requests: rows sorted by adapter, and their products
// with the first factors, t_m = s_a x_m A_a^T for row m of adapter a.
// The second factors join the projection's tiles (dense16.hpp, LORA).
#pragma once

#include "dense16_few.hpp"

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
  float* part;            // [K ranges][M][R], with more than one
  int64_t ldx;
  int32_t M, K, R, L;
};

// A row's results over the power of two above their largest, in two parts of the
// type, 16 significand bits or more together: what the second product loses by its 16-bit
// operands is far below the output's own rounding, and float16 keeps results of any size.
// v: this lane's ranks r0, r0 + LANES, ..; LANES lanes of the wave hold the row.
template <int DT, int LANES, int N>
__device__ __forceinline__ void store_parts(float (&v)[N], int r0, int R, uint16_t* t, float* tf) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(v[i]));
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
  // float32's ends keep the power and its inverse normal
  int e = most > 0.f && most < INFINITY ? ilogbf(most) + 1 : 0;
  e = min(max(e, -120), 120);
  const float inv = ldexpf(1.f, -e);
  if (r0 == 0) *tf = ldexpf(1.f, e);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * LANES;
    if (r >= R) continue;
    const float w = v[i] * inv, h = round_to<DT>(w);
    const float l = fabsf(h) < INFINITY ? w - h : 0.f;
    if constexpr (DT == T_BF16) {
      ((__bf16*)t)[r] = (__bf16)h;
      ((__bf16*)t)[R + r] = (__bf16)l;
    } else {
      ((_Float16*)t)[r] = (_Float16)h;
      ((_Float16*)t)[R + r] = (_Float16)l;
    }
  }
}

// 16 sorted rows to a workgroup (and a K range: blockIdx.y); its eight waves split K and join in LDS in wave order.
// RF: fragments of 16 ranks.
template <int DT, int RF>
__global__ __launch_bounds__(512) void k_lora_shrink(const ShrinkParams p) {
  constexpr int U = RF <= 2 ? 4 : RF == 4 ? 3 : RF == 8 ? 2 : 1;  // K steps whose loads are issued together
  constexpr int RC = RF < 4 ? RF : 4;                             // fragments joined at a time
  __shared__ float part[8][RC][16][17];
  __shared__ float sum[RF * 16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, kq = (lane >> 4) * 8;
  const int m0 = blockIdx.x * 16, last = min(m0 + 16, p.M);
  const int row = min(m0 + c, p.M - 1);
  const int id = m0 + c < p.M ? p.sid[row] : p.L;
  const uint16_t* xr = p.x + (int64_t)p.perm[row] * p.ldx;
  const int steps = (p.K + 31) / 32, nw = 8 * gridDim.y, w = blockIdx.y * 8 + wave;
  const int lo = (int)((int64_t)w * steps / nw), hi = (int)((int64_t)(w + 1) * steps / nw);
  f32x4 acc[RF];
#pragma unroll
  for (int i = 0; i < RF; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  int pos = m0;
  while (pos < last) {
    const int a = __builtin_amdgcn_readfirstlane(p.sid[pos]);
    if (a >= p.L) break;
    pos = max(pos + 1, __builtin_amdgcn_readfirstlane(p.ends[a]));
    f32x4 tmp[RF];
    const uint16_t* ar[RF];
#pragma unroll
    for (int i = 0; i < RF; ++i) {
      tmp[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      ar[i] = p.a + ((int64_t)a * p.R + min(i * 16 + c, p.R - 1)) * p.K;
    }
    for (int s = lo; s < hi; s += U) {
      u32x4 xv[U], av[U][RF];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + u) * 32 + kq;
        const bool in = s + u < hi && k < p.K;
        xv[u] = u32x4{0, 0, 0, 0};
        if (in) xv[u] = *(const u32x4*)(xr + k);
#pragma unroll
        for (int i = 0; i < RF; ++i) {
          av[u][i] = u32x4{0, 0, 0, 0};
          if (in) av[u][i] = *(const u32x4*)(ar[i] + k);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RF; ++i) tmp[i] = mfma16<DT>(av[u][i], xv[u], tmp[i]);
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
      for (int v = 0; v < 8; ++v) s += part[v][i][r][m];
      sum[(i0 + i) * 16 + r][m] = s;
    }
  }
  __syncthreads();
  // 32 lanes to a row
  const int m = tid >> 5, r0 = tid & 31;
  if (m0 + m >= p.M) return;
  const int a = p.sid[m0 + m];
  constexpr int N = RF < 2 ? 1 : RF / 2;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = r0 + 32 * i < p.R && a < p.L ? sum[min(r0 + 32 * i, RF * 16 - 1)][m] : 0.f;
  if (gridDim.y > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (r0 + 32 * i < p.R) p.part[((size_t)blockIdx.y * p.M + m0 + m) * p.R + r0 + 32 * i] = v[i];
    return;
  }
  const float sc = a < p.L ? p.scales[a] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= sc;
  store_parts<DT, 32, N>(v, r0, p.R, p.t + (int64_t)(m0 + m) * 2 * p.R, p.tf + m0 + m);
}

// The K ranges' results joined in their order, a row to a wave.
template <int DT>
__global__ __launch_bounds__(256) void k_lora_finish(const ShrinkParams p, int ranges) {
  const int lane = threadIdx.x & 63, m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= p.M) return;
  const int a = p.sid[m];
  const float sc = a < p.L ? p.scales[a] : 0.f;
  float v[kMaxRank / 64];
#pragma unroll
  for (int i = 0; i < kMaxRank / 64; ++i) v[i] = 0.f;
  if (a < p.L) {
    for (int k = 0; k < ranges; ++k)
#pragma unroll
      for (int i = 0; i < kMaxRank / 64; ++i)
        if (lane + 64 * i < p.R) v[i] += p.part[((size_t)k * p.M + m) * p.R + lane + 64 * i];
#pragma unroll
    for (int i = 0; i < kMaxRank / 64; ++i) v[i] *= sc;
  }
  store_parts<DT, 64, kMaxRank / 64>(v, lane, p.R, p.t + (int64_t)m * 2 * p.R, p.tf + m);
}

// Few rows: row blockIdx.x's products with eight ranks of its adapter, two to a wave, in float32, scaled;
// rows without an adapter are left out. p.sid: the ids, p.tf: [M, R].
template <int DT>
__global__ __launch_bounds__(256) void k_lora_shrink_few(const ShrinkParams p) {
  const int m = blockIdx.x, lane = threadIdx.x & 63, r = blockIdx.y * 8 + (threadIdx.x >> 6) * 2;
  const int a = p.sid[m];
  if (a < 0 || a >= p.L) return;
  const uint16_t* x = p.x + (int64_t)m * p.ldx;
  const uint16_t* ar = p.a + ((int64_t)a * p.R + r) * p.K;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int k = lane * 8; k < p.K; k += 512) {
    float xv[8], a0[8], a1[8];
    load8<DT>(x, k, xv);
    load8<DT>(ar, k, a0);
    load8<DT>(ar + p.K, k, a1);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s0 = fmaf(xv[j], a0[j], s0);
      s1 = fmaf(xv[j], a1[j], s1);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    s0 += __shfl_xor(s0, d);
    s1 += __shfl_xor(s1, d);
  }
  if (lane < 2) p.tf[(int64_t)m * p.R + r + lane] = (lane ? s1 : s0) * p.scales[a];
}

}  // namespace d16
}  // namespace moe
