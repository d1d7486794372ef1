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
    if (m >= p.M) return -1;
    const int a = p.ids[m];
    return a >= 0 && a < p.L ? a : p.L;
  };
  // one place for each lane with a key; a wave whose rows share one adapter counts them at once, by its first lane
  auto shared_by = [&](int a) {
    const int first = __builtin_amdgcn_readfirstlane(a);
    return __ballot(a >= 0 && a != first) == 0;
  };
  auto count = [&](int a) {
    const bool all = shared_by(a);
    const uint64_t live = __ballot(a >= 0);  // with all lanes active: in the branch below it would count the first alone
    const int n = all ? __popcll(live) : 1;
    int place = 0;
    if (a >= 0 && (!all || lane == 0)) place = atomicAdd(&at[a], n);
    return place;
  };
  // eight keys to a thread at a time, so that their loads overlap; the first 8192 rows' stay in registers
  constexpr int KEYS = 8;
  int keep[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; ++i) keep[i] = key(i * 1024 + tid);
#pragma unroll
  for (int i = 0; i < KEYS; ++i) count(keep[i]);
  for (int m = KEYS * 1024; m < p.M; m += KEYS * 1024) {
    int k[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) k[i] = key(m + i * 1024 + tid);
#pragma unroll
    for (int i = 0; i < KEYS; ++i) count(k[i]);
  }
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
  }
  __syncthreads();
  auto put = [&](int m0, const int (&k)[KEYS]) {
    int place[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) place[i] = count(k[i]);
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      if (shared_by(k[i])) place[i] = __builtin_amdgcn_readfirstlane(place[i]) + __popcll(__ballot(k[i] >= 0) & lanemask_lt());
      if (k[i] < 0) continue;
      p.perm[place[i]] = m0 + i * 1024 + tid;
      p.sid[place[i]] = k[i];
    }
  };
  put(0, keep);
  for (int m = KEYS * 1024; m < p.M; m += KEYS * 1024) {
    int k[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) k[i] = key(m + i * 1024 + tid);
    put(m, k);
  }
}

struct ShrinkParams {
  const uint16_t* x;
  const uint16_t* a;      // [L, R, K]
  const float* scales;    // [L]
  const int32_t *perm, *sid;
  uint16_t* t;            // see part_at
  float* tf;              // [M]
  float* part;            // [K ranges][M][R], with more than one
  int64_t ldx;
  int32_t M, K, R, L;
};

// A row's results over the power of two above their largest, in two parts of the
// type, 16 significand bits or more together: what the second product loses by its 16-bit
// operands is far below the output's own rounding, and float16 keeps results of any size.
// v: this lane's ranks r0, r0 + LANES, .. of row m; LANES lanes of the wave hold the row.
template <int DT, int LANES, int N>
__device__ __forceinline__ void store_parts(float (&v)[N], int r0, int R, int m, uint16_t* t, float* tf) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(v[i]));
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
  // float32's ends keep the power and its inverse normal
  int e = most > 0.f && most < INFINITY ? ilogbf(most) + 1 : 0;
  e = min(max(e, -120), 120);
  const float inv = ldexpf(1.f, -e);
  if (r0 == 0) tf[m] = ldexpf(1.f, e);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * LANES;
    if (r >= R) continue;
    const float w = v[i] * inv, h = round_to<DT>(w);
    const float l = fabsf(h) < INFINITY ? w - h : 0.f;
    store1<DT>(t, part_at(m, r, R), h);
    store1<DT>(t, part_at(m, R + r, R), l);
  }
}

// 16 FX sorted rows to a workgroup (and a K range: blockIdx.y); its eight waves split K and join in LDS in wave
// order. RF: fragments of 16 ranks.
template <int DT, int RF, int FX>
__global__ __launch_bounds__(512) void k_lora_shrink(const ShrinkParams p) {
  constexpr int ROWS = 16 * FX;
  constexpr int U = RF + FX <= 4 ? 6 : RF + FX <= 6 ? 4 : RF + FX <= 10 ? 2 : 1;  // K steps whose loads are issued together
  constexpr int RC = RF < 2 ? RF : 2;                                            // fragments joined at a time
  __shared__ float part[8][RC][16][ROWS + 1];
  __shared__ float sum[RF * 16][ROWS + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, kq = (lane >> 4) * 8;
  const int m0 = blockIdx.x * ROWS;
  int id[FX];
  const uint16_t* xr[FX];
#pragma unroll
  for (int j = 0; j < FX; ++j) {
    const int row = min(m0 + j * 16 + c, p.M - 1);
    id[j] = m0 + j * 16 + c < p.M ? p.sid[row] : p.L;
    xr[j] = p.x + (int64_t)p.perm[row] * p.ldx;
  }
  const int steps = (p.K + 31) / 32, nw = 8 * gridDim.y, w = blockIdx.y * 8 + wave;
  const int lo = (int)((int64_t)w * steps / nw), hi = (int)((int64_t)(w + 1) * steps / nw);
  f32x4 acc[RF][FX];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < FX; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint64_t rows[FX];  // those whose adapter is still to come
#pragma unroll
  for (int j = 0; j < FX; ++j) rows[j] = __ballot(id[j] < p.L);
  while (rows[0] | rows[FX - 1]) {
    const int a = rows[0] ? __builtin_amdgcn_readlane(id[0], __builtin_ctzll(rows[0])) : __builtin_amdgcn_readlane(id[FX - 1], __builtin_ctzll(rows[FX - 1]));
#pragma unroll
    for (int j = 0; j < FX; ++j) rows[j] &= ~__ballot(id[j] == a);
    f32x4 tmp[RF][FX];
    const uint16_t* ar[RF];
#pragma unroll
    for (int i = 0; i < RF; ++i) {
#pragma unroll
      for (int j = 0; j < FX; ++j) tmp[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      ar[i] = p.a + ((int64_t)a * p.R + min(i * 16 + c, p.R - 1)) * p.K;
    }
    for (int s = lo; s < hi; s += U) {
      u32x4 xv[U][FX], av[U][RF];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + u) * 32 + kq;
        const bool in = s + u < hi && k < p.K;
#pragma unroll
        for (int j = 0; j < FX; ++j) {
          xv[u][j] = u32x4{0, 0, 0, 0};
          if (in) xv[u][j] = *(const u32x4*)(xr[j] + k);
        }
#pragma unroll
        for (int i = 0; i < RF; ++i) {
          av[u][i] = u32x4{0, 0, 0, 0};
          if (in) av[u][i] = *(const u32x4*)(ar[i] + k);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RF; ++i)
#pragma unroll
          for (int j = 0; j < FX; ++j) tmp[i][j] = mfma16<DT>(av[u][i], xv[u][j], tmp[i][j]);
    }
#pragma unroll
    for (int j = 0; j < FX; ++j)
      if (id[j] == a) {
#pragma unroll
        for (int i = 0; i < RF; ++i) acc[i][j] = tmp[i][j];
      }
  }
  // rank 16 i + 4 (lane / 16) + q of row 16 j + c
#pragma unroll
  for (int i0 = 0; i0 < RF; i0 += RC) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RC; ++i)
#pragma unroll
      for (int j = 0; j < FX; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[wave][i][4 * (lane >> 4) + q][j * 16 + c] = acc[i0 + i][j][q];
    __syncthreads();
    for (int x = tid; x < RC * 16 * ROWS; x += 512) {
      const int i = x / (16 * ROWS), r = x / ROWS % 16, m = x % ROWS;
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < 8; ++v) s += part[v][i][r][m];
      sum[(i0 + i) * 16 + r][m] = s;
    }
  }
  __syncthreads();
  // 512 / ROWS lanes to a row
  constexpr int LANES = 512 / ROWS, N = (RF * 16 + LANES - 1) / LANES;
  const int m = tid / LANES, r0 = tid % LANES;
  if (m0 + m >= p.M) return;
  const int a = p.sid[m0 + m];
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = r0 + LANES * i < p.R && a < p.L ? sum[min(r0 + LANES * i, RF * 16 - 1)][m] : 0.f;
  if (gridDim.y > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (r0 + LANES * i < p.R) p.part[((size_t)blockIdx.y * p.M + m0 + m) * p.R + r0 + LANES * i] = v[i];
    return;
  }
  const float sc = a < p.L ? p.scales[a] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= sc;
  store_parts<DT, LANES, N>(v, r0, p.R, m0 + m, p.t, p.tf);
}

// The K ranges' results joined in their order, a row to a wave, N ranks to a lane.
template <int DT, int N>
__global__ __launch_bounds__(256) void k_lora_finish(const ShrinkParams p, int ranges) {
  const int lane = threadIdx.x & 63, m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= p.M) return;
  const int a = p.sid[m];
  const float sc = a < p.L ? p.scales[a] : 0.f;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = min(lane + 64 * i, p.R - 1);
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < ranges; ++k) s += p.part[((size_t)k * p.M + m) * p.R + r];
    v[i] = a < p.L && lane + 64 * i < p.R ? s * sc : 0.f;
  }
  store_parts<DT, 64, N>(v, lane, p.R, m, p.t, p.tf);
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

// The adapters' part alone (no projection): out = bias + add + f_m (t_m B_a^T). A workgroup owns 16 `frags` sorted rows
// and 256 columns, 64 to a wave; both operands go straight into registers in the MFMA's layout, the factor's
// rows once for all fragments of the same adapter. Bound by the factors' and outputs' bytes.
template <int DT>
__global__ __launch_bounds__(256) void k_lora_expand(const Params p, int frags) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int col0 = blockIdx.y * 256 + (threadIdx.x >> 6) * 64;
  if (col0 >= p.N) return;
  u32x4 b[4][2];
  int held = -1;
  for (int x = 0; x < frags; ++x) {
    const int r0 = (blockIdx.x * frags + x) * 16;
    if (r0 >= p.M) return;
    const int row = min(r0 + c, p.M - 1);
    const int id = r0 + c < p.M ? p.sid[row] : p.L;
    const float f = p.tf[row];
    const int64_t orow = p.perm[row];
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint64_t rows = __ballot(id < p.L);
    while (rows) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rows));
      rows &= ~__ballot(id == a);
      for (int c0 = 0; c0 < p.R; c0 += 64) {
        u32x4 hi[2], lo[2];
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const int k = c0 + 32 * ks + 8 * g;
          hi[ks] = lo[ks] = zero;
          if (k < p.R) {
            hi[ks] = *(const u32x4*)(p.t + part_at(row, k, p.R));
            lo[ks] = *(const u32x4*)(p.t + part_at(row, p.R + k, p.R));
          }
          if (held != a || p.R > 64) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = col0 + i * 16 + c;
              b[i][ks] = zero;
              if (k < p.R && col < p.N) b[i][ks] = *(const u32x4*)(p.b + ((int64_t)a * p.N + col) * p.R + k);
            }
          }
        }
        held = a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 tmp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            tmp = mfma16<DT>(b[i][ks], hi[ks], tmp);
            tmp = mfma16<DT>(b[i][ks], lo[ks], tmp);
          }
          if (id == a) {
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] += tmp[q] * f;
          }
        }
      }
    }
    if (r0 + c >= p.M) continue;
    uint16_t* out = (uint16_t*)p.out[0] + orow * p.ldo[0];
    const uint16_t* add = p.add ? (const uint16_t*)p.add + orow * p.ld_add : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = col0 + i * 16 + 4 * g;  // four neighbours
      if (p.vec && col + 4 <= p.N) {
        uint2 old = {0, 0}, res;
        if (add) old = *(const uint2*)(add + col);
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = acc[i][q] + (p.bias[0] ? p.bias[0][col + q] : 0.f);
        if (add) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += load1<DT>(&old, q);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) store1<DT>(&res, q, v[q]);
        *(uint2*)(out + col) = res;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (col + q >= p.N) break;
          float v = acc[i][q] + (p.bias[0] ? p.bias[0][col + q] : 0.f);
          if (add) v += load1<DT>(add, col + q);
          store1<DT>(out, col + q, v);
        }
      }
    }
  }
}

}  // namespace d16
}  // namespace moe
