// Low-rank adapters of many requests: rows sorted by adapter, and their products
// with the first factors, t_m = s_a x_m A_a^T for row m of adapter a.
// The second factors join the projection's tiles (dense16.hpp, LORA).
#pragma once

#include "dense16_few.hpp"

namespace moe {
namespace d16 {

constexpr int kMaxAdapters = 4096;

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
  int32_t *perm, *sid;    // of the sorted rows
  const int32_t* ids;     // k_lora_shrink_few and SORT
  uint16_t* t;            // see part_at
  float* tf;              // [M]
  float* part;            // [K ranges][M][R], with more than one
  int64_t ldx;
  int32_t M, K, R, L;
};

// the power of two above |v|; float32's ends keep it and its inverse normal
__device__ __forceinline__ int power_above(float most) {
  const int e = most > 0.f && most < INFINITY ? ilogbf(most) + 1 : 0;
  return min(max(e, -120), 120);
}
// w: a product with a power of two, so that however it is rounded the upper part is the same
template <int DT>
__device__ __forceinline__ void two_parts(float w, float& h, float& l) {
  h = round_to<DT>(w);
  l = fabsf(h) < INFINITY ? w - h : 0.f;
}

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
  const int e = power_above(most);
  const float inv = ldexpf(1.f, -e);
  if (r0 == 0) tf[m] = ldexpf(1.f, e);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * LANES;
    if (r >= R) continue;
    float h, l;
    two_parts<DT>(v[i] * inv, h, l);
    store1<DT>(t, part_at(m, r, R), h);
    store1<DT>(t, part_at(m, R + r, R), l);
  }
}

// Sorted rows m0 .. m0 + ROWS - 1 of at most kSortRows, found by a workgroup of 512 threads for itself: counts and
// places of the adapters as in k_lora_sort, but rows of one adapter keep their order, so that all workgroups agree. A row's
// place is its adapter's first one, the rows of it in the 64-row pieces before, and those in the lanes before. Two keys to a thread are
// the most. us of a call without a projection, rank 64, with k_lora_sort in place of this: 513 x 4096 x 2048 24.4 and 27.5, 1024 x 7168 x 2048 38.2 and 41.0.
constexpr int kSortRows = 1024;
template <int ROWS>
__device__ __forceinline__ void sort_here(const ShrinkParams& p, int m0, int (&perm)[ROWS], int (&sid)[ROWS]) {
  __shared__ int32_t at[kMaxAdapters + 1];
  __shared__ int32_t wave_sum[8];
  __shared__ __attribute__((aligned(16))) int32_t piece[ROWS][kSortRows / 64];  // rows of the adapter whose first place in the window this is
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int key[2] = {-1, -1};
  {
    const int m = min(tid, p.M - 1), m2 = min(tid + 512, p.M - 1);
    const int a = p.ids[m], a2 = p.ids[m2];
    if (tid < p.M) key[0] = a >= 0 && a < p.L ? a : p.L;
    if (tid + 512 < p.M) key[1] = a2 >= 0 && a2 < p.L ? a2 : p.L;
  }
  for (int i = tid; i <= p.L; i += 512) at[i] = 0;
  for (int i = tid; i < ROWS * (kSortRows / 64); i += 512) (&piece[0][0])[i] = 0;
  __syncthreads();
  if (key[0] >= 0) atomicAdd(&at[key[0]], 1);
  if (key[1] >= 0) atomicAdd(&at[key[1]], 1);
  __syncthreads();
  const int per = p.L / 512 + 1;  // counters to a thread: at most 9
  int sum = 0;
#pragma unroll 1
  for (int j = 0; j < per; ++j) {
    const int i = tid * per + j;
    if (i <= p.L) sum += at[i];
  }
  int run = sum;
#pragma unroll 1
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) wave_sum[wave] = run;
  __syncthreads();
  int base = run - sum;
#pragma unroll 1
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
#pragma unroll 1
  for (int j = 0; j < per; ++j) {
    const int i = tid * per + j;
    if (i > p.L) break;
    const int n = at[i];
    at[i] = base;
    base += n;
  }
  __syncthreads();
  // the adapters of the window in this wave's rows, one after the other
  int place[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = key[i], first = k < 0 ? 0 : at[k], end = k < 0 ? 0 : k < p.L ? at[k + 1] : p.M;
    const bool near = k >= 0 && first < m0 + ROWS && end > m0;
    place[i] = near ? first : -1;
    uint64_t left = __ballot(near);
#pragma unroll 1
    while (left) {
      const int a = __builtin_amdgcn_readlane(k, __builtin_ctzll(left));
      const uint64_t same = __ballot(k == a);
      left &= ~same;
      if (k == a) {
        place[i] += __popcll(same & lanemask_lt());
        piece[max(first - m0, 0)][i * 8 + wave] = __popcll(same);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (place[i] < 0) continue;
    const int slot = max(at[key[i]] - m0, 0);
    int before = 0;
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
      const int4 n = *(const int4*)&piece[slot][q];
      const int here = i * 8 + wave - q;
      before += (here > 0 ? n.x : 0) + (here > 1 ? n.y : 0) + (here > 2 ? n.z : 0) + (here > 3 ? n.w : 0);
    }
    const int at_row = place[i] + before - m0;
    if (at_row >= 0 && at_row < ROWS) {
      perm[at_row] = i * 512 + tid;
      sid[at_row] = key[i];
    }
  }
  __syncthreads();
}

// 16 FX sorted rows to a workgroup (and a K range: blockIdx.y); its eight waves split K and join in LDS in wave
// order. RF: fragments of 16 ranks. SORT: the rows are found here and their places stored for the kernels behind.
template <int DT, int RF, int FX, bool SORT>
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
  __shared__ int32_t perm_of[ROWS], id_of[ROWS];
  if constexpr (SORT) {
    sort_here<ROWS>(p, m0, perm_of, id_of);
    if (blockIdx.y == 0 && tid < ROWS && m0 + tid < p.M) {
      p.perm[m0 + tid] = perm_of[tid];
      p.sid[m0 + tid] = id_of[tid];
    }
  } else {
    if (tid < ROWS) {
      const int row = min(m0 + tid, p.M - 1);
      perm_of[tid] = p.perm[row];
      id_of[tid] = p.sid[row];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < FX; ++j) {
    const int row = min(j * 16 + c, p.M - 1 - m0);
    id[j] = m0 + j * 16 + c < p.M ? id_of[row] : p.L;
    xr[j] = p.x + (int64_t)perm_of[row] * p.ldx;
  }
  const int steps = (p.K + 31) / 32, nw = 8 * gridDim.y, w = blockIdx.y * 8 + wave;
  const int lo = (int)((uint32_t)(w * steps) / (uint32_t)nw), hi = (int)((uint32_t)((w + 1) * steps) / (uint32_t)nw);  // below 2^23
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
  const int a = id_of[m];
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

// The K ranges' results joined in their order, a row to a wave, N ranks to a lane. All ranges' loads at once, whatever
// their number, here and in k_lora_expand.
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
    float s = 0.f, x[kMaxRanges];
#pragma unroll
    for (int k = 0; k < kMaxRanges; ++k) x[k] = p.part[((size_t)min(k, ranges - 1) * p.M + m) * p.R + r];
#pragma unroll
    for (int k = 0; k < kMaxRanges; ++k) s = k < ranges ? s + x[k] : s;
    v[i] = a < p.L && lane + 64 * i < p.R ? s * sc : 0.f;
  }
  store_parts<DT, 64, N>(v, lane, p.R, m, p.t, p.tf);
}

// Few rows: row blockIdx.x's products with eight ranks of its adapter, two to a wave, in float32, scaled;
// rows without an adapter are left out. p.tf: [M, R].
template <int DT>
__global__ __launch_bounds__(256) void k_lora_shrink_few(const ShrinkParams p) {
  const int m = blockIdx.x, lane = threadIdx.x & 63, r = blockIdx.y * 8 + (threadIdx.x >> 6) * 2;
  const int a = p.ids[m];
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
// JOIN (frags = 1): the first product's K ranges are joined here, every column tile's workgroup for itself, and the parts
// stay in LDS.
template <int DT, bool JOIN>
__global__ __launch_bounds__(256) void k_lora_expand(const Params p, int frags, const ShrinkParams sh, int ranges) {
  constexpr int PITCH = 2 * kMaxRank + 8;
  __shared__ __attribute__((aligned(16))) uint16_t ts[JOIN ? 16 * PITCH : 8];
  __shared__ float fs[16];
  __shared__ __attribute__((aligned(16))) uint8_t strips[4][16 * kStripPitch];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int col0 = blockIdx.y * 256 + (threadIdx.x >> 6) * 64;
  u32x4 b[4][2];  // the factor's rows of adapter `held`, ranks c0 .. c0 + 63
  int held = -1;
  auto load_b = [&](int a, int c0) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int k = c0 + 32 * ks + 8 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = col0 + i * 16 + c;
        b[i][ks] = u32x4{0, 0, 0, 0};
        if (k < p.R && col < p.N) b[i][ks] = *(const u32x4*)(p.b + ((int64_t)a * p.N + col) * p.R + k);
      }
    }
    held = a;
  };
  // what a fragment needs besides its products: adapters and places of its rows, and the addend's values
  int id = 0;
  int64_t orow = 0;
  uint2 old[4];
  auto load_row = [&](int r0) {
    const int row = min(r0 + c, p.M - 1);
    id = r0 + c < p.M ? p.sid[row] : p.L;
    orow = p.perm[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = col0 + i * 16 + 4 * g;
      old[i] = uint2{0, 0};
      if (p.add && p.vec && r0 + c < p.M && col + 4 <= p.N) old[i] = *(const uint2*)((const uint16_t*)p.add + orow * p.ld_add + col);
    }
  };
  if constexpr (JOIN) {
    load_row(blockIdx.x * 16);
    const uint64_t rows = __ballot(id < p.L);
    if (rows) load_b(__builtin_amdgcn_readlane(id, __builtin_ctzll(rows)), 0);
    // sixteen lanes to a row, four neighbouring ranks of 64 to a lane
    const int r = threadIdx.x >> 4, l4 = (threadIdx.x & 15) * 4, m = blockIdx.x * 16 + r;
    const int a = m < p.M ? p.sid[m] : p.L;
    const float sc = a < p.L ? sh.scales[a] : 0.f;
    f32x4 v[kMaxRank / 64];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxRank / 64; ++i) {
      v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (l4 + 64 * i >= p.R || m >= p.M) continue;
      // rows without an adapter hold zeros
      f32x4 x[kMaxRanges];
#pragma unroll
      for (int k = 0; k < kMaxRanges; ++k) x[k] = *(const f32x4*)(sh.part + ((size_t)min(k, ranges - 1) * p.M + m) * p.R + l4 + 64 * i);
#pragma unroll
      for (int k = 0; k < kMaxRanges; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i][q] = k < ranges ? v[i][q] + x[k][q] : v[i][q];
      v[i] *= sc;
#pragma unroll
      for (int q = 0; q < 4; ++q) most = fmaxf(most, fabsf(v[i][q]));
    }
#pragma unroll
    for (int d = 1; d < 16; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
    const int e = power_above(most);
    const float inv = ldexpf(1.f, -e);
    if (l4 == 0) fs[r] = ldexpf(1.f, e);
#pragma unroll
    for (int i = 0; i < kMaxRank / 64; ++i) {
      if (l4 + 64 * i >= p.R) continue;
      float h[4], l[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) two_parts<DT>(v[i][q] * inv, h[q], l[q]);
      *(uint2*)(ts + r * PITCH + l4 + 64 * i) = pack4<DT>(h);
      *(uint2*)(ts + r * PITCH + p.R + l4 + 64 * i) = pack4<DT>(l);
    }
    __syncthreads();
  }
  if (col0 >= p.N) return;
  for (int x = 0; x < frags; ++x) {
    const int r0 = (blockIdx.x * frags + x) * 16;
    if (r0 >= p.M) return;
    const int row = min(r0 + c, p.M - 1);
    if constexpr (!JOIN) load_row(r0);
    const float f = JOIN ? fs[c] : p.tf[row];
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
            hi[ks] = *(const u32x4*)(JOIN ? ts + c * PITCH + k : p.t + part_at(row, k, p.R));
            lo[ks] = *(const u32x4*)(JOIN ? ts + c * PITCH + p.R + k : p.t + part_at(row, p.R + k, p.R));
          }
        }
        if (held != a || p.R > 64) load_b(a, c0);
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
    if (!p.vec) {  // rows that begin anywhere: see move_rows
      uint8_t* strip = strips[threadIdx.x >> 6];
      const int left = p.N - col0, rows = p.M - r0;
      if (p.add) {
        wave_sync();
        move_rows<16, true>(strip, (uint16_t*)p.add + col0, p.ld_add, (int)orow, rows, left, p.pair, lane);
        wave_sync();
      }
      uint2 res[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
        const uint2 x = *(const uint2*)(strip + c * kStripPitch + (i * 16 + 4 * g) * 2);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = col0 + i * 16 + 4 * g + q;
          v[q] = acc[i][q] + (p.bias[0] ? p.bias[0][min(col, p.N - 1)] : 0.f);
          if (p.add) v[q] += load1<DT>(&x, q);
        }
        res[i] = pack4<DT>(v);
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < 4; ++i) *(uint2*)(strip + c * kStripPitch + (i * 16 + 4 * g) * 2) = res[i];
      wave_sync();
      move_rows<16, false>(strip, (uint16_t*)p.out[0] + col0, p.ldo[0], (int)orow, rows, left, p.pair, lane);
      continue;
    }
    if (r0 + c >= p.M) continue;
    uint16_t* out = (uint16_t*)p.out[0] + orow * p.ldo[0];
    const uint16_t* add = p.add ? (const uint16_t*)p.add + orow * p.ld_add : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = col0 + i * 16 + 4 * g;  // four neighbours
      if (col + 4 <= p.N) {
        uint2 res;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = acc[i][q] + (p.bias[0] ? p.bias[0][col + q] : 0.f);
        if (add) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += load1<DT>(&old[i], q);
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
