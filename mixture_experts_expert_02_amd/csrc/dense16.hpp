// Dense products of 16-bit rows and weights on the MFMA: the gated feed-forward
// block, its backward pass and projections with low-rank adapters
// (moe_gated_linear, moe_gated_linear_backward, moe_lora_linear).
//
// moonep_experts page, module docstring (the gated block of one expert:
// gate and up projections, f(gate, up), here on all rows at once).
//
//   GATED  g = x Wg^T + bg, u = x Wu^T + bu, out = f(g, u)     K = H, both operands K-contiguous
//   DX     dx = dg Wg + du Wu                                   K = I twice, the weights K-major
//   DW     dWg = dg^T x, dWu = du^T x                           K = rows, both operands K-major
//   LORA   out = x W^T + bias + add + f_m (t_m B_a^T)           K = K, K-contiguous
//
// One output tile to a workgroup, 64 K values to a stage, both operands from
// memory straight into LDS. A K-contiguous operand keeps its rows there (128
// bytes of a row, 16-byte chunks XOR-swizzled) and is read by ds_read_b128; a
// K-major one keeps its K rows (64-byte pieces XOR-swizzled) and is read by
// ds_read_b64_tr_b16, which hands a lane four K values of its column, so nothing
// is transposed in memory first. What lies outside an operand reads as zero
// (bounds of the buffer descriptors), so K may end anywhere.
#pragma once

#include <type_traits>

#include "elem.hpp"

namespace moe {
namespace d16 {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) void lds_void;

enum Mode { GATED, DX, DW, LORA };

constexpr int BK = 64;                    // K values of a stage
constexpr uint32_t kNoLoad = 0x80000000u; // buffer offset past any operand: reads 0

// The M operand gives the output's rows, the N operand its columns.
struct Params {
  const uint16_t* m[2];    // DX: dg, du; DW: dg, du (by half); else x
  const uint16_t* n[2];    // GATED and DX: gate and up weights; else one
  void* out[2];            // DW: by half
  int64_t ldm[2], ldn[2], ldo[2];  // elements
  int32_t M, N, K;         // K of one product
  int32_t mt, nt;          // row and column tiles
  int32_t splits;          // K ranges, each with a partial result of its own (1 = none)
  float* part;             // partial results
  const float* bias[2];
  void* keep[2];           // GATED: g and u, or nullptr
  int64_t ld_keep[2];
  ActParams act;
  int32_t f32_out, accumulate;  // DW
  // LORA
  const void* add;
  int64_t ld_add;
  int32_t vec;             // out, add and bias take 16-byte accesses at multiples of 8 columns
  int32_t R, L;
  const uint16_t* t;       // [M, 2R] upper and lower parts of the scaled x A^T, rows in sorted order
  const float* tf;         // [M] their rows' powers of two
  const uint16_t* b;       // [L, N, R]
  const int32_t* perm;     // sorted row -> row
  const int32_t* sid;      // adapter of the sorted row, L where it has none
  const int32_t* ends;     // [L] sorted row behind an adapter's last
};

// ------------------------------------------------------------ activations
__device__ __forceinline__ float sigm(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// f(g, u) of common.hpp's ActParams; clamps let a NaN through.
template <int AK>
__device__ __forceinline__ float act_f(const ActParams& a, float g, float u) {
  if constexpr (AK == 0) return g * sigm(g) * u;
  if constexpr (AK == 2) return a.alpha * tanhf(g / a.alpha) * sigm(g) * (a.beta * tanhf(u / a.beta));
  g = g > a.limit ? a.limit : g;
  u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  return g * sigm(a.alpha * g) * (u + a.beta);
}

// Its derivatives. Behind the clamps they are 0, on the limit itself the inner ones.
template <int AK>
__device__ __forceinline__ void act_df(const ActParams& a, float g, float u, float& fg, float& fu) {
  if constexpr (AK == 0) {
    const float s = sigm(g);
    fg = u * s * (1.f + g * sigm(-g));
    fu = g * s;
  } else if constexpr (AK == 2) {
    const float s = sigm(g), tg = tanhf(g / a.alpha), tu = tanhf(u / a.beta);
    fg = s * (1.f - tg * tg + a.alpha * tg * sigm(-g)) * (a.beta * tu);
    fu = a.alpha * tg * s * (1.f - tu * tu);
  } else {
    const float gc = g > a.limit ? a.limit : g;
    const float uc = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
    const float s = sigm(a.alpha * gc);
    fg = g > a.limit ? 0.f : (uc + a.beta) * s * (1.f + a.alpha * gc * sigm(-a.alpha * gc));
    fu = u > a.limit || u < -a.limit ? 0.f : gc * s;
  }
}

template <class F>
__device__ __forceinline__ void with_act(const ActParams& a, F f) {
  if (a.kind == 0) f(std::integral_constant<int, 0>{});
  else if (a.kind == 1) f(std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 2>{});
}

// ------------------------------------------------------------ loads
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

// 16 bytes to a lane, straight into LDS from dst on
__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t rs, lds_u8* dst, uint32_t off, uint32_t uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)dst, 16, (int)off, (int)uniform, 0, 0);
}

// vmcnt(N), nothing else waited for
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// vmcnt(N) and every LDS access
template <int N>
__device__ __forceinline__ void wait_all_but() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void wave_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// K-contiguous block in LDS: chunk c (8 values) of row r sits in 16-byte slot
// 8 r + (c ^ ((r >> 1) & 7)): the 16 rows of one pass of an operand read fall on
// 16 different 16-byte banks of the 256-byte window.
__device__ __forceinline__ uint32_t row_slot(int r, int c) { return (uint32_t)(r * 8 + (c ^ ((r >> 1) & 7))); }

// K-major block of W columns: 64-byte piece p of K row k sits in piece p ^ major_xor(k)
// of its row, so that the four rows x 64 bytes of half a transposing read fall
// on different banks.
template <int W>
__device__ __forceinline__ int major_xor(int k) { return W == 64 ? (k >> 1) & 1 : k & 3; }

// Where lane `lane` of instruction `i` (1 KB) of such a block reads: K row and 16-byte chunk of the row.
template <int W>
__device__ __forceinline__ void major_src(int i, int lane, int& k, int& chunk) {
  constexpr int CPR = W / 8;  // chunks in a K row
  const int pos = i * 64 + lane;
  k = pos / CPR;
  const int d = pos % CPR;
  chunk = (((d >> 2) ^ major_xor<W>(k)) << 2) | (d & 3);
}

// One 32-value x 16-K operand of the MFMA: lane holds value lane & 31, K values 8 (lane >> 5)..+7.
template <bool MAJOR>
struct Frag {
  u32x4 v;
  __device__ __forceinline__ void read(uint32_t addr, uint32_t) { asm volatile("ds_read_b128 %0, %1" : "=v"(v) : "v"(addr)); }
  __device__ __forceinline__ void tie() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ u32x4 get() const { return v; }
};
template <>
struct Frag<true> {
  uint64_t a, b;
  // four K rows further on: `step` bytes
  __device__ __forceinline__ void read(uint32_t addr, uint32_t step) {
    asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(a) : "v"(addr));
    asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(b) : "v"(addr + step));
  }
  __device__ __forceinline__ void tie() {
    asm volatile("" : "+v"(a));
    asm volatile("" : "+v"(b));
  }
  __device__ __forceinline__ u32x4 get() const { return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)}; }
};

// The same with the offset in the instruction; K-major: rows of W columns.
template <bool MAJOR, int W>
struct BigFrag {
  u32x4 v;
  template <int AT>
  __device__ __forceinline__ void read(uint32_t addr) {
    asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(AT));
  }
  __device__ __forceinline__ void tie() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ u32x4 get() const { return v; }
};
template <int W>
struct BigFrag<true, W> {
  uint64_t a, b;
  template <int AT>
  __device__ __forceinline__ void read(uint32_t addr) {
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(a) : "v"(addr), "n"(AT));
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(b) : "v"(addr), "n"(AT + 8 * W));
  }
  __device__ __forceinline__ void tie() {
    asm volatile("" : "+v"(a));
    asm volatile("" : "+v"(b));
  }
  __device__ __forceinline__ u32x4 get() const {
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
  }
};

template <int DT>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == T_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Work item of this workgroup. Workgroup b runs on XCD b mod 8; each XCD takes a
// contiguous run of items, numbered in groups of 4 row tiles, row tile
// fastest, so that the tiles an XCD has in flight share operand panels in its L2.
struct Item { int mt, nt, z; };
__device__ __forceinline__ bool item_of(const Params& p, int nz, Item& it) {
  const int n = p.mt * p.nt * nz, per = (n + 7) >> 3;
  const int j = blockIdx.x >> 3;
  const int x = (blockIdx.x & 7) * per + j;
  if (j >= per || x >= n) return false;
  const int tiles = p.mt * p.nt;
  it.z = x / tiles;
  const int y = x - it.z * tiles;
  const int span = 4 * p.nt, grp = y / span, in = y - grp * span;
  const int rows = min(4, p.mt - 4 * grp);
  it.nt = in / rows;
  it.mt = 4 * grp + in % rows;
  return true;
}

template <int DT>
__device__ __forceinline__ float load1(const void* base, size_t i) {
  if constexpr (DT == T_BF16) return (float)((const __bf16*)base)[i];
  else return (float)((const _Float16*)base)[i];
}
template <int DT>
__device__ __forceinline__ void store1(void* base, size_t i, float v) {
  if constexpr (DT == T_BF16) ((__bf16*)base)[i] = (__bf16)v;
  else ((_Float16*)base)[i] = (_Float16)v;
}

// ------------------------------------------------------------ epilogue
// Eight neighbouring results of one output row (GATED: of both projections) get their bias, addend or
// activation, are rounded once and stored. row: LORA's in the output's order, not the sorted one.
template <int DT, int MODE>
__device__ __forceinline__ void finish8(const Params& p, int z, int64_t row, int col, float (&v)[8], float (&u)[8]) {
  if constexpr (MODE == GATED) {
    if (p.bias[0]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] += p.bias[0][col + j];
        u[j] += p.bias[1][col + j];
      }
    }
    if (p.keep[0]) {
      store8<DT>(p.keep[0], (size_t)(row * p.ld_keep[0] + col), v);
      store8<DT>(p.keep[1], (size_t)(row * p.ld_keep[1] + col), u);
    }
    with_act(p.act, [&](auto k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_f<decltype(k)::value>(p.act, v[j], u[j]);
    });
    store8<DT>(p.out[0], (size_t)(row * p.ldo[0] + col), v);
  } else if constexpr (MODE == DX) {
    store8<DT>(p.out[0], (size_t)(row * p.ldo[0] + col), v);
  } else if constexpr (MODE == DW) {
    const size_t at = (size_t)(row * p.ldo[z] + col);
    if (p.accumulate) {
      float old[8];
      if (p.f32_out) load8<T_FP32>(p.out[z], at, old);
      else load8<DT>(p.out[z], at, old);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    if (p.f32_out) store8<T_FP32>(p.out[z], at, v);
    else store8<DT>(p.out[z], at, v);
  } else {
    uint16_t* out = (uint16_t*)p.out[0] + row * p.ldo[0] + col;
    const uint16_t* add = p.add ? (const uint16_t*)p.add + row * p.ld_add + col : nullptr;
    if (p.vec && col + 8 <= p.N) {
      if (p.bias[0]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p.bias[0][col + j];
      }
      if (add) {
        float old[8];
        load8<DT>(add, 0, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += old[j];
      }
      store8<DT>(out, 0, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (col + j >= p.N) break;
        float s = v[j];
        if (p.bias[0]) s += p.bias[0][col + j];
        if (add) s += load1<DT>(add, j);
        store1<DT>(out, j, s);
      }
    }
  }
}

// Partial results: [K range][GATED: g, u; DW: half][row][columns rounded up to 8]
template <int MODE>
__device__ __forceinline__ float* part_of(const Params& p, int split, int which, int64_t row, int col) {
  const int64_t np = (p.N + 7) & ~7;
  const int planes = MODE == GATED || MODE == DW ? 2 : 1;
  return p.part + ((int64_t)(planes * split + which) * p.M + row) * np + col;
}

// A wave's results of 32 rows, staged in LDS as float32 (rows of COLS + 4 values),
// come back eight columns to a lane and leave as 16-byte stores.
template <int DT, int MODE, int COLS>
__device__ __forceinline__ void store_rows(const Params& p, const float* strip, int z, int split, int row0, int col0,
                                           int lane, const int* rows_lds) {
  constexpr int HALF = MODE == GATED ? COLS / 2 : COLS;  // output columns
  constexpr int PITCH = COLS + 4;
  constexpr int CPR = HALF / 8, RPP = 64 / CPR;
  const int c = 8 * (lane % CPR), col = col0 + c;
  if (col >= p.N) return;
#pragma unroll 1
  for (int r = lane / CPR; r < 32; r += RPP) {
    const int row = row0 + r;
    if (row >= p.M) return;
    float v[8], u[8];
    load8<T_FP32>(strip, r * PITCH + c, v);
    if constexpr (MODE == GATED) load8<T_FP32>(strip, r * PITCH + HALF + c, u);
    if (p.splits > 1) {
      store8<T_FP32>(part_of<MODE>(p, split, z, row, col), 0, v);
      if constexpr (MODE == GATED) store8<T_FP32>(part_of<MODE>(p, split, 1, row, col), 0, u);
    } else {
      finish8<DT, MODE>(p, z, MODE == LORA ? rows_lds[r] : row, col, v, u);
    }
  }
}

// Partial results joined in the order of their K ranges, eight columns to a thread.
template <int DT, int MODE>
__global__ __launch_bounds__(256) void k_join(const Params p) {
  const int cpr = (p.N + 7) / 8, z = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * cpr) return;
  const int row = (int)(i / cpr), col = (int)(i - (int64_t)row * cpr) * 8;
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    float a[8];
    load8<T_FP32>(part_of<MODE>(p, s, z, row, col), 0, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += a[j];
    if constexpr (MODE == GATED) {
      load8<T_FP32>(part_of<MODE>(p, s, 1, row, col), 0, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += a[j];
    }
  }
  finish8<DT, MODE>(p, z, MODE == LORA ? p.perm[row] : row, col, v, u);
}

// ------------------------------------------------------------ tiles by four waves
// BM x BN output tile (GATED: BN / 2 gate and the same up columns), waves 2 x 2.
// NBUF stages in LDS: NBUF - 1 of them loading while one is multiplied.
template <int DT, int MODE, int BM, int BN, int NBUF>
__global__ __launch_bounds__(256) void k_tile(const Params p) {
  constexpr bool MM = MODE == DW, NM = MODE == DX || MODE == DW;  // K-major operands
  constexpr int FM = BM / 64, FN = BN / 64;                        // 32-wide fragments of a wave
  constexpr int M_BYTES = BM * 128, STAGE = (BM + BN) * 128;
  constexpr int LM = BM / 32, LN = BN / 32, LT = LM + LN;          // load instructions of a wave and stage
  constexpr int COLS = FN * 32;
  static_assert(4 * 32 * (COLS + 4) * 4 <= NBUF * STAGE, "epilogue strips");
  __shared__ __attribute__((aligned(16))) uint8_t smem_arr[NBUF * STAGE];
  __shared__ int rows_lds[MODE == LORA ? BM : 1];
  lds_u8* smem = (lds_u8*)smem_arr;
  Item it;
  if (!item_of(p, MODE == DW ? 2 * p.splits : p.splits, it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, lr = lane & 31, lk = lane >> 5;
  constexpr int TN = MODE == GATED ? BN / 2 : BN;  // output columns of the tile
  const int m0 = it.mt * BM, n0 = it.nt * TN;
  const int z = MODE == DW ? it.z & 1 : 0, split = MODE == DW ? it.z >> 1 : it.z;

  // stages of this workgroup's K range
  const int kt = (p.K + BK - 1) / BK, all = MODE == DX ? 2 * kt : kt;
  const int s_lo = (int)((int64_t)split * all / p.splits), nst = (int)((int64_t)(split + 1) * all / p.splits) - s_lo;

  if constexpr (MODE == LORA) {
    for (int r = tid; r < BM; r += 256) rows_lds[r] = m0 + r < p.M ? p.perm[m0 + r] : 0;
    __syncthreads();
  }

  // ---- loads of one stage
  uint32_t m_row[LM];
  int m_chunk[LM], n_rowi[LN], n_chunk[LN];
#pragma unroll
  for (int q = 0; q < LM; ++q) {
    const int i = wave * LM + q;
    if constexpr (MM) {
      int k;
      major_src<BM>(i, lane, k, m_chunk[q]);
      m_row[q] = (uint32_t)k;
    } else {
      const int r = i * 8 + (lane >> 3);
      m_chunk[q] = (lane & 7) ^ ((r >> 1) & 7);
      m_row[q] = (uint32_t)r;
      if constexpr (MODE == LORA) m_row[q] = m0 + r < p.M ? (uint32_t)rows_lds[r] : 0xffffffffu;
    }
  }
#pragma unroll
  for (int q = 0; q < LN; ++q) {
    const int i = wave * LN + q;
    if constexpr (NM) {
      major_src<BN>(i, lane, n_rowi[q], n_chunk[q]);
    } else {
      const int r = i * 8 + (lane >> 3);
      n_chunk[q] = (lane & 7) ^ ((r >> 1) & 7);
      n_rowi[q] = MODE == GATED ? r % TN : r;
    }
  }
  auto load = [&](int st, int buf) {
    const bool live = st < nst;
    int s = s_lo + st, seg = 0;
    if (MODE == DX && s >= kt) {
      seg = 1;
      s -= kt;
    }
    const int k0 = s * BK;
    lds_u8* dst = smem + buf * STAGE;
    {
      const int mi = MODE == DX ? seg : MODE == DW ? z : 0;
      const int64_t ld = p.ldm[mi];
      if constexpr (MM) {
        const auto rs = rsrc(p.m[mi] + (int64_t)k0 * ld + m0, live ? ((min(BK, p.K - k0) - 1) * ld + p.M - m0) * 2 : 0);
#pragma unroll
        for (int q = 0; q < LM; ++q)
          dma(rs, dst + (wave * LM + q) * 1024, m_row[q] * (uint32_t)(ld * 2) + m_chunk[q] * 16, 0);
      } else {
        const int64_t base = MODE == LORA ? 0 : (int64_t)m0 * ld;
        const int64_t rows = MODE == LORA ? (int64_t)1 << 30 : min(BM, p.M - m0);
        const auto rs = rsrc(p.m[mi] + base, live ? ((rows - 1) * ld + p.K) * 2 : 0);
#pragma unroll
        for (int q = 0; q < LM; ++q) {
          uint32_t off = m_row[q] * (uint32_t)(ld * 2) + m_chunk[q] * 16;
          if (k0 + m_chunk[q] * 8 >= p.K || (MODE == LORA && m_row[q] == 0xffffffffu)) off = kNoLoad;
          dma(rs, dst + (wave * LM + q) * 1024, off, k0 * 2);
        }
      }
    }
    dst += M_BYTES;
    if constexpr (NM) {
      const int64_t ld = p.ldn[seg];
      const auto rs = rsrc(p.n[seg] + (int64_t)k0 * ld + n0, live ? ((min(BK, p.K - k0) - 1) * ld + p.N - n0) * 2 : 0);
#pragma unroll
      for (int q = 0; q < LN; ++q)
        dma(rs, dst + (wave * LN + q) * 1024, n_rowi[q] * (uint32_t)(ld * 2) + n_chunk[q] * 16, 0);
    } else {
      // GATED: waves 0 and 1 load gate rows, 2 and 3 up rows
      const int ni = MODE == GATED ? wave >> 1 : 0;
      const int64_t ld = p.ldn[ni];
      const auto rs = rsrc(p.n[ni] + (int64_t)n0 * ld, live ? ((min(TN, p.N - n0) - 1) * ld + p.K) * 2 : 0);
#pragma unroll
      for (int q = 0; q < LN; ++q) {
        uint32_t off = n_rowi[q] * (uint32_t)(ld * 2) + n_chunk[q] * 16;
        if (k0 + n_chunk[q] * 8 >= p.K) off = kNoLoad;
        dma(rs, dst + (wave * LN + q) * 1024, off, k0 * 2);
      }
    }
  };

  // ---- operand reads: bytes inside a stage
  auto m_col = [&](int j) { return wm * (BM / 2) + j * 32; };
  auto n_col = [&](int i) { return MODE == GATED ? (i < FN / 2 ? 0 : TN) + wn * (TN / 2) + (i % (FN / 2)) * 32 : wn * (BN / 2) + i * 32; };
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const int tr = (lane >> 2) & 3;  // K row of a transposing read
  auto major_at = [&](auto w, int col, int ks) {
    constexpr int W = decltype(w)::value;
    const int k = 16 * ks + 8 * lk + tr, cb = 2 * (col + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
    return (uint32_t)(k * 2 * W + (((cb >> 6) ^ major_xor<W>(k)) << 6) + (cb & 63));
  };
  auto m_at = [&](int j, int ks) {
    if constexpr (MM) return major_at(std::integral_constant<int, BM>{}, m_col(j), ks);
    else return 16 * row_slot(m_col(j) + lr, 2 * ks + lk);
  };
  auto n_at = [&](int i, int ks) {
    if constexpr (NM) return major_at(std::integral_constant<int, BN>{}, n_col(i), ks);
    else return 16 * row_slot(n_col(i) + lr, 2 * ks + lk);
  };

  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  Frag<MM> fm[2][FM];
  Frag<NM> fn[2][FN];
  auto read = [&](uint32_t at, int ks, int set) {
#pragma unroll
    for (int j = 0; j < FM; ++j) fm[set][j].read(at + m_at(j, ks), 4 * 2 * BM);
#pragma unroll
    for (int i = 0; i < FN; ++i) fn[set][i].read(at + M_BYTES + n_at(i, ks), 4 * 2 * BN);
  };
  auto landed = [&](int set) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int j = 0; j < FM; ++j) fm[set][j].tie();
#pragma unroll
    for (int i = 0; i < FN; ++i) fn[set][i].tie();
  };

  // ---- adapters of this tile's rows, one after the other. Rows are sorted by adapter; a
  // fragment that holds rows of several gets each one's product in registers
  // of its own and adds it to the rows it belongs to, so that what an adapter
  // holds (an infinity, say) reaches no other adapter's rows.
  if constexpr (MODE == LORA) {
    if (split == 0) {
      int id[FM];
      float f[FM];
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int row = m0 + m_col(j) + lr;
        id[j] = row < p.M ? p.sid[row] : p.L;
        f[j] = row < p.M ? p.tf[row] : 0.f;
      }
      const int rc = p.R / 8, last = min(m0 + BM, p.M), rst = (2 * rc + 7) / 8;
      const auto rs_t = rsrc(p.t + (int64_t)m0 * 2 * p.R, (int64_t)(last - m0) * 4 * p.R);
      int pos = m0;
      while (pos < last) {
        const int a = __builtin_amdgcn_readfirstlane(p.sid[pos]);
        if (a >= p.L) break;
        pos = max(pos + 1, __builtin_amdgcn_readfirstlane(p.ends[a]));
        const auto rs_b = rsrc(p.b + ((int64_t)a * p.N + n0) * p.R, (int64_t)min(BN, p.N - n0) * 2 * p.R);
        for (int st0 = 0; st0 < rst; st0 += NBUF) {
          const int some = min(NBUF, rst - st0);
          for (int x = 0; x < some; ++x) {
            lds_u8* dst = smem + x * STAGE;
#pragma unroll
            for (int q = 0; q < LM; ++q) {
              const int r = (wave * LM + q) * 8 + (lane >> 3), v = (st0 + x) * 8 + m_chunk[q];
              dma(rs_t, dst + (wave * LM + q) * 1024, v < 2 * rc ? (uint32_t)(r * 4 * p.R + v * 16) : kNoLoad, 0);
            }
#pragma unroll
            for (int q = 0; q < LN; ++q) {
              const int v = (st0 + x) * 8 + n_chunk[q];
              dma(rs_b, dst + M_BYTES + (wave * LN + q) * 1024, v < 2 * rc ? (uint32_t)(n_rowi[q] * 2 * p.R + (v < rc ? v : v - rc) * 16) : kNoLoad, 0);
            }
          }
          wait_loads<0>();
          barrier();
          for (int x = 0; x < some; ++x) {
            f32x16 tmp[FN][FM];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              read(lds0 + x * STAGE, ks, 0);
              landed(0);
#pragma unroll
              for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                  if (ks == 0) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) tmp[i][j][r] = 0.f;
                  }
                  tmp[i][j] = mfma<DT>(fn[0][i].get(), fm[0][j].get(), tmp[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j)
              if (id[j] == a) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                  for (int r = 0; r < 16; ++r) acc[i][j][r] += tmp[i][j][r] * f[j];
              }
          }
          barrier();  // the buffers are free
        }
      }
    }
  }

  // ---- main loop
  if (nst > 0) {
#pragma unroll
    for (int s = 0; s < NBUF - 1; ++s) load(s, s);
    int buf = 0;
    for (int s = 0; s < nst; ++s) {
      wait_loads<(NBUF - 2) * LT>();
      barrier();  // stage s is there for all, and all have read stage s - 1
      load(s + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
      const uint32_t at = lds0 + buf * STAGE;
      read(at, 0, 0);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        landed(ks & 1);
        if (ks < 3) read(at, ks + 1, (ks + 1) & 1);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) acc[i][j] = mfma<DT>(fn[ks & 1][i].get(), fm[ks & 1][j].get(), acc[i][j]);
      }
      buf = buf + 1 == NBUF ? 0 : buf + 1;
    }
    wait_loads<0>();
    barrier();
  }

  float* strip = (float*)(smem_arr + wave * 32 * (COLS + 4) * 4);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(strip + lr * (COLS + 4) + i * 32 + 8 * q + 4 * lk) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wave_sync();
    store_rows<DT, MODE, COLS>(p, strip, z, split, m0 + m_col(j), n0 + (MODE == GATED ? wn * (TN / 2) : wn * (BN / 2)), lane,
                               rows_lds + (MODE == LORA ? m_col(j) : 0));
    wave_sync();
  }
}

}  // namespace d16
}  // namespace moe
