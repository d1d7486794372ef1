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

#include "dense16_rule.hpp"
#include "elem.hpp"

namespace moe {
namespace d16 {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) void lds_void;

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
  int32_t fold;            // DX: rows m and m + fold are one row's upper and lower parts; DW: K rows k and k + fold; 0: none
  int64_t lower;           // k_big's PARTS: elements from dg's and du's upper parts to their lower ones
  // LORA
  const void* add;
  int64_t ld_add;
  int32_t vec;             // out and add take 16-byte accesses at multiples of 8 columns
  int32_t pair;            // and else 4-byte ones at even columns
  int32_t N8;              // N rounded down to a multiple of 8
  int32_t R, L;
  const uint16_t* t;       // upper and lower parts of the scaled x A^T, rows in sorted order (part_at)
  const float* tf;         // [M] their rows' powers of two
  const uint16_t* b;       // [L, N, R]
  const uint16_t* a;       // k_few's first products: [L, R, K]
  const float* scales;     // and [L]
  const int32_t* perm;     // sorted row -> row
  const int32_t* sid;      // adapter of the sorted row, L where it has none
};

// Where value r < 2 R of sorted row m of t is (the upper parts of R ranks, then the lower ones): eight values of 32 rows
// side by side, so that the MFMA's operand of 32 rows is 1 KB in one piece (rows of 2 R values cost the 256-row tiles
// of 8192 x 2048 x 7168 with rank 64 37 us in place of 12: an instruction then asks for 32 lines).
__host__ __device__ __forceinline__ int64_t part_at(int m, int r, int R) {
  return (((int64_t)(m >> 5) * (R >> 2) + (r >> 3)) * 32 + (m & 31)) * 8 + (r & 7);
}

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

// 1 - tanh(x)^2 = 4 q / (1 + q)^2 with q = exp(-2 |x|): the difference would lose every digit where tanh nears 1 (half
// of float16's at |x| = 5), this is within a few roundings of it anywhere.
__device__ __forceinline__ float sech2(float x) {
  const float q = __expf(-2.f * fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + q);
  return 4.f * q * r * r;
}

// Its derivatives. Behind the clamps they are 0, on the limit itself the inner ones.
template <int AK>
__device__ __forceinline__ void act_df(const ActParams& a, float g, float u, float& fg, float& fu) {
  if constexpr (AK == 0) {
    const float s = sigm(g);
    fg = u * s * (1.f + g * sigm(-g));
    fu = g * s;
  } else if constexpr (AK == 2) {
    const float s = sigm(g), tg = tanhf(g / a.alpha);
    fg = s * (sech2(g / a.alpha) + a.alpha * tg * sigm(-g)) * (a.beta * tanhf(u / a.beta));
    fu = a.alpha * tg * s * sech2(u / a.beta);
  } else {
    const float gc = g > a.limit ? a.limit : g;
    const float uc = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
    const float s = sigm(a.alpha * gc);
    // beyond 128 the sigmoid or its complement is 0 in float32, which an infinite product would make NaN
    const float t = __builtin_amdgcn_fmed3f(a.alpha * gc, -128.f, 128.f);
    fg = g > a.limit ? 0.f : (uc + a.beta) * s * (1.f + t * sigm(-t));
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

// an address that is the same in all lanes, in scalar registers
__device__ __forceinline__ const uint8_t* uniform(const void* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const uint8_t*)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t desc(const uint8_t* at, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(at), (short)0, bytes, 0x00020000);
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

// Stores from a 32 x 32 result fragment (N operand first): the lane holds columns 8 q + 4 lk .. + 3 of row lr in registers
// 4 q .. 4 q + 3. 16-bit values of an even q and the odd one behind it change places between the
// halves of the wave, so that a lane stores eight neighbours: q's in the lower half, q + 1's in the upper.
template <int DT>
__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
  uint2 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) store1<DT>(&r, j, v[j]);
  return r;
}
__device__ __forceinline__ u32x4 swap_halves(uint2 even, uint2 odd) {
  const auto a = __builtin_amdgcn_permlane32_swap(even.x, odd.x, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(even.y, odd.y, false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}
// v[q][j]: 4 x 4 values of the lane; base: the row's first value of the fragment's columns; left: columns from there to the end,
// a multiple of 8
template <int DT>
__device__ __forceinline__ void store_fragment(void* base, const float (&v)[4][4], int lk, int left, bool row_ok) {
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    const u32x4 x = swap_halves(pack4<DT>(v[q]), pack4<DT>(v[q + 1]));
    if (row_ok && 8 * (q + lk) < left) *(u32x4*)((uint16_t*)base + 8 * (q + lk)) = x;
  }
}
__device__ __forceinline__ void store_fragment_f32(float* base, const float (&v)[4][4], int lk, int left, bool row_ok) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (row_ok && 8 * q + 4 * lk < left) *(f32x4*)(base + 8 * q + 4 * lk) = f32x4{v[q][0], v[q][1], v[q][2], v[q][3]};
}

// Rows of 64 columns from out or add into a strip of LDS (LOAD), or back, where these rows begin anywhere: a row's
// columns side by side over the lanes, two to a lane where rows begin at multiples of 4 bytes (pair). Lane r < ROWS holds in
// `row` the place of the strip's row r; `rows` and `left`: how many rows and columns there are.
constexpr int kStripPitch = 144;
template <int ROWS, bool LOAD>
__device__ __forceinline__ void move_rows(uint8_t* strip, uint16_t* base, int64_t ld, int row, int rows, int left, bool pair, int lane) {
  constexpr int U = 8;  // accesses at a time
  const int per = pair ? 2 : 1, c = pair ? 2 * (lane & 31) : lane, n = ROWS / per;
  const int r1 = pair ? lane >> 5 : 0;
  const bool two = pair && c + 1 < left;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += U) {
    uint32_t x[U];
    uint16_t* at[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = (i0 + i) * per + r1;
      at[i] = base + (int64_t)__shfl(row, r) * ld + c;
      x[i] = 0;
      if constexpr (!LOAD) x[i] = pair ? *(const uint32_t*)(strip + r * kStripPitch + 2 * c) : *(const uint16_t*)(strip + r * kStripPitch + 2 * c);
    }
    if (c < left) {
      if (two) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if ((i0 + i) * per + r1 < rows) {
            if constexpr (LOAD) x[i] = *(const uint32_t*)at[i];
            else *(uint32_t*)at[i] = x[i];
          }
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if ((i0 + i) * per + r1 < rows) {
            if constexpr (LOAD) x[i] = *at[i];
            else *at[i] = (uint16_t)x[i];
          }
      }
    }
    if constexpr (LOAD) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint8_t* to = strip + ((i0 + i) * per + r1) * kStripPitch + 2 * c;
        if (pair) *(uint32_t*)to = x[i];
        else *(uint16_t*)to = (uint16_t)x[i];
      }
    }
  }
}

// DW's 4 x 4 values of the lane at the output's row and the fragment's first column
template <int DT>
__device__ __forceinline__ void finish_dw(const Params& p, int z, int64_t row, int col, float (&v)[4][4], int lk, bool ok) {
  const int64_t at = row * p.ldo[z] + col;
  const int left = p.N - col;
  if (p.accumulate) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!ok || 8 * q + 4 * lk >= left) continue;
      if (p.f32_out) {
        const f32x4 x = *(const f32x4*)((const float*)p.out[z] + at + 8 * q + 4 * lk);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q][i] += x[i];
      } else {
        const uint2 x = *(const uint2*)((const uint16_t*)p.out[z] + at + 8 * q + 4 * lk);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q][i] += load1<DT>(&x, i);
      }
    }
  }
  if (p.f32_out) store_fragment_f32((float*)p.out[z] + at, v, lk, left, ok);
  else store_fragment<DT>((uint16_t*)p.out[z] + at, v, lk, left, ok);
}

// Partial results joined in the order of their K ranges, eight columns to a thread; DX: upper and lower parts of rows too.
template <int DT, int MODE>
__global__ __launch_bounds__(256) void k_join(const Params p) {
  const int cpr = (p.N + 7) / 8, z = blockIdx.y, rows = MODE == DX && p.fold ? p.fold : p.M;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)rows * cpr) return;
  const int row = (int)(i / cpr), col = (int)(i - (int64_t)row * cpr) * 8;
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
  // eight ranges' loads at a time, whatever their number (77 x 2880 in 8 ranges 6.9 -> 4.0 us against a loop unrolled by
  // four; 300 x 2048 gated in 5 and 1000 x 4096 in 2 stay at 5.7 and 7.7, 4.3 TB/s of partial results)
  constexpr int AT = 8;
  for (int s0 = 0; s0 < p.splits; s0 += AT) {
    float a[AT][8], b[MODE == GATED || MODE == DX ? AT : 1][8];
#pragma unroll
    for (int i = 0; i < AT; ++i) {
      const int s = min(s0 + i, p.splits - 1);
      load8<T_FP32>(part_of<MODE>(p, s, z, row, col), 0, a[i]);
      if constexpr (MODE == GATED) load8<T_FP32>(part_of<MODE>(p, s, 1, row, col), 0, b[i]);
      if constexpr (MODE == DX) {
        if (p.fold) load8<T_FP32>(part_of<MODE>(p, s, z, row + p.fold, col), 0, b[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < AT; ++i) {
      if (s0 + i >= p.splits) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] += a[i][j];
        if constexpr (MODE == GATED) u[j] += b[i][j];
        if constexpr (MODE == DX) {
          if (p.fold) v[j] += b[i][j];
        }
      }
    }
  }
  finish8<DT, MODE>(p, z, MODE == LORA ? p.perm[row] : row, col, v, u);
}

}  // namespace d16
}  // namespace moe
