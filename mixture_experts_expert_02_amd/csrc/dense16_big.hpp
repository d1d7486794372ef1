// Tiles of 256 x 256 or 128 x 256 outputs by eight waves (GATED: 128 gate and the same 128 up columns).
//
// A stage of 64 K values is four half operands: M0, M1 (the two halves of the rows, 16 KB each, or 8 with 128 rows) and N0, N1 (16 KB). Wave
// (wm, wn) of 2 x 4 owns a half of each M half's rows and 32 columns of each N half, and the two waves of a SIMD (wm = 0 and 1)
// work half a phase apart: while one multiplies, the other reads the operands of its own next products from LDS and starts loads;
// a barrier ends each turn, two a phase.
//   256 rows: a stage is four phases of 64 x 32 x 64 products, eight MFMAs a wave: M0 N0, M0 N1, M1 N1, M1 N0, each behind the reads of
//   the half that is new to it (four or eight fragments; the next stage's N0 in the last one). Two buffers of 64 KB: a phase loads the half whose
//   buffer the phase before has read for the last time, for the stage after the next, so every half has six phases to arrive
//   (3000 cycles at the MFMA rate), and a wave waits for all loads but its twelve youngest.
//   128 rows: a stage is two phases, all four blocks of two K steps each; three buffers of 48 KB, each loaded anew in the two phases behind its
//   last read.
#pragma once

#include "dense16.hpp"

namespace moe {
namespace d16 {

// PARTS (DX and DW): dg and du are two parts each, and every part is a product of its own over the same K values, its upper
// part's before its lower one's.
template <int DT, int MODE, int BM, bool PARTS>
__global__ __launch_bounds__(512) void k_big(const Params p) {
  constexpr bool MM = MODE == DW, NM = MODE == DX || MODE == DW;  // K-major operands
  static_assert(NM || !PARTS, "gradients only");
  constexpr int SEGS = (MODE == DX ? 2 : 1) * (PARTS ? 2 : 1);  // products added, one after the other
  constexpr int HM = BM / 2, J = BM / 128, NB = BM == 256 ? 2 : 3;  // rows of an M half, a wave's 32-row fragments of it, buffers
  constexpr int TN = MODE == GATED ? 128 : 256, HALF = 16384, HALF_M = HM * 128;
  constexpr int N_AT = NB * 2 * HALF_M;  // M halves [stage buffer][half], then N halves
  constexpr int LM = BM / 128, LN = 2, LS = 2 * (LM + LN);  // a wave's load instructions for a half, and for a stage
  __shared__ __attribute__((aligned(16))) uint8_t smem_arr[NB * 2 * (HALF_M + HALF)];
  lds_u8* smem = (lds_u8*)smem_arr;
  Item it;
  if (!item_of(p, MODE == DW ? 2 * p.splits : p.splits, it)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lk = lane >> 5;
  const int m0 = it.mt * BM, n0 = it.nt * TN;
  const int z = MODE == DW ? it.z & 1 : 0, split = MODE == DW ? it.z >> 1 : it.z;
  const int kt = (p.K + BK - 1) / BK, all = SEGS * kt;
  const int s_lo = (int)((int64_t)split * all / p.splits), nst = (int)((int64_t)(split + 1) * all / p.splits) - s_lo;

  // ---- loads: instructions 2 wave and 2 wave + 1 of the 16 of a half (BM = 128: instruction `wave` of the 8 of an M half)
  // columns of N half h: 128 h + i where N is K-major or GATED (half = gate or up); else 32 columns of each half
  // side by side, 64 (i / 32) + 32 h + i % 32, so that a wave's columns are 64 neighbours
  int m_row[LM], m_chunk[LM], n_row[2], n_chunk[2];
  uint32_t g_off[2][LM];  // LORA: rows of x are gathered
  int g_row[2][LM];
#pragma unroll
  for (int q = 0; q < LM; ++q) {
    const int i = LM * wave + q, r = i * 8 + (lane >> 3);
    if constexpr (MM) major_src<HM>(i, lane, m_row[q], m_chunk[q]);
    else {
      m_row[q] = r;
      m_chunk[q] = (lane & 7) ^ ((r >> 1) & 7);
    }
    if constexpr (MODE == LORA) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
      {
        const bool in = m0 + h * HM + r < p.M;
        g_row[h][q] = in ? p.perm[m0 + h * HM + r] : -1;
        g_off[h][q] = in ? (uint32_t)g_row[h][q] * (uint32_t)(p.ldm[0] * 2) + m_chunk[q] * 16 : kNoLoad;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = 2 * wave + q, r = i * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    if constexpr (NM) major_src<128>(i, lane, n_row[q], n_chunk[q]);
    else {
      n_row[q] = MODE == GATED ? r : (r >> 5) * 64 + (r & 31);
      n_chunk[q] = c;
    }
  }
  // Where each half's next stage begins, at the operand's row k (K-major) or at its first row; the operands change from
  // product to product (DX: the gate's, then the up one). All of it in scalar registers and in 32 bits where they suffice, for a
  // wave's turn beside the other's 256 cycles of MFMAs is short (among the MFMAs the same instructions cost more:
  // a stage 1.30 us in place of 1.10 for DX, 0.97 in place of 0.91 for GATED).
  struct Cursor {
    const uint8_t* at;
    int k, end;     // next K value, and the end of this workgroup's in the operand: beyond it nothing is loaded
    uint32_t ld2;   // bytes between rows
    int bytes;      // K-contiguous: of the half; K-major: of a row from its first column on
  };
  const int seg0 = SEGS > 2 ? s_lo / kt : SEGS > 1 && s_lo >= kt ? 1 : 0;
  const int second = SEGS == 2 && !seg0 ? kt - s_lo : 0x7fffffff;  // the first stage of the second of two products
  auto first_k = [&](int seg) { return seg == seg0 ? (s_lo - seg * kt) * BK : 0; };
  auto end_k = [&](int seg) { return __builtin_amdgcn_readfirstlane(min(p.K, (s_lo + nst - seg * kt) * BK)); };
  auto m_cursor = [&](int h, int seg) {
    const int i = MODE == DX ? PARTS ? seg >> 1 : seg : z, k = first_k(seg);
    const int64_t ld = p.ldm[i], part = PARTS ? (seg & 1) * p.lower : 0;
    const int64_t at = MODE == LORA ? 0 : (MM ? k * ld + m0 + h * HM : (m0 + h * HM) * ld) + part;
    const int rows = min(HM, p.M - m0 - h * HM);
    const int bytes = MM ? (p.M - m0 - h * HM) * 2 : MODE == LORA ? 0x7fffffff : rows > 0 ? (rows - 1) * (int)ld * 2 + p.K * 2 : 0;
    return Cursor{uniform(p.m[i] + at), k, end_k(seg), (uint32_t)__builtin_amdgcn_readfirstlane((int)ld * 2),
                  __builtin_amdgcn_readfirstlane(bytes)};
  };
  auto n_cursor = [&](int h, int seg) {
    const int i = MODE == GATED ? h : MODE == DX ? PARTS ? seg >> 1 : seg : 0, k = first_k(seg);
    const int64_t ld = p.ldn[i], at = NM ? k * ld + n0 + h * 128 : (n0 + (MODE == GATED ? 0 : h * 32)) * ld;
    const int rows = min(MODE == GATED ? 128 : 224, p.N - n0 - (MODE == GATED ? 0 : h * 32));
    const int bytes = NM ? (p.N - n0 - h * 128) * 2 : rows > 0 ? (rows - 1) * (int)ld * 2 + p.K * 2 : 0;
    return Cursor{uniform(p.n[i] + at), k, end_k(seg), (uint32_t)__builtin_amdgcn_readfirstlane((int)ld * 2),
                  __builtin_amdgcn_readfirstlane(bytes)};
  };
  Cursor cm[2] = {m_cursor(0, seg0), m_cursor(1, seg0)};
  Cursor cn[2] = {n_cursor(0, seg0), n_cursor(1, seg0)};
  // the next stage's part of a half into LDS from dst on; `major`: the operand is K-major
  auto load = [&](auto major, auto count, Cursor& c, const int (&row)[decltype(count)::value], const int (&chunk)[decltype(count)::value],
                  const uint32_t* gathered, lds_u8* dst) {
    constexpr int L = decltype(count)::value;
    if constexpr (decltype(major)::value) {
      // a row's bytes are at most those between rows, so without rows this is not positive
      const auto rs = desc(c.at, max(0, (min(BK, c.end - c.k) - 1) * (int)c.ld2 + c.bytes));
#pragma unroll
      for (int q = 0; q < L; ++q) dma(rs, dst + q * 1024, __umul24(row[q], c.ld2) + chunk[q] * 16, 0);
      c.at += c.ld2 * BK;
    } else {
      const auto rs = desc(c.at, c.bytes);
#pragma unroll
      for (int q = 0; q < L; ++q) {
        uint32_t off = gathered ? gathered[q] : __umul24(row[q], c.ld2) + chunk[q] * 16;
        if (chunk[q] * 8 >= c.end - c.k) off = kNoLoad;
        dma(rs, dst + q * 1024, off, c.k * 2);
      }
    }
    c.k += BK;
  };
  // with more than two products: which one a half is in, and the stage at which its next one begins (none behind the last)
  int in_m[2] = {seg0, seg0}, in_n[2] = {seg0, seg0};
  auto next_of = [&](int seg) { return seg + 1 < SEGS ? (seg + 1) * kt - s_lo : 0x7fffffff; };
  auto load_m = [&](int h, int st, int buf) {
    if constexpr (SEGS == 2) {
      if (st == second) cm[h] = m_cursor(h, 1);
    } else if constexpr (SEGS > 2) {
      if (st == next_of(in_m[h])) cm[h] = m_cursor(h, ++in_m[h]);
    }
    load(std::bool_constant<MM>{}, std::integral_constant<int, LM>{}, cm[h], m_row, m_chunk, MODE == LORA ? g_off[h] : nullptr,
         smem + (buf * 2 + h) * HALF_M + wave * LM * 1024);
  };
  auto load_n = [&](int h, int st, int buf) {
    if constexpr (SEGS == 2) {
      if (st == second) cn[h] = n_cursor(h, 1);
    } else if constexpr (SEGS > 2) {
      if (st == next_of(in_n[h])) cn[h] = n_cursor(h, ++in_n[h]);
    }
    load(std::bool_constant<NM>{}, std::integral_constant<int, 2>{}, cn[h], n_row, n_chunk, nullptr,
         smem + N_AT + (buf * 2 + h) * HALF + wave * 2048);
  };

  // LORA: the addend's lines of this tile are asked for a few stages before the end, by loads whose values nobody
  // reads, so that the epilogue, in which all workgroups of a round meet, finds them nearer than memory.
  __shared__ __attribute__((aligned(16))) uint8_t unread[MODE == LORA ? 256 : 16];
  auto touch_addend = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < LM; ++q) {
        const int c = n0 + (lane & 7) * 64;
        if (g_row[h][q] >= 0 && (lane & 7) < 4 && c < p.N8)
          __builtin_amdgcn_global_load_lds((const uint16_t*)p.add + (int64_t)g_row[h][q] * p.ld_add + c, (lds_void*)(lds_u8*)unread, 4, 0, 0);
      }
  };
  const bool touch = MODE == LORA && p.add && p.vec && p.splits == 1;
  const int touch_at = max(0, (nst - 8) & ~1);

  // ---- operand reads: bytes inside a half
  const int tr = (lane >> 2) & 3;
  auto major_at = [&](int col, bool narrow) {  // rows of 128 columns, or of 64
    const int cb = 2 * (col + 16 * ((lane >> 4) & 1) + 4 * (lane & 3)), k = 8 * lk + tr;
    return (uint32_t)(k * (narrow ? 128 : 256) + (((cb >> 6) ^ (narrow ? tr >> 1 : tr)) << 6) + (cb & 63));
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  // K-major: by fragment; else by K step. An instruction's offset reaches 64 KB: the third buffer's N halves have addresses of their own.
  uint32_t m_at[MM ? J : 4], n_at[NB == 3 ? 2 : 1][NM ? 1 : 4];
  if constexpr (MM) {
#pragma unroll
    for (int j = 0; j < J; ++j) m_at[j] = lds0 + major_at(wm * (HM / 2) + j * 32, HM == 64);
  } else {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) m_at[ks] = lds0 + 16 * row_slot(wm * (HM / 2) + lr, 2 * ks + lk);
  }
#pragma unroll
  for (int b = 0; b < (NB == 3 ? 2 : 1); ++b) {
    if constexpr (NM) {
      n_at[b][0] = lds0 + N_AT + b * 4 * HALF + major_at(wn * 32, false);
    } else {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) n_at[b][ks] = lds0 + N_AT + b * 4 * HALF + 16 * row_slot(wn * 32 + lr, 2 * ks + lk);
    }
  }

  f32x16 acc[2][2][J];  // [N half][M half][32 rows]
  auto clear = [&](int hm, int j) {
#pragma unroll
    for (int hn = 0; hn < 2; ++hn)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[hn][hm][j][r] = 0.f;
  };

  BigFrag<MM, HM> fm[J][4];   // 256 rows: an M half's [32 rows][K step]
  BigFrag<NM, 128> fn[3][4];  // and N halves' [set][K step]
  BigFrag<MM, HM> gm[2][2];   // 128 rows: [M half][K step of a pair]
  BigFrag<NM, 128> gn[2][2];  // and [N half][K step]

  // fragment x (0..7) of an M half, (0..3) of an N half
#define MOE_D16_READ_M(h, buf, x)                                                                             \
  {                                                                                                           \
    constexpr int j_ = (x) % J, k_ = (x) / J;                                                                 \
    if constexpr (MM) fm[j_][k_].template read<((buf) * 2 + (h)) * HALF_M + k_ * 32 * HM>(m_at[j_]);          \
    else fm[j_][k_].template read<((buf) * 2 + (h)) * HALF_M + j_ * 4096>(m_at[k_]);                         \
  }
#define MOE_D16_READ_N(set, h, buf, x)                                                                        \
  {                                                                                                           \
    if constexpr (NM) fn[set][x].template read<((buf) * 2 + (h)) * HALF + (x) * 4096>(n_at[0][0]);            \
    else fn[set][x].template read<((buf) * 2 + (h)) * HALF>(n_at[0][x]);                                      \
  }
#define MOE_D16_ALL_M(h, buf)                                                                                 \
  MOE_D16_READ_M(h, buf, 0) MOE_D16_READ_M(h, buf, 1) MOE_D16_READ_M(h, buf, 2) MOE_D16_READ_M(h, buf, 3)     \
  MOE_D16_READ_M(h, buf, 4) MOE_D16_READ_M(h, buf, 5) MOE_D16_READ_M(h, buf, 6) MOE_D16_READ_M(h, buf, 7)
#define MOE_D16_ALL_N(set, h, buf) \
  MOE_D16_READ_N(set, h, buf, 0) MOE_D16_READ_N(set, h, buf, 1) MOE_D16_READ_N(set, h, buf, 2) MOE_D16_READ_N(set, h, buf, 3)
  auto tie_m = [&]() {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) fm[j][ks].tie();
  };
  auto tie_n = [&](int set) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) fn[set][ks].tie();
  };

  // ---- adapters, a fragment of 32 sorted rows at a time, while the first stages load: both operands straight
  // into registers (t and the factor's rows are as the MFMA wants them), t of all the wave's fragments at once, in the
  // registers that their results take over. A fragment that holds rows of several adapters gets each one's product in
  // registers of its own and adds it to the rows it belongs to, so that what an adapter holds (an infinity, say) reaches
  // no other adapter's rows.
  auto adapters = [&]() {
    constexpr int F = 2 * J;
    int id[F];
    float f[F];
    u32x4 hi[F][4], lo[F][4], b[2][4];
    const u32x4 zero = {0, 0, 0, 0};
    auto first_row = [&](int x) { return m0 + (x / J) * HM + wm * (HM / 2) + (x % J) * 32; };
    // addresses as one for the wave and 32 bits for the lane
    auto load_t = [&](int x, int c0) {
      const uint8_t* t = uniform(p.t + part_at(min(first_row(x), p.M - 1) & ~31, c0, p.R));
      const uint8_t* l = t + p.R * 64;
      const uint32_t at = lk * 512 + lr * 16;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        hi[x][ks] = lo[x][ks] = zero;
        if (c0 + 16 * ks + 8 * lk < p.R) {
          hi[x][ks] = *(const u32x4*)(t + (at + ks * 1024));
          lo[x][ks] = *(const u32x4*)(l + (at + ks * 1024));
        }
      }
    };
    auto load_b = [&](int a, int c0) {
#pragma unroll
      for (int hn = 0; hn < 2; ++hn) {
        const int col = n0 + wn * 64 + hn * 32;
        const uint8_t* w = uniform(p.b + ((int64_t)a * p.N + col) * p.R + c0);
        const uint32_t at = lr * (p.R * 2) + lk * 16;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          b[hn][ks] = zero;
          if (c0 + 16 * ks + 8 * lk < p.R && col + lr < p.N) b[hn][ks] = *(const u32x4*)(w + (at + ks * 32));
        }
      }
    };
#pragma unroll
    for (int x = 0; x < F; ++x) {
      const int row = first_row(x) + lr;
      id[x] = row < p.M ? p.sid[row] : p.L;
      f[x] = p.tf[min(row, p.M - 1)];
    }
#pragma unroll
    for (int x = 0; x < F; ++x) load_t(x, 0);
    int held = -1;  // whose factor b holds
#pragma unroll
    for (int x = 0; x < F; ++x) {
      clear(x / J, x % J);
      uint64_t rows = __ballot(id[x] < p.L);
      while (rows) {
        const int a = __builtin_amdgcn_readlane(id[x], __builtin_ctzll(rows));
        const bool mine = id[x] == a;
        rows &= ~__ballot(mine);
        for (int c0 = 0; c0 < p.R; c0 += 64) {
          if (held != a || p.R > 64) load_b(a, c0);
          held = a;
#pragma unroll
          for (int hn = 0; hn < 2; ++hn) {
            f32x16 tmp;
#pragma unroll
            for (int r = 0; r < 16; ++r) tmp[r] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              if (c0 + 16 * ks >= p.R) break;
              tmp = mfma<DT>(b[hn][ks], hi[x][ks], tmp);
              tmp = mfma<DT>(b[hn][ks], lo[x][ks], tmp);
            }
            if (mine) {
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[hn][x / J][x % J][r] += tmp[r] * f[x];
            }
          }
          if (p.R > 64) load_t(x, c0 + 64 < p.R ? c0 + 64 : 0);
        }
      }
    }
  };
  if (MODE != LORA || split != 0) {
#pragma unroll
    for (int hm = 0; hm < 2; ++hm)
#pragma unroll
      for (int j = 0; j < J; ++j) clear(hm, j);
  }

  // ---- main loop
  // The two waves of a SIMD (wm = 0 and 1) work half a phase apart: while one multiplies, the other reads the operands
  // of its next phase and starts a half's loads, and a barrier ends each turn. Waves with wm = 1 begin one
  // barrier later and end one earlier. Before the barrier behind its reads a wave has them all, and those of its loads
  // have landed that the next phase's reads need: all but the twelve youngest.
#define MOE_D16_MFMA(hn, hm, set, x) \
  acc[hn][hm][(x) % J] = mfma<DT>(fn[set][(x) / J % 4].get(), fm[(x) % J][(x) / J % 4].get(), acc[hn][hm][(x) % J]);
#define MOE_D16_PHASE(hn, hm, set, READS, LOAD, TIE)                                                   \
  {                                                                                                    \
    READS;                                                                                             \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    LOAD;                                                                                              \
    wait_all_but<12>();                                                                                \
    TIE;                                                                                               \
    barrier();                                                                                         \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    __builtin_amdgcn_s_setprio(1);                                                                     \
    _Pragma("unroll") for (int x = 0; x < 8; ++x) MOE_D16_MFMA(hn, hm, set, x)                         \
    __builtin_amdgcn_s_setprio(0);                                                                     \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    barrier();                                                                                         \
  }
  // Stage st in buffer B: its N half 0 is in set X already, the next stage's comes into set Y. Every half is
  // loaded for the stage after the next in the phase behind the one that read it.
#define MOE_D16_STAGE(st, B, X, Y)                                                                     \
  {                                                                                                    \
    MOE_D16_PHASE(0, 0, X, MOE_D16_ALL_M(0, B), load_n(0, (st) + 2, B), tie_m())                   \
    MOE_D16_PHASE(1, 0, 2, MOE_D16_ALL_N(2, 1, B), load_m(0, (st) + 2, B), tie_n(2))               \
    MOE_D16_PHASE(1, 1, 2, MOE_D16_ALL_M(1, B), load_n(1, (st) + 2, B), tie_m())                   \
    MOE_D16_PHASE(0, 1, X, MOE_D16_ALL_N(Y, 0, 1 - B), load_m(1, (st) + 2, B), tie_n(Y))           \
  }
  // 128 rows: a phase is all four blocks of two K steps, and the buffer read last is loaded anew, for the stage after the next,
  // in the two phases behind its last read.
#define MOE_D16_READ_P(B, p_)                                                                          \
  _Pragma("unroll") for (int x = 0; x < 2; ++x) {                                                      \
    if constexpr (MM) {                                                                                \
      if (x == 0) { gm[0][0].template read<(B) * 2 * HALF_M + (2 * (p_)) * 32 * HM>(m_at[0]); gm[1][0].template read<((B) * 2 + 1) * HALF_M + (2 * (p_)) * 32 * HM>(m_at[0]); } \
      else { gm[0][1].template read<(B) * 2 * HALF_M + (2 * (p_) + 1) * 32 * HM>(m_at[0]); gm[1][1].template read<((B) * 2 + 1) * HALF_M + (2 * (p_) + 1) * 32 * HM>(m_at[0]); } \
    } else {                                                                                           \
      gm[0][x].template read<(B) * 2 * HALF_M>(m_at[(2 * (p_) + x) % 4]);                                    \
      gm[1][x].template read<((B) * 2 + 1) * HALF_M>(m_at[(2 * (p_) + x) % 4]);                              \
    }                                                                                                  \
    if constexpr (NM) {                                                                                \
      if (x == 0) { gn[0][0].template read<((B) & 1) * 2 * HALF + (2 * (p_)) * 4096>(n_at[(B) >> 1][0]); gn[1][0].template read<(((B) & 1) * 2 + 1) * HALF + (2 * (p_)) * 4096>(n_at[(B) >> 1][0]); } \
      else { gn[0][1].template read<((B) & 1) * 2 * HALF + (2 * (p_) + 1) * 4096>(n_at[(B) >> 1][0]); gn[1][1].template read<(((B) & 1) * 2 + 1) * HALF + (2 * (p_) + 1) * 4096>(n_at[(B) >> 1][0]); } \
    } else {                                                                                           \
      gn[0][x].template read<((B) & 1) * 2 * HALF>(n_at[(B) >> 1][(2 * (p_) + x) % 4]);                      \
      gn[1][x].template read<(((B) & 1) * 2 + 1) * HALF>(n_at[(B) >> 1][(2 * (p_) + x) % 4]);                \
    }                                                                                                  \
  }
#define MOE_D16_MFMA_P(x) \
  acc[((x) >> 1) & 1][(x) & 1][0] = mfma<DT>(gn[((x) >> 1) & 1][(x) >> 2].get(), gm[(x) & 1][(x) >> 2].get(), acc[((x) >> 1) & 1][(x) & 1][0]);
#define MOE_D16_PHASE_P(B, p_, LOAD, LEFT)                                                             \
  {                                                                                                    \
    MOE_D16_READ_P(B, p_)                                                                              \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    LOAD;                                                                                              \
    wait_all_but<LEFT>();                                                                              \
    _Pragma("unroll") for (int x = 0; x < 4; ++x) {                                                    \
      gm[x >> 1][x & 1].tie();                                                                         \
      gn[x >> 1][x & 1].tie();                                                                         \
    }                                                                                                  \
    barrier();                                                                                         \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    __builtin_amdgcn_s_setprio(1);                                                                     \
    _Pragma("unroll") for (int x = 0; x < 8; ++x) MOE_D16_MFMA_P(x)                                    \
    __builtin_amdgcn_s_setprio(0);                                                                     \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
    barrier();                                                                                         \
  }
  // stage st in buffer B, the last one read in buffer A
#define MOE_D16_STAGE_P(st, B, A)                                                                      \
  {                                                                                                    \
    MOE_D16_PHASE_P(B, 0, { load_m(0, (st) + 2, A); load_n(0, (st) + 2, A); }, 9)                      \
    MOE_D16_PHASE_P(B, 1, { load_n(1, (st) + 2, A); load_m(1, (st) + 2, A); }, 6)                      \
  }
  if (nst > 0) {
    if constexpr (J == 2) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        load_n(0, s, s);
        load_m(0, s, s);
        load_n(1, s, s);
        load_m(1, s, s);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        load_m(0, s, s);
        load_n(0, s, s);
        load_n(1, s, s);
        load_m(1, s, s);
      }
    }
    if constexpr (MODE == LORA) {
      if (split == 0) adapters();
    }
    if constexpr (J == 2) {
      wait_loads<12>();
      barrier();
      MOE_D16_ALL_N(0, 0, 0)
      wait_all_but<12>();
      tie_n(0);
      barrier();
      if (wm) barrier();
      for (int s = 0; s < nst; s += 2) {
        if (MODE == LORA && touch && s == touch_at) touch_addend();
        MOE_D16_STAGE(s, 0, 0, 1)
        if (s + 1 >= nst) break;
        MOE_D16_STAGE(s + 1, 1, 1, 0)
      }
    } else {
      wait_loads<LS>();
      barrier();
      if (wm) barrier();
      for (int s = 0; s < nst; s += 3) {
        MOE_D16_STAGE_P(s, 0, 2)
        if (s + 1 >= nst) break;
        MOE_D16_STAGE_P(s + 1, 1, 0)
        if (s + 2 >= nst) break;
        MOE_D16_STAGE_P(s + 2, 2, 1)
      }
    }
    if (!wm) barrier();
    wait_loads<0>();
    barrier();
  }
#undef MOE_D16_STAGE_P
#undef MOE_D16_PHASE_P
#undef MOE_D16_MFMA_P
#undef MOE_D16_READ_P

  // ---- epilogue, from registers
  const int colw = n0 + (MODE == GATED || NM ? wn * 32 : wn * 64);      // the wave's first column of N half 0
  constexpr int STEP = NM ? 128 : 32;                                   // from there to half 1's (GATED: the same)
  auto add_bias = [&](int w, int col, float (&v)[4][4]) {               // the lane's 16 columns from col on
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int c = col + 8 * (r >> 2) + 4 * lk + (r & 3);
      v[r >> 2][r & 3] += p.bias[w][min(c, p.N - 1)];
    }
  };
  int orow[2][J];
#pragma unroll
  for (int hm = 0; hm < 2; ++hm)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = m0 + hm * HM + wm * (HM / 2) + j * 32 + lr;
      orow[hm][j] = MODE == LORA ? p.perm[min(row, p.M - 1)] : row;
    }
  // LORA's addend comes as whole lines, eight lanes to a row's 64 columns, all of it before the first result is stored,
  // and takes its place beside the results through LDS (asked for in their order, 16 bytes of 32 rows an instruction,
  // it cost the 256-row tiles of 8192 x 2048 x 7168 33 us).
  constexpr int PITCH = kStripPitch;
  uint8_t* strip = smem_arr + wave * 32 * PITCH;
  if constexpr (MODE == LORA) {
    if (!p.vec && p.splits == 1) {
#pragma unroll
      for (int hm = 0; hm < 2; ++hm)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float v[2][4][4];
#pragma unroll
          for (int hn = 0; hn < 2; ++hn)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[hn][r >> 2][r & 3] = acc[hn][hm][j][r];
          // rows that begin anywhere go through the strip both ways (a lane's values on their own, 2 bytes of 64 places an
          // instruction, cost 3330 x 264 x 8940 132 us, here 71 us)
          const int left = p.N - colw, rows = p.M - (m0 + hm * HM + wm * (HM / 2) + j * 32);
          if (left > 0 && rows > 0) {
            if (p.add) {
              wave_sync();
              move_rows<32, true>(strip, (uint16_t*)p.add + colw, p.ld_add, orow[hm][j], rows, left, p.pair, lane);
              wave_sync();
            }
#pragma unroll
            for (int hn = 0; hn < 2; ++hn) {
              if (p.bias[0]) add_bias(0, colw + hn * STEP, v[hn]);
              if (p.add) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint2 x = *(const uint2*)(strip + lr * PITCH + (hn * 32 + 8 * q + 4 * lk) * 2);
#pragma unroll
                  for (int i = 0; i < 4; ++i) v[hn][q][i] += load1<DT>(&x, i);
                }
              }
            }
            wave_sync();
#pragma unroll
            for (int hn = 0; hn < 2; ++hn)
#pragma unroll
              for (int q = 0; q < 4; ++q) *(uint2*)(strip + lr * PITCH + (hn * 32 + 8 * q + 4 * lk) * 2) = pack4<DT>(v[hn][q]);
            wave_sync();
            move_rows<32, false>(strip, (uint16_t*)p.out[0] + colw, p.ldo[0], orow[hm][j], rows, left, p.pair, lane);
          }
        }
      return;
    }
  }
  u32x4 line[2][J][4];
  const bool with_add = MODE == LORA && p.add && p.vec && p.splits == 1;
  if constexpr (MODE == LORA) {
    if (with_add) {
      const int c = colw + (lane & 7) * 8;
#pragma unroll
      for (int hm = 0; hm < 2; ++hm)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 3), o = __shfl(orow[hm][j], r);
            line[hm][j][i] = u32x4{0, 0, 0, 0};  // columns behind the last multiple of 8 get theirs where they are stored
            if (m0 + hm * HM + wm * (HM / 2) + j * 32 + r < p.M && c < p.N8)
              line[hm][j][i] = *(const u32x4*)((const uint16_t*)p.add + o * p.ld_add + c);
          }
    }
  }
#pragma unroll
  for (int hm = 0; hm < 2; ++hm) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = m0 + hm * HM + wm * (HM / 2) + j * 32 + lr;
      const bool ok = row < p.M;
      const int64_t o = orow[hm][j];
      float v[2][4][4];
#pragma unroll
      for (int hn = 0; hn < 2; ++hn)
#pragma unroll
        for (int r = 0; r < 16; ++r) v[hn][r >> 2][r & 3] = acc[hn][hm][j][r];
      if (p.splits > 1 || (MODE == DX && p.fold)) {
#pragma unroll
        for (int hn = 0; hn < 2; ++hn) {
          const int col = MODE == GATED ? colw : colw + hn * STEP;
          store_fragment_f32(part_of<MODE>(p, split, MODE == GATED ? hn : z, row, col), v[hn], lk, p.N - col, ok);
        }
      } else if constexpr (MODE == GATED) {
#pragma unroll
        for (int hn = 0; hn < 2; ++hn) {
          if (p.bias[0]) add_bias(hn, colw, v[hn]);
          if (p.keep[0]) store_fragment<DT>((uint16_t*)p.keep[hn] + o * p.ld_keep[hn] + colw, v[hn], lk, p.N - colw, ok);
        }
        with_act(p.act, [&](auto k) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            v[0][r >> 2][r & 3] = act_f<decltype(k)::value>(p.act, v[0][r >> 2][r & 3], v[1][r >> 2][r & 3]);
            if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // more evaluations at once do not fit the registers
          }
        });
        store_fragment<DT>((uint16_t*)p.out[0] + o * p.ldo[0] + colw, v[0], lk, p.N - colw, ok);
      } else if constexpr (MODE == DX) {
#pragma unroll
        for (int hn = 0; hn < 2; ++hn)
          store_fragment<DT>((uint16_t*)p.out[0] + o * p.ldo[0] + colw + hn * STEP, v[hn], lk, p.N - colw - hn * STEP, ok);
      } else if constexpr (MODE == DW) {
#pragma unroll
        for (int hn = 0; hn < 2; ++hn) finish_dw<DT>(p, z, o, colw + hn * STEP, v[hn], lk, ok);
      } else {
        if (with_add) {
          wave_sync();
#pragma unroll
          for (int i = 0; i < 4; ++i) *(u32x4*)(strip + (i * 8 + (lane >> 3)) * PITCH + (lane & 7) * 16) = line[hm][j][i];
          wave_sync();
        }
#pragma unroll
        for (int hn = 0; hn < 2; ++hn) {
          const int col = colw + hn * STEP;
          uint16_t* out = (uint16_t*)p.out[0] + o * p.ldo[0] + col;
          if (p.bias[0]) add_bias(0, col, v[hn]);
          if (with_add) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint2 x = *(const uint2*)(strip + lr * PITCH + (hn * 32 + 8 * q + 4 * lk) * 2);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[hn][q][i] += load1<DT>(&x, i);
            }
          }
          store_fragment<DT>(out, v[hn], lk, p.N8 - col, ok);
          // the columns behind the last multiple of 8
          if (ok && col + 32 > p.N8) {
            const uint16_t* add = p.add ? (const uint16_t*)p.add + o * p.ld_add + col : nullptr;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int c = 8 * (r >> 2) + 4 * lk + (r & 3);
              if (col + c < p.N && col + c >= p.N8) store1<DT>(out, c, v[hn][r >> 2][r & 3] + (add ? load1<DT>(add, c) : 0.f));
            }
          }
        }
      }
    }
  }
#undef MOE_D16_STAGE
#undef MOE_D16_PHASE
#undef MOE_D16_MFMA
#undef MOE_D16_ALL_M
#undef MOE_D16_ALL_N
#undef MOE_D16_READ_N
#undef MOE_D16_READ_M
}

}  // namespace d16
}  // namespace moe
