// General expert routing (moe_route_topk): logits -> scores -> (bias, groups)
// -> top-k ids and weights.
//
// trtllm_mxfp4_moe page, TrtLlmMxfp4ExpertsMonolithic.apply (correction bias,
// expert groups, groups kept, routed scaling factor). Scores are a softmax
// over all experts or sigmoids, evaluated in double and rounded once to fp32;
// selection scores and group scores are single fp32 additions of them, so the
// picks do not depend on how the work is split over lanes.
//
// L lanes per token (16: four tokens per wave, up to 256 experts; 64: up to
// 1024), lane l holding experts PER l .. PER l + PER - 1, so that a group of
// experts is a whole number of neighbouring lanes in the usual cases.
// Cross-lane steps stay inside the token's lanes: with 16 they are four DPP
// rotations, so four tokens share every instruction.
//
// Selection works on order-preserving 32-bit keys of the scores. The k-th
// largest of the lanes' own maxima (or two largest) is at most the k-th largest key, so
// the picks are among the keys that reach it, usually few more than k: those are
// listed in LDS in index order and each counts the ones that beat it (a larger
// key, or an equal one earlier in the list), which is its place in the output.
// With more than kList of them (many equal scores) the wave takes the picks
// one by one instead, each the largest key and among its holders the lowest index.
//
// Bound by instructions: 16384 x 256 fp32 in 8 groups 14.5 us (17.8 MB, 1.2 TB/s), most of it the
// sigmoids in double; 65536 x 256 softmax 34 us (2.1 TB/s); 32 x 128 4.0 us, the chain of one token.
#pragma once

#include "elem.hpp"
#include "router.hpp"

namespace moe {

struct RouteTopkParams {
  const void* logits;  // [T, ld] bf16 / fp16 / fp32
  const float* bias;   // [E] or nullptr
  int32_t* ids;        // [T, k]
  float* w;            // [T, k]
  int64_t ld;
  int32_t T, E, k;
  int32_t sigmoid;     // scores: 1 sigmoid, 0 softmax
  int32_t n_group, topk_group;  // n_group 0: no groups
  int32_t per_group;            // E / n_group
  int32_t top2;        // group score: 1 sum of the two largest, 0 the largest
  int32_t renorm;
  float scale;
};

template <int DT>
__device__ __forceinline__ float load1(const void* base, size_t i) {
  if constexpr (DT == T_FP32) return ((const float*)base)[i];
  else if constexpr (DT == T_FP16) return (float)((const _Float16*)base)[i];
  else return bf16_bits_to_f32(((const uint16_t*)base)[i]);
}

// value of lane (lane rotated by N within its 16)
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);
}

// Reductions over a token's L lanes; every lane gets the result.
template <int L, class F>
__device__ __forceinline__ uint32_t token_reduce(uint32_t v, F f) {
  v = f(v, row_ror<8>(v));
  v = f(v, row_ror<4>(v));
  v = f(v, row_ror<2>(v));
  v = f(v, row_ror<1>(v));
  if (L == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
  return token_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t token_min(uint32_t v) {
  return token_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L>
__device__ __forceinline__ float token_maxf(float v) {
  return __uint_as_float(token_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int N>
__device__ __forceinline__ double row_ror_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)row_ror<N>((uint32_t)(u >> 32)) << 32 | row_ror<N>((uint32_t)u));
}
template <int L>
__device__ __forceinline__ double token_sum(double v) {
  v += row_ror_f64<8>(v);
  v += row_ror_f64<4>(v);
  v += row_ror_f64<2>(v);
  v += row_ror_f64<1>(v);
  if (L == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
// value of the lane N below within its 16, 0 for the first N
template <int N>
__device__ __forceinline__ int row_shr(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x110 + N, 0xf, 0xf, true);
}
// sum of v over the token's lanes up to this one
template <int L>
__device__ __forceinline__ int token_upto(int v, int l) {
  v += row_shr<1>(v);
  v += row_shr<2>(v);
  v += row_shr<4>(v);
  v += row_shr<8>(v);
  if (L == 64) {
    const int o = __shfl(v, (l & 48) - 1 < 0 ? 0 : (l & 48) - 1);  // the row before's sum
    const int a = l >= 16 ? o : 0;
    const int o2 = __shfl(v, 15), o3 = __shfl(v, 31);
    v += l < 16 ? 0 : l < 32 ? a : l < 48 ? a + o2 : a + o2 + o3;
  }
  return v;
}

// e^t in double, to a few 2^-52: t = n ln 2 + r with |r| <= ln 2 / 2, e^r
// by its Taylor sum to r^12 (the next term is below 2^-52). n ln 2 is subtracted in two parts, as Cody and Waite
// do it: ln 2 rounded to a multiple of 2^-42, whose product with n (8 bits) is exact, and the rest. t is taken within
// +-120: e^-120 is near 1e-52, which no fp32 score or sum can tell from 0.
__device__ __forceinline__ double exp_120(double t) {
  t = fmin(fmax(t, -120.0), 120.0);
  const double n = __builtin_rint(t * 1.4426950408889634074);
  double r = fma(n, -0x1.62e42fefa38p-1, t);
  r = fma(n, -0x1.ef35793c7673p-45, r);
  double p = 1.0 / 479001600.0;
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / v for v in [1, 2^200), to a few 2^-52: v_rcp_f64 and two Newton steps
__device__ __forceinline__ double rcp_f64(double v) {
  double y = __builtin_amdgcn_rcp(v);
  y = fma(fma(-v, y, 1.0), y, y);
  return fma(fma(-v, y, 1.0), y, y);
}

// the two largest of (a1 >= a2) and (b1 >= b2)
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

constexpr int kTopkGroups = 64;
constexpr int kList = 64;  // candidates listed per token

// VEC: rows, row starts and bias are 16-byte aligned and E is a multiple of PER
template <int DT, int L, int PER, bool VEC>
__global__ __launch_bounds__(256) void k_route_topk(const RouteTopkParams p) {
  constexpr int TPW = 64 / L;      // tokens per wave
  constexpr int TPB = 4 * TPW;     // per workgroup
  const int slot = threadIdx.x / L;
  __shared__ float sel_lds[TPB][L * PER + 4];
  __shared__ __attribute__((aligned(16))) uint32_t max_lds[TPB][2 * L];
  __shared__ __attribute__((aligned(16))) uint64_t list[TPB][kList + 2];  // expert, key
  float* const grp = (float*)list[slot];  // group scores, before the list
  static_assert(kTopkGroups * 4 <= (kList + 2) * 8, "group scores fit the list");
  const int lane = threadIdx.x & 63, l = lane & (L - 1);
  const int t_in = blockIdx.x * TPB + slot;
  const int t = min(t_in, p.T - 1);  // lanes past the last token repeat it and store nothing
  const size_t row = (size_t)t * p.ld;
  const int e0 = l * PER;
  constexpr float kMax = 3.402823466e38f;

  float sc[PER], bias[PER];
  float top = -kMax;
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = 0.f;
  if constexpr (VEC) {
    if (p.bias && e0 < p.E) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const f32x4 b = *(const f32x4*)(p.bias + e0 + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) bias[i + j] = b[j];
      }
    }
#pragma unroll
    for (int i = 0; i < PER; i += 8) {
      float v[8] = {-kMax, -kMax, -kMax, -kMax, -kMax, -kMax, -kMax, -kMax};
      if (e0 < p.E) load8<DT>(p.logits, row + e0 + i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sc[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      sc[i] = load1<DT>(p.logits, row + min(e0 + i, p.E - 1));
      if (e0 + i >= p.E) sc[i] = -kMax;
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i) bias[i] = p.bias[min(e0 + i, p.E - 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    sc[i] = fminf(fmaxf(sc[i], -kMax), kMax);  // NaN becomes the most negative value
    top = fmaxf(top, sc[i]);
  }
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) sc[i] = (float)rcp_f64(1.0 + exp_120(-(double)sc[i]));
  } else {
    top = token_maxf<L>(top);
    double ex[PER], sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      ex[i] = exp_120((double)sc[i] - (double)top);
      if (e0 + i >= p.E) ex[i] = 0.0;
      sum += ex[i];
    }
    sum = rcp_f64(token_sum<L>(sum));
#pragma unroll
    for (int i = 0; i < PER; ++i) sc[i] = (float)(ex[i] * sum);
  }
  // selection scores
  float sel[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) sel[i] = sc[i] + bias[i];
  auto wave_sync = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  uint64_t kept = ~0ull;  // groups that stay
  int G = 1;
  bool lanes_whole = true;  // a lane's experts are all of one group
  bool lane_kept = true;    // and that group stays
  if (p.n_group) {
    G = p.per_group;
    const int span = G / PER;  // lanes of a group
    lanes_whole = G % PER == 0 && (span & (span - 1)) == 0 && span <= L;
    if (lanes_whole) {
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) merge_top2(m1, m2, sel[i], -INFINITY);
      for (int d = 1; d < span; d <<= 1) {
        const float o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
        merge_top2(m1, m2, o1, o2);
      }
      const float score = p.top2 ? m1 + m2 : m1;  // the same in all lanes of the group
      if constexpr (L == 16) {
        // the group stays if fewer than topk_group groups beat it, counted by lanes
        max_lds[slot][l] = __float_as_uint(e0 < p.E ? score : -INFINITY);
        wave_sync();
        const int first = l & ~(span - 1), lanes = p.E / PER;
        int beat = 0;
#pragma unroll
        for (int m = 0; m < L; ++m) {
          const float o = __uint_as_float(max_lds[slot][m]);
          beat += m < lanes && (o > score || (o == score && m < first));
        }
        wave_sync();
        lane_kept = beat < p.topk_group * span;
      } else if (e0 < p.E && l % span == 0) {
        grp[l / span] = score;
      }
    } else {  // groups that cut lanes apart: through LDS
#pragma unroll
      for (int i = 0; i < PER; ++i) sel_lds[slot][e0 + i] = sel[i];
      wave_sync();
      for (int g = l; g < p.n_group; g += L) {
        float m1 = -INFINITY, m2 = -INFINITY;
        for (int j = 0; j < G; ++j) merge_top2(m1, m2, sel_lds[slot][g * G + j], -INFINITY);
        grp[g] = p.top2 ? m1 + m2 : m1;
      }
    }
    wave_sync();
    // a group stays if fewer than topk_group groups beat it (larger score, or equal and lower index)
    const bool ranked = L == 16 && lanes_whole;
    if (!ranked) kept = 0;
    for (int g0 = ranked ? p.n_group : 0; g0 < p.n_group; g0 += L) {
      const int g = g0 + l;
      bool in = false;
      if (g < p.n_group) {
        const float mine = grp[g];
        int beat = 0;
        for (int o = 0; o < p.n_group; ++o) {
          const float v = grp[o];
          beat += v > mine || (v == mine && o < g);
        }
        in = beat < p.topk_group;
      }
      const uint64_t m = __ballot(in);
      kept |= (L == 64 ? m : (m >> (lane & ~(L - 1))) & ((1ull << (L & 63)) - 1)) << g0;
    }
  }
  uint32_t key[PER];  // 0: not a candidate
  uint32_t top_key = 0;
  if (L == 64 && p.n_group && lanes_whole) lane_kept = (kept >> (min(e0, p.E - 1) / G)) & 1ull;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    key[i] = e < p.E && lane_kept ? max(route_key(sel[i]), 1u) : 0u;
  }
  if (!lanes_whole) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!((kept >> (min(e0 + i, p.E - 1) / G)) & 1ull)) key[i] = 0u;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) top_key = max(top_key, key[i]);

  // A key that the picks reach: the k-th largest of the lanes' maxima, or, where
  // those are few for k (only the kept groups' lanes have any), of their two largest.
  uint32_t thr = 1u;
  int upto = 0, mine = 0, count = kList + 1;
  const bool two = (L == 16 && p.n_group) || p.k > L / 2;
  if (p.k <= 2 * L) {
    if (!two) {
      max_lds[slot][l] = top_key;
      wave_sync();
      int above = 0;
#pragma unroll
      for (int m = 0; m < L; ++m) above += max_lds[slot][m] > top_key;
      thr = token_min<L>(above < p.k ? top_key : 0xffffffffu);
    } else {
      uint32_t next = 0;
      top_key = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        next = max(next, min(top_key, key[i]));
        top_key = max(top_key, key[i]);
      }
      max_lds[slot][l] = top_key;
      max_lds[slot][L + l] = next;
      wave_sync();
      int above = 0, above2 = 0;
#pragma unroll
      for (int m = 0; m < 2 * L; ++m) {
        const uint32_t o = max_lds[slot][m];
        above += o > top_key;
        above2 += o > next;
      }
      thr = token_min<L>(above2 < p.k ? next : above < p.k ? top_key : 0xffffffffu);
    }
    thr = max(thr, 1u);
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += key[i] >= thr;
    upto = token_upto<L>(mine, l);
    count = (int)token_max<L>((uint32_t)upto);
  }
  if (__all(count <= kList)) {
    uint64_t* at = &list[slot][upto - mine];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] >= thr) *at++ = (uint64_t)key[i] << 32 | (uint32_t)(e0 + i);
    if (l < 2) list[slot][count + l] = 0u;  // whole pairs below
    if (p.bias) {  // the picks' weights are their scores without the bias
#pragma unroll
      for (int i = 0; i < PER; ++i) sel_lds[slot][e0 + i] = sc[i];
    }
    wave_sync();
    double total = 0.0;
    constexpr int CPL = kList / L;  // candidates per lane, nearly always one
    int place[CPL], id[CPL];
    float s[CPL];
#pragma unroll
    for (int h = 0; h < CPL; ++h) {
      place[h] = -1;
      if (!__any(L * h < count)) continue;
      const int j = l + L * h;
      const uint64_t c = j < count ? list[slot][j] : ~0ull;
      const uint32_t ck = (uint32_t)(c >> 32);
      id[h] = (int)(uint32_t)c;
      int n = 0;
      for (int x = 0; x < count; x += 2) {
        const u32x4 o = *(const u32x4*)&list[slot][x];
        n += o[1] > ck || (o[1] == ck && x < j);
        n += o[3] > ck || (o[3] == ck && x + 1 < j);
      }
      if (j < count && n < p.k) {
        place[h] = n;
        s[h] = p.bias ? sel_lds[slot][id[h]]
                      : __uint_as_float((ck & 0x80000000u) ? ck & 0x7fffffffu : ~ck);
        total += (double)s[h];
      }
    }
    if (p.renorm) total = token_sum<L>(total);
    if (t_in >= p.T) return;
#pragma unroll
    for (int h = 0; h < CPL; ++h) {
      if (place[h] < 0) continue;
      float w = s[h];
      if (p.renorm) w = total > 0.0 ? (float)((double)w / total) : 0.f;
      p.ids[(size_t)t * p.k + place[h]] = id[h];
      p.w[(size_t)t * p.k + place[h]] = w * p.scale;
    }
    return;
  }

  double total = 0.0;
  int my_id[2] = {0, 0};
  float my_sc[2] = {0.f, 0.f};
  for (int r = 0; r < p.k; ++r) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    best = token_max<L>(best);
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) at = (uint32_t)(e0 + i);
    at = token_min<L>(at);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == (uint32_t)(e0 + i)) {
        s = sc[i];
        key[i] = 0u;
      }
    s = __shfl(s, (int)((lane & ~(L - 1)) | (at / PER & (L - 1))));
    total += (double)s;
    if (l == (r & (L - 1))) {
      my_id[r >= L] = (int)at;
      my_sc[r >= L] = s;
    }
  }
  if (t_in >= p.T) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = l + L * h;
    if (r >= p.k) break;
    float w = my_sc[h];
    if (p.renorm) w = total > 0.0 ? (float)((double)w / total) : 0.f;
    p.ids[(size_t)t * p.k + r] = my_id[h];
    p.w[(size_t)t * p.k + r] = w * p.scale;
  }
}

}  // namespace moe
