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
// 1024), lane l holding experts l, l + L, ... (PER of them). Cross-lane steps
// stay inside the token's lanes: with 16 they are four DPP rotations, so four
// tokens share every instruction. Each of the k rounds takes the largest
// order-preserving 32-bit key and, among its holders, the lowest index.
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
template <int L>
__device__ __forceinline__ double token_sum(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kTopkGroups = 64;

template <int DT, int L, int PER>
__global__ __launch_bounds__(256) void k_route_topk(const RouteTopkParams p) {
  constexpr int TPW = 64 / L;      // tokens per wave
  constexpr int TPB = 4 * TPW;     // per workgroup
  __shared__ float sel_lds[TPB][L * PER + 4];
  __shared__ float grp_lds[TPB][kTopkGroups];
  const int lane = threadIdx.x & 63, l = lane & (L - 1);
  const int slot = threadIdx.x / L;
  const int t_in = blockIdx.x * TPB + slot;
  const int t = min(t_in, p.T - 1);  // lanes past the last token repeat it and store nothing
  const size_t row = (size_t)t * p.ld;
  constexpr float kMax = 3.402823466e38f;

  float sc[PER];
  uint32_t key[PER];
  float top = -kMax;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = l + L * i;
    float x = -kMax;
    if (e < p.E) x = load1<DT>(p.logits, row + e);
    sc[i] = x != x ? -kMax : fminf(fmaxf(x, -kMax), kMax);  // NaN counts as the most negative value
    top = fmaxf(top, sc[i]);
  }
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) sc[i] = (float)(1.0 / (1.0 + exp(-(double)sc[i])));
  } else {
    top = token_maxf<L>(top);
    double ex[PER], sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      ex[i] = l + L * i < p.E ? exp((double)sc[i] - (double)top) : 0.0;
      sum += ex[i];
    }
    sum = 1.0 / token_sum<L>(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) sc[i] = (float)(ex[i] * sum);
  }
  auto wave_sync = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  // selection keys (0: not a candidate)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = l + L * i;
    float v = sc[i];
    if (p.bias && e < p.E) v += p.bias[e];
    key[i] = e < p.E ? max(route_key(v), 1u) : 0u;
    if (p.n_group) sel_lds[slot][e] = v;
  }
  if (p.n_group) {
    wave_sync();
    const int G = p.E / p.n_group;
    for (int g = l; g < p.n_group; g += L) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int j = 0; j < G; ++j) {
        const float v = sel_lds[slot][g * G + j];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      grp_lds[slot][g] = p.top2 ? m1 + m2 : m1;
    }
    wave_sync();
    // a group stays if fewer than topk_group groups beat it (larger score, or equal and lower index)
    uint64_t kept = 0;
    for (int g0 = 0; g0 < p.n_group; g0 += L) {
      const int g = g0 + l;
      bool in = false;
      if (g < p.n_group) {
        const float mine = grp_lds[slot][g];
        int beat = 0;
        for (int o = 0; o < p.n_group; ++o) {
          const float v = grp_lds[slot][o];
          beat += v > mine || (v == mine && o < g);
        }
        in = beat < p.topk_group;
      }
      const uint64_t m = __ballot(in);
      kept |= (L == 64 ? m : (m >> (lane & ~(L - 1))) & ((1ull << (L & 63)) - 1)) << g0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = l + L * i;
      if (e < p.E && !((kept >> (e / G)) & 1ull)) key[i] = 0u;
    }
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
      if (key[i] == best) at = (uint32_t)(l + L * i);
    at = token_min<L>(at);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == (uint32_t)(l + L * i)) {
        s = sc[i];
        key[i] = 0u;
      }
    s = __shfl(s, (int)((lane & ~(L - 1)) | (at & (L - 1))));
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
