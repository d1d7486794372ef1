// Host side of the dense 16-bit projections: the gated block, its backward pass and
// projections with adapters. Argument checks, workspace and launches; no
// host synchronisation.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_experts.h"
#include "dense16.hpp"
#include "dense16_big.hpp"
#include "dense16_outer.hpp"
#include "gated_grad.hpp"
#include "lora.hpp"

namespace {

using namespace moe::d16;

int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t or_default(int64_t ld, int64_t d) { return ld ? ld : d; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxWidth = 1 << 20;
constexpr int64_t kMaxLd = (int64_t)1 << 21, kMaxLdOut = (int64_t)1 << 40;
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;  // workgroups: threads count in 32 bits

int check_ld(int64_t ld, int64_t n, int64_t per = 8, int64_t most = kMaxLd) {
  if (ld < n) return MOE_EINVAL;
  return ld % per || ld > most ? MOE_ENOTSUP : MOE_OK;
}
int first_of(std::initializer_list<int> rcs) {
  for (int rc : rcs)
    if (rc) return rc;
  return MOE_OK;
}
bool given16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned(p, 16)) return false;
  return true;
}

int type16(int32_t t) {
  if (t == MOE_T_BF16 || t == MOE_T_FP16) return MOE_OK;
  return t == MOE_T_FP32 ? MOE_ENOTSUP : MOE_EINVAL;
}

int check_act(const moe_gated_problem& p) {
  if (p.act != MOE_ACT_SILU && p.act != MOE_ACT_SWIGLU_OAI && p.act != MOE_ACT_SITU) return MOE_EINVAL;
  if (p.act == MOE_ACT_SILU) return MOE_OK;
  if (!std::isfinite(p.alpha) || !std::isfinite(p.beta)) return MOE_EINVAL;
  if (p.act == MOE_ACT_SITU) return p.alpha > 0.f && p.beta > 0.f ? MOE_OK : MOE_ENOTSUP;
  if (std::isnan(p.limit)) return MOE_EINVAL;
  return p.limit > 0.f ? MOE_OK : MOE_ENOTSUP;
}

// sizes, type and activation of a gated problem, and its leading dimensions
struct Gated {
  int64_t ldx, ld_wg, ld_wu, ld_out, ld_gate, ld_up;
};
int gated_sizes(const moe_gated_problem* p, Gated& g) {
  if (!p || p->M < 0 || p->H <= 0 || p->I <= 0) return MOE_EINVAL;
  int rc = first_of({type16(p->type), check_act(*p)});
  if (rc) return rc;
  if (p->M >= kMaxRows || p->H % 8 || p->I % 8 || p->H > kMaxWidth || p->I > kMaxWidth ||
      (int64_t)p->H * p->I > (int64_t)1 << 32)
    return MOE_ENOTSUP;
  g = {or_default(p->ldx, p->H),     or_default(p->ld_wg, p->H),   or_default(p->ld_wu, p->H),
       or_default(p->ld_out, p->I), or_default(p->ld_gate, p->I), or_default(p->ld_up, p->I)};
  return first_of({check_ld(g.ldx, p->H), check_ld(g.ld_wg, p->H), check_ld(g.ld_wu, p->H), check_ld(g.ld_out, p->I),
                   check_ld(g.ld_gate, p->I), check_ld(g.ld_up, p->I)});
}

moe::ActParams act_of(const moe_gated_problem& p) { return {p.act, p.alpha, p.beta, p.limit}; }

template <class F>
int with_type16(int32_t type, F f) {
  if (type == MOE_T_BF16) return f(std::integral_constant<int, moe::T_BF16>{});
  return f(std::integral_constant<int, moe::T_FP16>{});
}

// ------------------------------------------------------------ tiles
template <int DT, int MODE, int BM, bool PARTS>
int launch_big(Params& q, hipStream_t s) {
  q.mt = (int)cdiv(q.M, BM);
  q.nt = (int)cdiv(q.N, MODE == GATED ? 128 : 256);
  const int64_t n = cdiv((int64_t)q.mt * q.nt * (MODE == DW ? 2 : 1) * q.splits, 8) * 8;
  if (n > kMaxGrid / 2) return MOE_ENOTSUP;
  hipLaunchKernelGGL((k_big<DT, MODE, BM, PARTS>), dim3((unsigned)n), dim3(512), 0, s, q);
  const bool fold = MODE == DX && q.fold;
  if (q.splits > 1 || fold)
    hipLaunchKernelGGL((k_join<DT, MODE>), dim3((unsigned)cdiv((int64_t)(fold ? q.fold : q.M) * ((q.N + 7) / 8), 256), MODE == DW ? 2 : 1),
                       dim3(256), 0, s, q);
  return launch_status();
}

template <int DT>
int launch_outer(Params& q, hipStream_t s) {
  q.mt = (int)cdiv(q.M, 128);
  q.nt = (int)cdiv(q.N, 128);
  const int64_t n = cdiv((int64_t)q.mt * q.nt * 2, 8) * 8;
  if (n > kMaxGrid) return MOE_ENOTSUP;
  hipLaunchKernelGGL((k_outer<DT>), dim3((unsigned)n), dim3(256), outer_lds(q.K), s, q);
  return launch_status();
}

// q.K: of one product; PARTS: dg and du in two parts (k_big); part: room for plan_of's partial results
template <int DT, int MODE, bool PARTS = false>
int launch(Params& q, void* part, hipStream_t s) {
  const Plan plan = plan_of(MODE, q.M, q.N, PARTS ? parts_k(q.K) : q.K);
  q.splits = plan.splits;
  q.part = (float*)part;
  return plan.bm == 256 ? launch_big<DT, MODE, 256, PARTS>(q, s) : launch_big<DT, MODE, 128, PARTS>(q, s);
}

// ------------------------------------------------------------ few rows
// Rows up to which the weights are streamed (k_few), by what the present kernels gain on either side (us in a graph, rank 32):
//   adapters, 64: 33 x 2048 x 7168 (rows, in, out) 20.7 (tiles 37.2), 64 x 2880 x 2895 16.8 (35.3). The limit is a low one: 65 to 128 rows would
//   take 28 to 34 and 22 to 24 in place of tiles' 33 to 37 and 36 to 38.
//   gated, 32: 17 x 7168 x 2048 12.0 (tiles 21.1), 32 x 2880 x 2880 9.0 (16.2). Low, too: 33 to 64 rows in two workgroups of 32
//   would take 18 to 20 and 13 to 13.5 in place of 22 to 23 and 17 to 18.
constexpr int kFewRows = 64;  // of a projection with adapters
constexpr int kFewGated = 32;

template <int DT, int MODE, int S, int FN, int XI, int D, bool OWN = false>
int launch_few(Params& q, hipStream_t s) {
  q.mt = (int)cdiv(q.M, 8 * XI);
  q.nt = (int)cdiv(q.N, MODE == GATED ? 8 * FN : 16 * FN);
  hipLaunchKernelGGL((k_few<DT, MODE, S, FN, XI, D, OWN>), dim3((unsigned)(q.mt * q.nt)), dim3(64 * S), 0, s, q);
  return launch_status();
}

// Whether every workgroup finds the adapters' first products for itself: a wave has its four ranks' 2048 values on
// their way at once, so these are the times it waits for memory. us in a graph with a launch of their own, and without (M x K x N,
// rank): once 1 x 2048 x 7168, 16 11.1 and 9.9; twice 1 x 2048 x 7168, 32 11.5 and 11.7, 1 x 4096 x 4096, 32 13.8 and 13.9 (called
// from Python the launch costs 2 more); four times 4 x 2048 x 7168, 16 11.5 and 14.6; eight 8 x 2048 x 7168, 16 11.6 and 20.6.
bool own_products(int M, int N, int K, int R) {
  const int waves = cdiv(N, 16) <= 256 ? 8 : 4;
  return M <= 8 && cdiv((int64_t)M * R / 4, waves) * cdiv(K, 2048) <= 2;
}

// One weight fragment to eight waves where that makes at most a workgroup for every compute unit, else two fragments to four waves (us, the
// other form second; gated: 16 x 7168 x 2048 11.6 and 11.8, 32 12.8 and 14.5, 16 x 2880 x 2880 7.9 and 10.3; adapters: 16 x 4096 x 4096 11.6 and 12.7,
// 16 x 2048 x 7168 10.5 and 13.7).
template <int DT, int MODE>
int launch_rows(Params& q, hipStream_t s) {
  const bool few = cdiv(q.N, MODE == GATED ? 8 : 16) <= 256;
  if constexpr (MODE == LORA) {
    if (q.a) return few ? launch_few<DT, MODE, 8, 1, 1, 6, true>(q, s) : launch_few<DT, MODE, 4, 2, 1, 3, true>(q, s);
    // two workgroups of 32 rows to the same weights, both on a compute unit (64 x 2880 x 2895 with 64 rows in one: 13.2 us, here 12.4)
    if (q.M > 32) return launch_few<DT, MODE, 4, 1, 4, 3>(q, s);
  }
  if (q.M <= 8) return few ? launch_few<DT, MODE, 8, 1, 1, 6>(q, s) : launch_few<DT, MODE, 4, 2, 1, 3>(q, s);
  if (q.M <= 16) return few ? launch_few<DT, MODE, 8, 1, 2, 4>(q, s) : launch_few<DT, MODE, 4, 2, 2, 3>(q, s);
  return few ? launch_few<DT, MODE, 8, 1, 4, 3>(q, s) : launch_few<DT, MODE, 4, 2, 4, 2>(q, s);
}

// ------------------------------------------------------------ backward workspace
// dg and du of so few values (see gated_grad.hpp) go in two parts, others where the caller asks for it.
constexpr int kPartValues = 16384;
int grad_parts(const moe_gated_grad_problem& p) { return p.two_parts || (int64_t)p.fwd.M * p.fwd.I <= kPartValues ? 2 : 1; }
// The two parts of so few rows are further rows of dx's product, which a tile of 128 has room for, and further K rows of the weights',
// which k_outer holds; beyond, they are products of their own in k_big (us of a backward pass in one part and two: 100 x 2048 x 160
// 18.8 and 27.8, 200 x 264 x 72 24.3 and 36.3, 2048 x 4096 x 8 27.9 and 36.8).
bool parts_as_rows(const moe_gated_grad_problem& p) { return grad_parts(p) == 2 && 2 * p.fwd.M <= kOuterRows; }
// Rows of k_gated_grad's workgroups: all of them up to 256, so that the columns' sums need no second kernel, which pays where there are
// biases and columns enough (us of this step and the sums, 64 rows second: 128 x 2048 5.0 and 5.9, 256 x 14336 9.3 and 10.6; but 256 x 512 7.0 and
// 6.1). Without biases' gradients 64 rows would be the faster ones (with the weights' products 256 x 2048 15.5 and 12.5).
int grad_rows(int M) { return M <= 256 ? (M + 31) / 32 * 32 : 64; }
struct GradLayout {
  size_t dg, du, sums, part, bytes;
};
GradLayout grad_layout(const moe_gated_grad_problem& g) {
  GradLayout l;
  const moe_gated_problem& p = g.fwd;
  const int parts = grad_parts(g), M = parts_as_rows(g) ? 2 * p.M : p.M;
  const bool apart = parts == 2 && M == p.M;
  const size_t mi = up256((size_t)parts * p.M * p.I * 2);
  l.dg = 0;
  l.du = mi;
  l.sums = 2 * mi;
  l.part = l.sums + up256((size_t)cdiv(p.M, grad_rows(p.M)) * 2 * p.I * 4);
  // two parts of a row always meet in the join
  size_t dx = plan_of(DX, M, p.H, apart ? parts_k(p.I) : p.I).part;
  if (M > p.M) dx = std::max(dx, up256((size_t)M * p.H * 4));
  const bool outer = !apart && p.M <= kOuterRows;
  l.bytes = l.part + std::max(dx, outer ? 0 : plan_of(DW, p.I, p.H, apart ? parts_k(p.M) : p.M).part);
  return l;
}

int grad_sizes(const moe_gated_grad_problem* p, Gated& g, int64_t& ld_dx, int64_t& ld_dwg, int64_t& ld_dwu) {
  if (!p) return MOE_EINVAL;
  int rc = gated_sizes(&p->fwd, g);
  if (rc) return rc;
  if ((p->accumulate != 0 && p->accumulate != 1) || (p->two_parts != 0 && p->two_parts != 1)) return MOE_EINVAL;
  const bool f32 = p->dw_type == MOE_T_FP32;
  if (!f32 && p->dw_type != p->fwd.type) return p->dw_type == MOE_T_BF16 || p->dw_type == MOE_T_FP16 ? MOE_ENOTSUP : MOE_EINVAL;
  const int H = p->fwd.H;
  ld_dx = or_default(p->ld_dx, H);
  ld_dwg = or_default(p->ld_dwg, H);
  ld_dwu = or_default(p->ld_dwu, H);
  return first_of({check_ld(ld_dx, H, 8, kMaxLdOut), check_ld(ld_dwg, H, f32 ? 4 : 8, kMaxLdOut),
                   check_ld(ld_dwu, H, f32 ? 4 : 8, kMaxLdOut)});
}

// ------------------------------------------------------------ adapters
// Rows of x are read by 32-bit offsets from its start, so a call of more goes in parts.
int lora_rows(const moe_lora_problem& p, int64_t ldx) {
  return (int)std::min<int64_t>({(int64_t)p.M, (0x7fffffff - 2 * (int64_t)p.K) / (2 * ldx) / 256 * 256, (int64_t)1 << 20});
}
struct LoraLayout {
  size_t perm, sid, tf, t, part, bytes;
};
LoraLayout lora_layout(const moe_lora_problem& p, int rows) {
  LoraLayout l{};
  if (p.M <= kFewRows) {
    l.bytes = (size_t)p.M * p.R * 4;
    return l;
  }
  l.perm = 0;
  l.sid = up256((size_t)rows * 4);
  l.tf = l.sid + up256((size_t)rows * 4);
  l.t = l.tf + up256((size_t)rows * 4);
  l.part = l.t + up256((size_t)cdiv(rows, 32) * 32 * 4 * p.R);
  // partial results of the first product, then of the second; the last part of a call may be its smallest, with the most ranges
  size_t part = 0;
  for (int64_t n : {(int64_t)rows, (int64_t)p.M % rows})
    if (n) {
      if (shrink_ranges(n, p.K, p.R) > 1) part = std::max(part, (size_t)shrink_ranges(n, p.K, p.R) * n * p.R * 4);
      part = std::max(part, plan_of(LORA, n, p.N, p.K).part);
    }
  l.bytes = l.part + up256(part);
  return l;
}
int lora_sizes(const moe_lora_problem* p, int64_t& ldx, int64_t& ldw, int64_t& ldo, int64_t& lda) {
  if (!p || p->M < 0 || p->N <= 0 || p->K <= 0 || p->R <= 0 || p->L <= 0) return MOE_EINVAL;
  int rc = type16(p->type);
  if (rc) return rc;
  if (p->M >= kMaxRows || p->N > kMaxWidth || p->K > kMaxWidth || p->K % 8 || p->R % 8 || p->R > kMaxRank ||
      p->L > kMaxAdapters)
    return MOE_ENOTSUP;
  ldx = or_default(p->ldx, p->K);
  ldw = or_default(p->ldw, p->K);
  ldo = or_default(p->ld_out, p->N);
  lda = or_default(p->ld_add, p->N);
  return first_of({check_ld(ldx, p->K), check_ld(ldw, p->K), check_ld(ldo, p->N, 1, kMaxLdOut),
                   check_ld(lda, p->N, 1, kMaxLdOut)});
}

template <int DT, int RF>
void launch_shrink_of(const ShrinkParams& q, int ranges, hipStream_t s) {
  if constexpr (RF <= 4) {
    if (shrink_frags(q.M, q.R) == 2) {
      hipLaunchKernelGGL((k_lora_shrink<DT, RF, 2, false>), dim3((unsigned)cdiv(q.M, 32), (unsigned)ranges), dim3(512), 0, s, q);
      return;
    }
  }
  const dim3 g((unsigned)cdiv(q.M, 16), (unsigned)ranges);
  if (q.M <= kSortRows) hipLaunchKernelGGL((k_lora_shrink<DT, RF, 1, true>), g, dim3(512), 0, s, q);
  else hipLaunchKernelGGL((k_lora_shrink<DT, RF, 1, false>), g, dim3(512), 0, s, q);
}

template <int DT>
void launch_shrink(const ShrinkParams& q, int ranges, bool join, hipStream_t s) {
  if (q.R <= 16) launch_shrink_of<DT, 1>(q, ranges, s);
  else if (q.R <= 32) launch_shrink_of<DT, 2>(q, ranges, s);
  else if (q.R <= 64) launch_shrink_of<DT, 4>(q, ranges, s);
  else if (q.R <= 128) launch_shrink_of<DT, 8>(q, ranges, s);
  else launch_shrink_of<DT, 16>(q, ranges, s);
  if (!join) return;
  const dim3 g((unsigned)cdiv(q.M, 4)), b(256);
  if (q.R <= 64) hipLaunchKernelGGL((k_lora_finish<DT, 1>), g, b, 0, s, q, ranges);
  else if (q.R <= 128) hipLaunchKernelGGL((k_lora_finish<DT, 2>), g, b, 0, s, q, ranges);
  else hipLaunchKernelGGL((k_lora_finish<DT, 4>), g, b, 0, s, q, ranges);
}

template <int DT>
int launch_expand(const Params& q, const ShrinkParams& sh, int ranges, hipStream_t s) {
  const int frags = expand_frags(q.M);
  const dim3 g((unsigned)cdiv(q.M, 16 * frags), (unsigned)cdiv(q.N, 256));
  if (ranges > 1) hipLaunchKernelGGL((k_lora_expand<DT, true>), g, dim3(256), 0, s, q, frags, sh, ranges);
  else hipLaunchKernelGGL((k_lora_expand<DT, false>), g, dim3(256), 0, s, q, frags, sh, 1);
  return launch_status();
}

}  // namespace

extern "C" {

size_t moe_gated_linear_workspace_bytes(const moe_gated_problem* p) {
  Gated g;
  if (gated_sizes(p, g) || p->M <= kFewGated) return 0;
  return plan_of(GATED, p->M, p->I, p->H).part;
}

int moe_gated_linear(const moe_gated_problem* p, const void* x, const void* w_gate, const void* w_up,
                     const float* bias_gate, const float* bias_up, void* out, void* gate, void* up, void* workspace,
                     size_t workspace_bytes, moe_stream_t stream) {
  Gated g;
  int rc = gated_sizes(p, g);
  if (rc) return rc;
  if (p->M == 0) return MOE_OK;
  if (!given16({x, w_gate, w_up, out}) || !gate != !up || !aligned(gate, 16) || !aligned(up, 16) ||
      !bias_gate != !bias_up || !aligned(bias_gate, 4) || !aligned(bias_up, 4))
    return MOE_EINVAL;
  const size_t need = moe_gated_linear_workspace_bytes(p);
  if (need && (!workspace || !aligned(workspace, 16))) return MOE_EINVAL;
  if (workspace_bytes < need) return MOE_ENOSPC;
  Params q{};
  q.m[0] = (const uint16_t*)x;
  q.n[0] = (const uint16_t*)w_gate;
  q.n[1] = (const uint16_t*)w_up;
  q.ldm[0] = g.ldx;
  q.ldn[0] = g.ld_wg;
  q.ldn[1] = g.ld_wu;
  q.out[0] = out;
  q.ldo[0] = g.ld_out;
  q.M = p->M;
  q.N = p->I;
  q.K = p->H;
  q.splits = 1;
  q.bias[0] = bias_gate;
  q.bias[1] = bias_up;
  q.keep[0] = gate;
  q.keep[1] = up;
  q.ld_keep[0] = g.ld_gate;
  q.ld_keep[1] = g.ld_up;
  q.act = act_of(*p);
  hipStream_t s = (hipStream_t)stream;
  return with_type16(p->type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return p->M <= kFewGated ? launch_rows<DT, GATED>(q, s) : launch<DT, GATED>(q, workspace, s);
  });
}

size_t moe_gated_linear_backward_workspace_bytes(const moe_gated_grad_problem* p) {
  Gated g;
  int64_t a, b, c;
  if (grad_sizes(p, g, a, b, c) || p->fwd.M == 0) return 0;
  return grad_layout(*p).bytes;
}

int moe_gated_linear_backward(const moe_gated_grad_problem* p, const void* dout, const void* x, const void* w_gate,
                              const void* w_up, const void* gate, const void* up, void* dx, void* dw_gate, void* dw_up,
                              float* dbias_gate, float* dbias_up, void* workspace, size_t workspace_bytes,
                              moe_stream_t stream) {
  Gated g;
  int64_t ld_dx, ld_dwg, ld_dwu;
  int rc = grad_sizes(p, g, ld_dx, ld_dwg, ld_dwu);
  if (rc) return rc;
  if (!dw_gate != !dw_up || !dbias_gate != !dbias_up || (!dx && !dw_gate && !dbias_gate)) return MOE_EINVAL;
  if (!aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(dbias_gate, 4) || !aligned(dbias_up, 4))
    return MOE_EINVAL;
  const moe_gated_problem& f = p->fwd;
  hipStream_t s = (hipStream_t)stream;
  const bool f32 = p->dw_type == MOE_T_FP32;
  if (f.M == 0) {
    if (p->accumulate) return MOE_OK;
    if (dw_gate) {
      const dim3 grid((unsigned)cdiv((int64_t)f.I * f.H / 8, 256), 2);
      if (f32) hipLaunchKernelGGL((k_zero_rows<moe::T_FP32>), grid, dim3(256), 0, s, dw_gate, dw_up, ld_dwg, ld_dwu, f.I, f.H);
      else hipLaunchKernelGGL((k_zero_rows<moe::T_BF16>), grid, dim3(256), 0, s, dw_gate, dw_up, ld_dwg, ld_dwu, f.I, f.H);
    }
    if (dbias_gate)
      hipLaunchKernelGGL(k_column_sums, dim3((unsigned)cdiv(f.I, 256), 2), dim3(256), 0, s, (const float*)nullptr, 0, f.I,
                         dbias_gate, dbias_up, 0);
    return launch_status();
  }
  if (!given16({dout, gate, up, workspace}) || (dw_gate && !given16({x})) || (dx && !given16({w_gate, w_up}))) return MOE_EINVAL;
  const GradLayout l = grad_layout(*p);
  if (workspace_bytes < l.bytes) return MOE_ENOSPC;
  uint8_t* ws = (uint8_t*)workspace;
  GradParams r{};
  r.dout = dout;
  r.gate = gate;
  r.up = up;
  r.dg = ws + l.dg;
  r.du = ws + l.du;
  r.sums = dbias_gate ? (float*)(ws + l.sums) : nullptr;
  r.dbias[0] = dbias_gate;
  r.dbias[1] = dbias_up;
  r.accumulate = p->accumulate;
  r.parts = grad_parts(*p) == 2;
  r.ld_dout = g.ld_out;
  r.ld_gate = g.ld_gate;
  r.ld_up = g.ld_up;
  r.M = f.M;
  r.I = f.I;
  r.rows = grad_rows(f.M);
  r.act = act_of(f);
  const int blocks = (int)cdiv(f.M, r.rows);
  const bool as_rows = parts_as_rows(*p), apart = r.parts && !as_rows;
  Params q{};
  q.m[0] = (const uint16_t*)r.dg;
  q.m[1] = (const uint16_t*)r.du;
  q.ldm[0] = q.ldm[1] = f.I;
  q.splits = 1;
  q.fold = as_rows ? f.M : 0;
  q.lower = (int64_t)f.M * f.I;
  return with_type16(f.type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipLaunchKernelGGL((k_gated_grad<DT>), dim3((unsigned)blocks, (unsigned)cdiv(f.I, 64)), dim3(256), 0, s, r);
    if (dbias_gate && blocks > 1)
      hipLaunchKernelGGL(k_column_sums, dim3((unsigned)cdiv(f.I, 256), 2), dim3(256), 0, s, (const float*)r.sums, blocks, f.I,
                         dbias_gate, dbias_up, p->accumulate);
    int rc = launch_status();
    if (!rc && dx) {
      Params d = q;
      d.n[0] = (const uint16_t*)w_gate;
      d.n[1] = (const uint16_t*)w_up;
      d.ldn[0] = g.ld_wg;
      d.ldn[1] = g.ld_wu;
      d.out[0] = dx;
      d.ldo[0] = ld_dx;
      d.M = as_rows ? 2 * f.M : f.M;
      d.N = f.H;
      d.K = f.I;
      rc = apart ? launch<DT, DX, true>(d, ws + l.part, s) : launch<DT, DX>(d, ws + l.part, s);
    }
    if (!rc && dw_gate) {
      Params d = q;
      d.n[0] = (const uint16_t*)x;
      d.ldn[0] = g.ldx;
      d.out[0] = dw_gate;
      d.out[1] = dw_up;
      d.ldo[0] = ld_dwg;
      d.ldo[1] = ld_dwu;
      d.M = f.I;
      d.N = f.H;
      d.K = as_rows ? 2 * f.M : f.M;
      d.f32_out = f32;
      d.accumulate = p->accumulate;
      rc = apart ? launch<DT, DW, true>(d, ws + l.part, s)
                 : f.M <= kOuterRows ? launch_outer<DT>(d, s) : launch<DT, DW>(d, ws + l.part, s);
    }
    return rc;
  });
}

size_t moe_lora_linear_workspace_bytes(const moe_lora_problem* p) {
  int64_t ldx, ldw, ldo, lda;
  if (lora_sizes(p, ldx, ldw, ldo, lda) || p->M == 0) return 0;
  return lora_layout(*p, lora_rows(*p, ldx)).bytes;
}

int moe_lora_linear(const moe_lora_problem* p, const void* x, const void* w, const void* lora_a, const void* lora_b,
                    const int32_t* ids, const float* scales, const float* bias, const void* add, void* out,
                    void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int64_t ldx, ldw, ldo, lda;
  int rc = lora_sizes(p, ldx, ldw, ldo, lda);
  if (rc) return rc;
  if (p->M == 0) return MOE_OK;
  if (!given16({x, lora_a, lora_b, workspace}) || !aligned(w, 16) || !ids || !scales || !out || !aligned(ids, 4) ||
      !aligned(scales, 4) || !aligned(bias, 4) || !aligned(add, 2) || !aligned(out, 2))
    return MOE_EINVAL;
  const int rows = lora_rows(*p, ldx);
  const LoraLayout l = lora_layout(*p, rows);
  if (workspace_bytes < l.bytes) return MOE_ENOSPC;
  uint8_t* ws = (uint8_t*)workspace;
  hipStream_t s = (hipStream_t)stream;
  Params q{};
  q.n[0] = (const uint16_t*)w;
  q.ldm[0] = ldx;
  q.ldn[0] = ldw;
  q.ldo[0] = ldo;
  q.N = p->N;
  q.K = w ? p->K : 0;
  q.splits = 1;
  q.bias[0] = bias;
  q.ld_add = lda;
  q.vec = aligned(out, 16) && ldo % 8 == 0 && (!add || (aligned(add, 16) && lda % 8 == 0));
  q.pair = aligned(out, 4) && ldo % 2 == 0 && (!add || (aligned(add, 4) && lda % 2 == 0));
  q.N8 = p->N / 8 * 8;
  q.R = p->R;
  q.L = p->L;
  q.t = (const uint16_t*)(ws + l.t);
  q.tf = (const float*)(ws + l.tf);
  q.b = (const uint16_t*)lora_b;
  q.perm = (const int32_t*)(ws + l.perm);
  q.sid = (const int32_t*)(ws + l.sid);
  if (p->M <= kFewRows) {
    q.m[0] = (const uint16_t*)x;
    q.out[0] = out;
    q.add = add;
    q.M = p->M;
    q.tf = (const float*)ws;
    q.sid = ids;
    return with_type16(p->type, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      const ShrinkParams sh{q.m[0], (const uint16_t*)lora_a, scales, nullptr, nullptr, ids, nullptr, (float*)ws, nullptr, ldx,
                            p->M, p->K, p->R, p->L};
      if (w && own_products(p->M, p->N, p->K, p->R)) {
        q.a = sh.a;
        q.scales = scales;
      } else {
        hipLaunchKernelGGL((k_lora_shrink_few<DT>), dim3((unsigned)p->M, (unsigned)p->R / 8), dim3(256), 0, s, sh);
      }
      return launch_rows<DT, LORA>(q, s);
    });
  }
  return with_type16(p->type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    for (int64_t m = 0; m < p->M; m += rows) {
      const int n = (int)std::min<int64_t>(rows, p->M - m);
      q.m[0] = (const uint16_t*)x + m * ldx;
      q.out[0] = (uint16_t*)out + m * ldo;
      q.add = add ? (const uint16_t*)add + m * lda : nullptr;
      q.M = n;
      const SortParams sp{ids + m, (int32_t*)(ws + l.perm), (int32_t*)(ws + l.sid), n, p->L};
      if (n > kSortRows) hipLaunchKernelGGL(k_lora_sort, dim3(1), dim3(1024), 0, s, sp);
      const ShrinkParams sh{q.m[0], (const uint16_t*)lora_a, scales, sp.perm, sp.sid, sp.ids, (uint16_t*)(ws + l.t),
                            (float*)(ws + l.tf), (float*)(ws + l.part), ldx, n, p->K, p->R, p->L};
      const int ranges = shrink_ranges(n, p->K, p->R);
      const bool join = ranges > 1 && (w || expand_frags(n) > 1);
      launch_shrink<DT>(sh, ranges, join, s);
      int rc = launch_status();
      if (!rc) rc = w ? launch<DT, LORA>(q, ws + l.part, s) : launch_expand<DT>(q, sh, join ? 1 : ranges, s);
      if (rc) return rc;
    }
    return (int)MOE_OK;
  });
}

}  // extern "C"
