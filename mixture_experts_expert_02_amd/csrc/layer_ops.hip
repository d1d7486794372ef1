// Host side of the operators around the experts step: row norm, microscaled
// quantization, the dense MXFP4 product, general routing. Argument checks and
// launches; one kernel per call, no workspace, no host synchronisation.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_experts.h"
#include "mx_linear.hpp"
#include "mx_linear_rule.hpp"
#include "mx_quant.hpp"
#include "norm.hpp"
#include "route_topk.hpp"

namespace {

int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool type_ok(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_FP16 || t == MOE_T_FP32; }
int64_t or_default(int64_t ld, int64_t d) { return ld ? ld : d; }

constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int kMaxRows = 1 << 24;                        // routing: 64 threads to a row still count in 32 bits
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;     // workgroups of 256 threads

// rows of n values of the type, ld elements apart: 16-byte accesses at every multiple of 8
int check_rows(const void* p, int64_t ld, int64_t n, int32_t type) {
  if (!p || !aligned(p, 16) || ld < n) return MOE_EINVAL;
  if ((ld * moe::elem_size(type)) % 16 || ld > kMaxLd) return MOE_ENOTSUP;
  return MOE_OK;
}
// rows of codes and scales, byte strides
int check_codes(const void* codes, int64_t ld, const void* scales, int64_t lds, int64_t K, int32_t fmt) {
  if (!codes || !scales || !aligned(codes, 16)) return MOE_EINVAL;
  if (ld < moe::mxf::code_bytes(fmt, K) || lds < K / 32) return MOE_EINVAL;
  if (ld % 16 || ld > kMaxLd || lds > kMaxLd) return MOE_ENOTSUP;
  return MOE_OK;
}

// Calls f with the element type (and the block format) as compile-time constants.
template <class F>
void with_type(int32_t type, F f) {
  if (type == MOE_T_BF16) f(std::integral_constant<int, moe::T_BF16>{});
  else if (type == MOE_T_FP16) f(std::integral_constant<int, moe::T_FP16>{});
  else f(std::integral_constant<int, moe::T_FP32>{});
}

// ------------------------------------------------------------- quantization
int rows_params(const moe_mx_rows* p, moe::mxf::RowsParams& q, bool& flat) {
  if (!p || p->rows < 0 || p->K <= 0 || !type_ok(p->type)) return MOE_EINVAL;
  if (p->fmt != MOE_MX_FP4 && p->fmt != MOE_MX_FP8) return MOE_EINVAL;
  if (p->K % 32) return MOE_ENOTSUP;
  if ((int64_t)p->rows * p->K > (int64_t)1 << 34) return MOE_ENOTSUP;
  const int64_t cb = moe::mxf::code_bytes(p->fmt, p->K);
  q.ld = or_default(p->ld, p->K);
  q.ld_codes = or_default(p->ld_codes, cb);
  q.ld_scales = or_default(p->ld_scales, p->K / 32);
  q.per_row = (uint32_t)p->K / 8;
  q.n = (uint32_t)((int64_t)p->rows * p->K / 8);
  flat = q.ld == p->K && q.ld_codes == cb && q.ld_scales == p->K / 32;
  return MOE_OK;
}

int check_mx_rows(const moe_mx_rows* p, const moe::mxf::RowsParams& q, const void* values) {
  int rc = check_rows(values, q.ld, p->K, p->type);
  if (rc) return rc;
  return check_codes(q.codes, q.ld_codes, q.scales, q.ld_scales, p->K, p->fmt);
}

// ------------------------------------------------------------------- norm
constexpr int kNormRows = 1 << 21;  // rows to a launch: a grid's threads count in 32 bits, up to 1024 to a row

// the rows from row t on
template <int DT>
moe::NormParams norm_from(const moe::NormParams& p, int64_t t) {
  moe::NormParams q = p;
  auto at = [&](const void* base, int64_t ld) { return base ? (uint8_t*)base + t * ld * moe::elem_size(DT) : nullptr; };
  q.x = at(p.x, p.ldx);
  q.res = at(p.res, p.ld_res);
  q.res_out = at(p.res_out, p.ld_res_out);
  q.y = at(p.y, p.ldy);
  q.codes = p.codes ? p.codes + t * p.ld_codes : nullptr;
  q.scales = p.scales ? p.scales + t * p.ld_scales : nullptr;
  return q;
}

template <int DT, int FMT>
void launch_norm(const moe::NormParams& q, int T, hipStream_t s) {
  if (T > kNormRows) {
    for (int t = 0; t < T; t += kNormRows) launch_norm<DT, FMT>(norm_from<DT>(q, t), std::min(T - t, kNormRows), s);
    return;
  }
  const int n8 = q.H / 8;
  const dim3 g((unsigned)T);
#define MOE_NORM(NT, C) hipLaunchKernelGGL((moe::k_add_rmsnorm<DT, FMT, NT, C>), g, dim3(NT), 0, s, q)
  if (n8 <= 64) MOE_NORM(64, 1);
  else if (n8 <= 128) MOE_NORM(128, 1);
  else if (n8 <= 256) MOE_NORM(256, 1);
  // Rows of more than 8192 values: two chunks to a thread (us, MXFP8 output, against four on 512 threads and
  // eight on 256): 1024 x 8224 17.4, 17.1 and 20.9, 4096 x 14336 80, 86 and 112, 4096 x 16384 91, 95 and 124.
  else if (n8 > 1024) MOE_NORM(1024, 2);
  else if (T <= 512) {
    // Too few rows to fill the card: a row's chunks side by side, against several to a thread as below
    // (us, MXFP8 output): 1 x 7168 4.1 and 5.7, 64 x 7168 4.4 and 6.0, 512 x 7168 7.8 and 8.3; 1024 x 7168 14.1 and 13.4,
    // 8192 x 7168 91 and 86 (y alone: 82 and 89), 1024 x 4096 the same.
    if (n8 <= 512) MOE_NORM(512, 1);
    else MOE_NORM(1024, 1);
  } else if (n8 <= 512) MOE_NORM(256, 2);
  else MOE_NORM(256, 4);
#undef MOE_NORM
}

// ------------------------------------------------------------------ linear
int mx_linear_params(const moe_mx_linear_problem* p, moe::mxl::Params& q, bool& exact) {
  if (!p || p->M < 0 || p->N <= 0 || p->K <= 0 || !type_ok(p->out_type) || !std::isfinite(p->alpha)) return MOE_EINVAL;
  if ((p->a_fmt != MOE_MX_FP4 && p->a_fmt != MOE_MX_FP8) || (p->exact != 0 && p->exact != 1)) return MOE_EINVAL;
  if (p->K % 32 || p->K > 1 << 20 || p->M >= kMaxRows || p->N >= kMaxRows) return MOE_ENOTSUP;
  const int64_t cb = moe::mxf::code_bytes(p->a_fmt, p->K);
  q.lda = or_default(p->lda, cb);
  q.ld_as = or_default(p->ld_as, p->K / 32);
  q.ldo = or_default(p->ldo, p->N);
  q.ld_add = or_default(p->ld_add, p->N);
  if (q.lda < cb || q.ld_as < p->K / 32 || q.ldo < p->N || q.ld_add < p->N) return MOE_EINVAL;
  if (q.lda % 16 || q.lda > 1 << 22 || q.ld_as > 1 << 22 || q.ldo > kMaxLd || q.ld_add > kMaxLd) return MOE_ENOTSUP;
  q.M = p->M;
  q.N = p->N;
  q.K = p->K;
  q.out_type = p->out_type;
  q.alpha = p->alpha;
  exact = p->a_fmt == MOE_MX_FP8 && (p->exact || p->out_type == MOE_T_FP32);
  return MOE_OK;
}

template <int AF, int BM, int BN, int BK, int NBUF>
int launch_tile(moe::mxl::Params& q, bool exact, hipStream_t s) {
  q.mt = (q.M + BM - 1) / BM;
  q.nt = (q.N + BN - 1) / BN;
  const int64_t n = ((int64_t)q.mt * q.nt + 7) / 8 * 8;
  if (n > kMaxGrid) return MOE_ENOTSUP;
  if constexpr (AF == moe::mxf::MXFP8 && NBUF == 4) {
    if (exact) {
      hipLaunchKernelGGL((moe::mxl::k_tile<AF, BM, BN, BK, NBUF, true>), dim3((unsigned)n), dim3(256), 0, s, q);
      return launch_status();
    }
  }
  hipLaunchKernelGGL((moe::mxl::k_tile<AF, BM, BN, BK, NBUF, false>), dim3((unsigned)n), dim3(256), 0, s, q);
  return launch_status();
}

template <int AF, int S, int FN, int FM, bool LITE>
int launch_skinny(moe::mxl::Params& q, bool exact, hipStream_t s) {
  q.nt = (q.N + 16 * FN - 1) / (16 * FN);
  q.mt = (q.M + 16 * FM - 1) / (16 * FM);
  const dim3 g((unsigned)(q.mt * q.nt));
  if constexpr (AF == moe::mxf::MXFP8) {
    if (exact) {
      hipLaunchKernelGGL((moe::mxl::k_skinny<AF, S, FN, FM, LITE, true>), g, dim3(64 * S), 0, s, q);
      return launch_status();
    }
  }
  hipLaunchKernelGGL((moe::mxl::k_skinny<AF, S, FN, FM, LITE, false>), g, dim3(64 * S), 0, s, q);
  return launch_status();
}

template <int AF>
int launch_linear(moe::mxl::Params& q, bool exact, hipStream_t s) {
  constexpr bool F8 = AF == moe::mxf::MXFP8;
  // Stages of 256 K values where they take the room of 128 MXFP8 ones: 300 x 7168 x 7168 MXFP4 27.5 -> 23.5,
  // 128 x 7168 x 7168 19.6 -> 15.4 (half the barriers, whole lines of a weight row); 64 x 128 and 64 x 64 MXFP8 gain
  // nothing (200 x 14336 x 4096 20.7 and 20.9, 512 x 4096 x 4096 12.9 and 13.8).
  constexpr int BM = F8 ? 128 : 256, BK = F8 ? 128 : 256;
  using moe::mxl::Kernel;
  switch (moe::mxl::choose(F8, exact, q.M, q.N, q.K)) {
    case Kernel::SKINNY_8_1_1_LITE: return launch_skinny<AF, 8, 1, 1, true>(q, exact, s);
    case Kernel::SKINNY_4_1_1_LITE: return launch_skinny<AF, 4, 1, 1, true>(q, exact, s);
    case Kernel::SKINNY_8_1_1: return launch_skinny<AF, 8, 1, 1, false>(q, exact, s);
    case Kernel::SKINNY_4_2_1: return launch_skinny<AF, 4, 2, 1, false>(q, exact, s);
    case Kernel::SKINNY_4_1_2: return launch_skinny<AF, 4, 1, 2, false>(q, exact, s);
    case Kernel::SKINNY_X_2_2: return launch_skinny<AF, F8 ? 2 : 4, 2, 2, false>(q, exact, s);
    case Kernel::TILE_LARGEST: return launch_tile<AF, BM, 256, BK, 2>(q, exact, s);
    case Kernel::TILE_128_128: return launch_tile<AF, 128, 128, BK, 4>(q, exact, s);
    case Kernel::TILE_64_128: return launch_tile<AF, 64, 128, BK, 4>(q, exact, s);
    case Kernel::TILE_64_64: return launch_tile<AF, 64, 64, BK, 4>(q, exact, s);
  }
  return MOE_EINVAL;
}

// ----------------------------------------------------------------- routing
// A token takes 16 lanes, four tokens to a wave, where tokens are many: us with 16 and with 64 lanes:
// 65536 x 256 softmax, top 8, 34 and 60, 16384 x 256 sigmoid in 8 groups 14.5 and 22, 65536 x 128 20 and 50, 4096 x 128
// 4.4 and 6.0, 4096 x 64 4.1 and 5.4. Up to 256 experts 16 lanes hold 16 each, and few tokens wait for that chain:
// 1 x 256 sigmoid in 8 groups 6.6 and 4.8, 2048 x 256 7.4 and 6.3, 4096 x 256 7.4 and 8.5; with 128 experts 16 lanes
// are not behind (1 x 128 3.7 and 3.7). Vector loads of 8 or more, against value by value: 65536 x 256 34 and 61,
// 1 x 128 3.7 and 5.1.
template <int DT>
void launch_route(const moe::RouteTopkParams& q, hipStream_t s) {
  const bool row16 = aligned(q.logits, 16) && aligned(q.bias, 16) && q.ld * moe::elem_size(DT) % 16 == 0;
#define MOE_ROUTE_TOPK(L, PER)                                                                              \
  {                                                                                                         \
    const dim3 g((unsigned)((q.T + 256 / L - 1) / (256 / L)));                                              \
    if (PER >= 8 && row16 && q.E % PER == 0)                                                                \
      hipLaunchKernelGGL((moe::k_route_topk<DT, L, PER, PER >= 8>), g, dim3(256), 0, s, q);                 \
    else                                                                                                    \
      hipLaunchKernelGGL((moe::k_route_topk<DT, L, PER, false>), g, dim3(256), 0, s, q);                    \
  }
  if (q.E <= 64) MOE_ROUTE_TOPK(16, 4)
  else if (q.E <= 128) MOE_ROUTE_TOPK(16, 8)
  else if (q.E <= 256 && q.T <= 2048) MOE_ROUTE_TOPK(64, 4)
  else if (q.E <= 256) MOE_ROUTE_TOPK(16, 16)
  else if (q.E <= 512) MOE_ROUTE_TOPK(64, 8)
  else MOE_ROUTE_TOPK(64, 16)
#undef MOE_ROUTE_TOPK
}

}  // namespace

extern "C" {

int moe_mx_quantize(const moe_mx_rows* p, const void* x, void* codes, uint8_t* scales, moe_stream_t stream) {
  moe::mxf::RowsParams q{};
  bool flat = false;
  int rc = rows_params(p, q, flat);
  if (rc) return rc;
  if (p->rows == 0) return MOE_OK;
  q.x = x;
  q.codes = (uint8_t*)codes;
  q.scales = scales;
  if ((rc = check_mx_rows(p, q, x))) return rc;
  hipStream_t s = (hipStream_t)stream;
  const dim3 g((q.n + 256 * moe::mxf::kUnroll - 1) / (256 * moe::mxf::kUnroll)), b(256);
  with_type(p->type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using namespace moe::mxf;
    if (p->fmt == MOE_MX_FP4) {
      if (flat) hipLaunchKernelGGL((k_quantize<DT, MXFP4, true>), g, b, 0, s, q);
      else hipLaunchKernelGGL((k_quantize<DT, MXFP4, false>), g, b, 0, s, q);
    } else {
      if (flat) hipLaunchKernelGGL((k_quantize<DT, MXFP8, true>), g, b, 0, s, q);
      else hipLaunchKernelGGL((k_quantize<DT, MXFP8, false>), g, b, 0, s, q);
    }
  });
  return launch_status();
}

int moe_mx_dequantize(const moe_mx_rows* p, const void* codes, const uint8_t* scales, void* out, moe_stream_t stream) {
  moe::mxf::RowsParams q{};
  bool flat = false;
  int rc = rows_params(p, q, flat);
  if (rc) return rc;
  if (p->rows == 0) return MOE_OK;
  q.out = out;
  q.codes = (uint8_t*)const_cast<void*>(codes);
  q.scales = const_cast<uint8_t*>(scales);
  if ((rc = check_mx_rows(p, q, out))) return rc;
  hipStream_t s = (hipStream_t)stream;
  const dim3 g((q.n + 256 * moe::mxf::kUnroll - 1) / (256 * moe::mxf::kUnroll)), b(256);
  with_type(p->type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using namespace moe::mxf;
    if (p->fmt == MOE_MX_FP4) {
      if (flat) hipLaunchKernelGGL((k_dequantize<DT, MXFP4, true>), g, b, 0, s, q);
      else hipLaunchKernelGGL((k_dequantize<DT, MXFP4, false>), g, b, 0, s, q);
    } else {
      if (flat) hipLaunchKernelGGL((k_dequantize<DT, MXFP8, true>), g, b, 0, s, q);
      else hipLaunchKernelGGL((k_dequantize<DT, MXFP8, false>), g, b, 0, s, q);
    }
  });
  return launch_status();
}

int moe_add_rmsnorm(const moe_norm_problem* p, const void* x, const void* residual, const void* weight,
                    void* residual_out, void* y, void* codes, uint8_t* scales, moe_stream_t stream) {
  if (!p || p->T < 0 || p->H <= 0 || !type_ok(p->type) || !type_ok(p->w_type)) return MOE_EINVAL;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return MOE_EINVAL;
  if (p->mx_fmt != MOE_MX_NONE && p->mx_fmt != MOE_MX_FP4 && p->mx_fmt != MOE_MX_FP8) return MOE_EINVAL;
  const bool mx = p->mx_fmt != MOE_MX_NONE;
  if (p->T >= kMaxRows || p->H > 16384 || p->H % (mx ? 32 : 8)) return MOE_ENOTSUP;
  if (p->T == 0) return MOE_OK;
  if (!x || !weight || !aligned(weight, 16) || !residual != !residual_out || (!y && !mx)) return MOE_EINVAL;
  moe::NormParams q{};
  q.x = x;
  q.res = residual;
  q.w = weight;
  q.res_out = residual_out;
  q.y = y;
  q.codes = mx ? (uint8_t*)codes : nullptr;
  q.scales = mx ? scales : nullptr;
  q.ldx = or_default(p->ldx, p->H);
  q.ld_res = or_default(p->ld_res, p->H);
  q.ld_res_out = or_default(p->ld_res_out, p->H);
  q.ldy = or_default(p->ldy, p->H);
  q.ld_codes = or_default(p->ld_codes, moe::mxf::code_bytes(p->mx_fmt, p->H));
  q.ld_scales = or_default(p->ld_scales, p->H / 32);
  q.H = p->H;
  q.w_type = p->w_type;
  q.eps = p->eps;
  q.inv_h = 1.0 / p->H;
  int rc = check_rows(x, q.ldx, p->H, p->type);
  if (!rc && residual) rc = check_rows(residual, q.ld_res, p->H, p->type);
  if (!rc && residual) rc = check_rows(residual_out, q.ld_res_out, p->H, p->type);
  if (!rc && y) rc = check_rows(y, q.ldy, p->H, p->type);
  if (!rc && mx) rc = check_codes(codes, q.ld_codes, scales, q.ld_scales, p->H, p->mx_fmt);
  if (rc) return rc;
  hipStream_t s = (hipStream_t)stream;
  with_type(p->type, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p->mx_fmt == MOE_MX_FP4) launch_norm<DT, moe::mxf::MXFP4>(q, p->T, s);
    else if (p->mx_fmt == MOE_MX_FP8) launch_norm<DT, moe::mxf::MXFP8>(q, p->T, s);
    else launch_norm<DT, 0>(q, p->T, s);
  });
  return launch_status();
}

int moe_mx_linear(const moe_mx_linear_problem* p, const void* a, const uint8_t* a_scales, const void* w,
                  const uint8_t* w_scales, const float* bias, const void* add, void* out, moe_stream_t stream) {
  moe::mxl::Params q{};
  bool exact = false;
  int rc = mx_linear_params(p, q, exact);
  if (rc) return rc;
  if (p->M == 0) return MOE_OK;
  if (!a || !a_scales || !w || !w_scales || !out) return MOE_EINVAL;
  const size_t size = (size_t)moe::elem_size(p->out_type);
  if (!aligned(bias, 4) || !aligned(out, size) || !aligned(add, size) || !aligned(a, 16) || !aligned(w, 16))
    return MOE_EINVAL;
  q.a = (const uint8_t*)a;
  q.a_sc = a_scales;
  q.w = (const uint8_t*)w;
  q.w_sc = w_scales;
  q.bias = bias;
  q.add = add;
  q.out = out;
  auto wide = [&](const void* t, int64_t ld) {
    return aligned(t, 16) && ld * (int64_t)size % 16 == 0 && ld * (int64_t)size < (int64_t)1 << 22;
  };
  q.vec = q.N % 8 == 0 && wide(out, q.ldo) && aligned(bias, 16) && (!add || wide(add, q.ld_add));
  hipStream_t s = (hipStream_t)stream;
  return p->a_fmt == MOE_MX_FP8 ? launch_linear<moe::mxf::MXFP8>(q, exact, s) : launch_linear<moe::mxf::MXFP4>(q, exact, s);
}

int moe_route_topk(const moe_route_topk_problem* p, const void* logits, const float* bias, int32_t* topk_ids,
                   float* topk_weights, moe_stream_t stream) {
  if (!p || p->T < 0 || p->E <= 0 || p->k <= 0 || p->k > p->E || !type_ok(p->type)) return MOE_EINVAL;
  if (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if (p->group_score != MOE_GROUP_MAX && p->group_score != MOE_GROUP_TOP2) return MOE_EINVAL;
  if (p->renormalize != 0 && p->renormalize != 1) return MOE_EINVAL;
  if (p->n_group < 0 || !std::isfinite(p->routed_scaling_factor)) return MOE_EINVAL;
  if (p->T >= kMaxRows || p->E > moe::kRouteMaxE || p->k > moe::kRouteMaxK || p->n_group > moe::kTopkGroups)
    return MOE_ENOTSUP;
  const bool grouped = p->n_group > 1;
  if (grouped && (p->E % p->n_group || p->topk_group < 1 || p->topk_group > p->n_group ||
                  (p->group_score == MOE_GROUP_TOP2 && p->E / p->n_group < 2) ||
                  (int64_t)p->k > (int64_t)p->topk_group * (p->E / p->n_group)))
    return MOE_EINVAL;
  const int64_t ld = or_default(p->ld, p->E);
  if (ld < p->E) return MOE_EINVAL;
  if (ld > kMaxLd) return MOE_ENOTSUP;
  if (p->T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_EINVAL;
  if (!aligned(logits, (size_t)moe::elem_size(p->type)) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(bias, 4))
    return MOE_EINVAL;
  moe::RouteTopkParams q;
  q.logits = logits;
  q.bias = bias;
  q.ids = topk_ids;
  q.w = topk_weights;
  q.ld = ld;
  q.T = p->T;
  q.E = p->E;
  q.k = p->k;
  q.sigmoid = p->score == MOE_SCORE_SIGMOID;
  q.n_group = grouped ? p->n_group : 0;
  q.topk_group = p->topk_group;
  q.per_group = grouped ? p->E / p->n_group : 0;
  q.top2 = p->group_score == MOE_GROUP_TOP2;
  q.renorm = p->renormalize;
  q.scale = p->routed_scaling_factor;
  hipStream_t s = (hipStream_t)stream;
  with_type(p->type, [&](auto dt) { launch_route<decltype(dt)::value>(q, s); });
  return launch_status();
}

}  // extern "C"
