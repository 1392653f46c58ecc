// C-ABI entry points of the 8-bit training operators: argument checks and
// launches.  The contract is in include/zshard.h; the kernels are in
// zs_q8_rows.hip and zs_q8_gemm.hip.
#include "zs_matrix_args.h"
#include "zs_q8.h"

namespace {

using namespace zs::args;
using zs::api_fail;

constexpr int64_t kMaxCodesK = 131071;          // 131071 * 128 * 128 < 2^31

}  // namespace

extern "C" {

zs_status zs_q8_save(const void* x, int32_t x_format, int64_t ld_x, int64_t rows, int64_t cols,
                     const float* col_scale, int32_t scale_rule, int8_t* codes, int64_t ld_codes, float* scales,
                     zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_dim("rows", rows));
  ZS_TRY(check_dim("cols", cols));
  ZS_TRY(check_format("x_format", x_format, true));
  if (scale_rule != ZS_Q8_SCALE_AMAX && scale_rule != ZS_Q8_SCALE_POW2)
    return api_fail(ZS_ERR_RANGE, "scale_rule must be ZS_Q8_SCALE_AMAX or ZS_Q8_SCALE_POW2 (got %d)", scale_rule);
  if (rows == 0) return ZS_OK;
  const int eb = elem_bytes(x_format);
  if (rows == 1) ld_x = ld_codes = cols;
  const Region rx = matrix("x", x, rows, cols, ld_x, eb), rq = matrix("codes", codes, rows, cols, ld_codes, 1);
  const Region rc = vector_of("col_scale", col_scale, cols), rs = vector_of("scales", scales, rows);
  ZS_TRY(check_vector(rs));
  if (cols > 0) {
    ZS_TRY(check_matrix(rx, ld_x, cols, eb));
    ZS_TRY(check_matrix(rq, ld_codes, cols, 1));
    if (col_scale) ZS_TRY(check_vector(rc));
    ZS_TRY(check_disjoint(rq, rx));
    ZS_TRY(check_disjoint(rq, rc));
    ZS_TRY(check_disjoint(rq, rs));
    ZS_TRY(check_disjoint(rs, rx));
    ZS_TRY(check_disjoint(rs, rc));
  }
  const zs::Q8Save a{x, ld_x, cols > 0 ? col_scale : nullptr, codes, ld_codes, scales, rows, cols, x_format, scale_rule};
  return zs::api_after_launch(zs::launch_q8_save(a, (hipStream_t)stream), (hipStream_t)stream, "zs_q8_save");
}

zs_status zs_q8_load(const int8_t* codes, int64_t ld_codes, const float* scales, int64_t rows, int64_t cols, void* out,
                     int32_t out_format, int64_t ld_out, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_dim("rows", rows));
  ZS_TRY(check_dim("cols", cols));
  ZS_TRY(check_format("out_format", out_format, true));
  if (rows == 0 || cols == 0) return ZS_OK;
  const int eb = elem_bytes(out_format);
  if (rows == 1) ld_out = ld_codes = cols;
  const Region rq = matrix("codes", codes, rows, cols, ld_codes, 1), ro = matrix("out", out, rows, cols, ld_out, eb);
  const Region rs = vector_of("scales", scales, rows);
  ZS_TRY(check_matrix(rq, ld_codes, cols, 1));
  ZS_TRY(check_vector(rs));
  ZS_TRY(check_matrix(ro, ld_out, cols, eb));
  ZS_TRY(check_disjoint(ro, rq));
  ZS_TRY(check_disjoint(ro, rs));
  const zs::Q8Load a{codes, ld_codes, scales, out, ld_out, rows, cols, out_format};
  return zs::api_after_launch(zs::launch_q8_load(a, (hipStream_t)stream), (hipStream_t)stream, "zs_q8_load");
}

zs_status zs_q8_matmul(const int8_t* x_codes, int64_t ld_x, const float* x_scales, const int8_t* w_codes, int64_t ld_w,
                       const float* w_scales, int64_t T, int64_t N, int64_t K, int32_t layout, void* y,
                       int32_t y_format, int64_t ld_y, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_dim("T", T));
  ZS_TRY(check_dim("N", N));
  ZS_TRY(check_dim("K", K));
  ZS_TRY(check_format("y_format", y_format, true));
  if (layout != ZS_Q8_XWT && layout != ZS_Q8_XW)
    return api_fail(ZS_ERR_RANGE, "layout must be ZS_Q8_XWT or ZS_Q8_XW (got %d)", layout);
  const bool nt = layout == ZS_Q8_XWT;
  const int64_t inner = nt ? K : N, outer = nt ? N : K;
  if (inner > kMaxCodesK)
    return api_fail(ZS_ERR_RANGE, "the summed axis must be at most %lld long, for sums exact in 32 bits (got %lld)",
                    (long long)kMaxCodesK, (long long)inner);
  if (T == 0 || outer == 0) return ZS_OK;
  const int eb = elem_bytes(y_format);
  if (T == 1) ld_x = inner, ld_y = outer;
  if (N == 1) ld_w = K;
  const Region rx = matrix("x_codes", x_codes, T, inner, ld_x, 1), rw = matrix("w_codes", w_codes, N, K, ld_w, 1);
  const Region ry = matrix("y", y, T, outer, ld_y, eb);
  const Region rsx = vector_of("x_scales", x_scales, T), rsw = vector_of("w_scales", w_scales, outer);
  if (inner > 0) {
    ZS_TRY(check_matrix(rx, ld_x, inner, 1));
    ZS_TRY(check_matrix(rw, ld_w, K, 1));
  }
  ZS_TRY(check_vector(rsx));
  if (w_scales) ZS_TRY(check_vector(rsw));
  ZS_TRY(check_matrix(ry, ld_y, outer, eb));
  for (const Region& r : {rx, rw, rsx, rsw}) ZS_TRY(check_disjoint(ry, r));
  zs::Q8Gemm a{};
  a.a = x_codes;
  a.lda = ld_x;
  a.b = w_codes;
  a.ldb = ld_w;
  a.rs = x_scales;
  a.cs = w_scales;
  a.d = y;
  a.ldd = ld_y;
  a.M = T;
  a.N = outer;
  a.K = inner;
  a.format = y_format;
  return zs::api_after_launch(zs::launch_q8_gemm(nt ? zs::Q8Op::kNT : zs::Q8Op::kNN, a, (hipStream_t)stream),
                              (hipStream_t)stream, "zs_q8_matmul");
}

zs_status zs_q8_weight_grad(const void* dy, int32_t dy_format, int64_t ld_dy, const int8_t* x_codes, int64_t ld_x,
                            const float* x_scales, int64_t T, int64_t N, int64_t K, const void* add, void* dw,
                            int32_t dw_format, int64_t ld_dw, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_dim("T", T));
  ZS_TRY(check_dim("N", N));
  ZS_TRY(check_dim("K", K));
  ZS_TRY(check_format("dy_format", dy_format, false));
  ZS_TRY(check_format("dw_format", dw_format, true));
  if (N == 0 || K == 0) return ZS_OK;
  const int eb = elem_bytes(dw_format);
  if (T <= 1) ld_dy = N, ld_x = K;
  if (N == 1) ld_dw = K;
  const Region rdy = matrix("dy", dy, T, N, ld_dy, 2), rx = matrix("x_codes", x_codes, T, K, ld_x, 1);
  const Region rdw = matrix("dw", dw, N, K, ld_dw, eb), radd = matrix("add", add, add ? N : 0, K, ld_dw, eb);
  const Region rs = vector_of("x_scales", x_scales, T);
  if (T > 0) {
    ZS_TRY(check_matrix(rdy, ld_dy, N, 2));
    ZS_TRY(check_matrix(rx, ld_x, K, 1));
    ZS_TRY(check_vector(rs));
  }
  ZS_TRY(check_matrix(rdw, ld_dw, K, eb));
  if (add) ZS_TRY(check_matrix(radd, ld_dw, K, eb));
  for (const Region& r : {rdy, rx, rs}) ZS_TRY(check_disjoint(rdw, r));
  if (add && add != dw) ZS_TRY(check_disjoint(rdw, radd));
  zs::Q8Gemm a{};
  a.a = dy;
  a.lda = ld_dy;
  a.b = x_codes;
  a.ldb = ld_x;
  a.rs = x_scales;
  a.add = add;
  a.d = dw;
  a.ldd = ld_dw;
  a.M = N;
  a.N = K;
  a.K = T;
  a.a_format = dy_format;
  a.format = dw_format;
  return zs::api_after_launch(zs::launch_q8_gemm(zs::Q8Op::kTN, a, (hipStream_t)stream), (hipStream_t)stream,
                              "zs_q8_weight_grad");
}

}  // extern "C"
