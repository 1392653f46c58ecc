// C-ABI entry points of the 8-bit training operators: argument checks and
// launches.  The contract is in include/zshard.h; the kernels are in
// zs_q8_rows.hip and zs_q8_gemm.hip.
#include "zs_q8.h"

namespace {

using zs::api_fail;

constexpr int64_t kMaxDim = INT32_MAX;          // rows and columns
constexpr double kMaxBytes = 0x1p56;            // a matrix's extent
constexpr int64_t kMaxCodesK = 131071;          // 131071 * 128 * 128 < 2^31

int elem_bytes(int32_t format) { return format == ZS_FORMAT_FP32 ? 4 : 2; }

// A matrix in memory: rows of `width` bytes, `pitch` bytes apart.
struct Region {
  const char* name;
  uintptr_t base;
  int64_t rows, width, pitch;
  uintptr_t end() const { return base + (uintptr_t)((rows - 1) * pitch + width); }
  bool empty() const { return rows == 0 || width == 0; }
};

// A leading dimension past 2^56 is refused by check_matrix; until then it must not overflow here.
Region matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  return Region{name, (uintptr_t)p, rows, cols * bytes, ld > (int64_t(1) << 56) ? 0 : ld * bytes};
}
Region vector_of(const char* name, const void* p, int64_t n) {
  return Region{name, (uintptr_t)p, 1, p ? n * 4 : 0, n * 4};
}

// Whether two matrices share a byte.  Column ranges of one buffer (the same
// pitch) may interleave without sharing any, and a single row (a vector too)
// may lie in a gap between a matrix's rows.  Matrices of several rows at
// different pitches count as sharing one where their ranges meet.
bool overlap(const Region& a, const Region& b) {
  if (a.empty() || b.empty() || a.end() <= b.base || b.end() <= a.base) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const Region &many = a.rows > 1 ? a : b, &other = a.rows > 1 ? b : a;
  const uintptr_t p = (uintptr_t)many.pitch;
  // where the other begins in the rows' period: behind a row's bytes, with its own ending before the next?
  const int64_t d = (int64_t)(many.base < other.base ? (other.base - many.base) % p
                                                     : (p - (many.base - other.base) % p) % p);
  return !(d >= many.width && d + other.width <= many.pitch);
}

zs_status check_dim(const char* name, int64_t n) {
  if (n < 0 || n > kMaxDim) return api_fail(ZS_ERR_RANGE, "%s must be in [0, 2^31 - 1] (got %lld)", name, (long long)n);
  return ZS_OK;
}
// rows > 0 and cols > 0 here
zs_status check_matrix(const Region& r, int64_t ld, int64_t cols, int align) {
  if (!r.base) return api_fail(ZS_ERR_NULL, "%s is NULL", r.name);
  if (r.rows > 1 && ld < cols)
    return api_fail(ZS_ERR_RANGE, "%s: the leading dimension must be at least the columns (got %lld for %lld)", r.name,
                    (long long)ld, (long long)cols);
  if ((double)r.rows * (double)ld * 4.0 > kMaxBytes)
    return api_fail(ZS_ERR_RANGE, "%s spans too many bytes (%lld rows, leading dimension %lld)", r.name,
                    (long long)r.rows, (long long)ld);
  if (r.base % (uintptr_t)align) return api_fail(ZS_ERR_ALIGN, "%s must be %d-byte aligned", r.name, align);
  return ZS_OK;
}
zs_status check_vector(const Region& r) {
  if (!r.base) return api_fail(ZS_ERR_NULL, "%s is NULL", r.name);
  if (r.base % 4) return api_fail(ZS_ERR_ALIGN, "%s must be 4-byte aligned", r.name);
  return ZS_OK;
}
zs_status check_disjoint(const Region& out, const Region& other) {
  if (overlap(out, other)) return api_fail(ZS_ERR_ALIAS, "%s overlaps %s", out.name, other.name);
  return ZS_OK;
}
zs_status check_format(const char* name, int32_t format, bool fp32) {
  if (format == ZS_FORMAT_BF16 || format == ZS_FORMAT_FP16 || (fp32 && format == ZS_FORMAT_FP32)) return ZS_OK;
  return api_fail(ZS_ERR_RANGE, "%s must be %s (got %d)", name,
                  fp32 ? "ZS_FORMAT_BF16, ZS_FORMAT_FP16 or ZS_FORMAT_FP32" : "ZS_FORMAT_BF16 or ZS_FORMAT_FP16", format);
}

#define ZS_TRY(call)                \
  do {                              \
    const zs_status st_ = (call);   \
    if (st_ != ZS_OK) return st_;   \
  } while (0)

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
