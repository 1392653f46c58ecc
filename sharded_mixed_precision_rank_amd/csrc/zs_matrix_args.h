// Checks of matrix arguments shared by the C-ABI front ends of the operators on
// matrices: dimensions, leading dimensions, alignment, which outputs share bytes
// with other operands.
#pragma once

#include "zs_internal.h"

namespace zs {

// From zs_api.cpp: a status with its thread-local detail string ("" clears
// it), and the common end of a call that launched something.
zs_status api_fail(zs_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void api_clear();
zs_status api_after_launch(hipError_t e, hipStream_t stream, const char* what);

namespace args {

constexpr int64_t kMaxDim = INT32_MAX;          // rows and columns
constexpr double kMaxBytes = 0x1p56;            // a matrix's extent

inline int elem_bytes(int32_t format) { return format == ZS_FORMAT_FP32 ? 4 : 2; }

// A matrix in memory: rows of `width` bytes, `pitch` bytes apart.
struct Region {
  const char* name;
  uintptr_t base;
  int64_t rows, width, pitch;
  uintptr_t end() const { return base + (uintptr_t)((rows - 1) * pitch + width); }
  bool empty() const { return rows == 0 || width == 0; }
};

// A leading dimension past 2^56 is refused by check_matrix; until then it must not overflow here.
inline Region matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  return Region{name, (uintptr_t)p, rows, cols * bytes, ld > (int64_t(1) << 56) ? 0 : ld * bytes};
}
inline Region vector_of(const char* name, const void* p, int64_t n) {
  return Region{name, (uintptr_t)p, 1, p ? n * 4 : 0, n * 4};
}

// Whether two matrices share a byte.  Column ranges of one buffer (the same
// pitch) may interleave without sharing any, and a single row (a vector too)
// may lie in a gap between a matrix's rows.  Matrices of several rows at
// different pitches count as sharing one where their ranges meet.
inline bool overlap(const Region& a, const Region& b) {
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

inline zs_status check_dim(const char* name, int64_t n) {
  if (n < 0 || n > kMaxDim) return api_fail(ZS_ERR_RANGE, "%s must be in [0, 2^31 - 1] (got %lld)", name, (long long)n);
  return ZS_OK;
}
// rows > 0 and cols > 0 here
inline zs_status check_matrix(const Region& r, int64_t ld, int64_t cols, int align) {
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
inline zs_status check_vector(const Region& r) {
  if (!r.base) return api_fail(ZS_ERR_NULL, "%s is NULL", r.name);
  if (r.base % 4) return api_fail(ZS_ERR_ALIGN, "%s must be 4-byte aligned", r.name);
  return ZS_OK;
}
inline zs_status check_disjoint(const Region& out, const Region& other) {
  if (overlap(out, other)) return api_fail(ZS_ERR_ALIAS, "%s overlaps %s", out.name, other.name);
  return ZS_OK;
}
inline zs_status check_format(const char* name, int32_t format, bool fp32) {
  if (format == ZS_FORMAT_BF16 || format == ZS_FORMAT_FP16 || (fp32 && format == ZS_FORMAT_FP32)) return ZS_OK;
  return api_fail(ZS_ERR_RANGE, "%s must be %s (got %d)", name,
                  fp32 ? "ZS_FORMAT_BF16, ZS_FORMAT_FP16 or ZS_FORMAT_FP32" : "ZS_FORMAT_BF16 or ZS_FORMAT_FP16", format);
}

#define ZS_TRY(call)                \
  do {                              \
    const zs_status st_ = (call);   \
    if (st_ != ZS_OK) return st_;   \
  } while (0)

}  // namespace args
}  // namespace zs
