// Internal interface of the 8-bit training operators: row codes (save, load),
// the 8-bit matrix product and the weight gradient from a checkpoint.  Host
// checks are in zs_q8.cpp, kernels in zs_q8_rows.hip and zs_q8_gemm.hip.  Not
// installed; not part of the ABI.
#pragma once

#include "zs_internal.h"

namespace zs {

// Leading dimensions are in elements of their own array.
struct Q8Save {
  const void* x;
  int64_t ld_x;
  const float* col_scale;  // NULL: none
  int8_t* codes;
  int64_t ld_codes;
  float* scales;
  int64_t rows, cols;
  int32_t format;  // ZS_FORMAT_* of x
  int32_t rule;    // ZS_Q8_SCALE_*
};

struct Q8Load {
  const int8_t* codes;
  int64_t ld_codes;
  const float* scales;
  void* out;
  int64_t ld_out;
  int64_t rows, cols;
  int32_t format;  // ZS_FORMAT_* of out
};

// d[m][n] = sum over k of the operands, by op:
//   kNT  a [M][K] codes, b [N][K] codes   int32 sum, times rs[m], times cs[n] (cs may be NULL)
//   kNN  a [M][K] codes, b [K][N] codes   the same
//   kTN  a [K][M] bf16 or fp16, b [K][N] codes times rs[k]   fp32 sum, plus add[m][n] (add may be NULL)
enum class Q8Op : int32_t { kNT = 0, kNN = 1, kTN = 2 };
struct Q8Gemm {
  const void* a;
  int64_t lda;
  const int8_t* b;
  int64_t ldb;
  const float* rs;
  const float* cs;
  const void* add;
  void* d;
  int64_t ldd;
  int64_t M, N, K;
  int32_t a_format;  // kTN: ZS_FORMAT_BF16 or ZS_FORMAT_FP16
  int32_t format;    // ZS_FORMAT_* of d (and add)
};

hipError_t launch_q8_save(const Q8Save& a, hipStream_t stream);
hipError_t launch_q8_load(const Q8Load& a, hipStream_t stream);
hipError_t launch_q8_gemm(Q8Op op, const Q8Gemm& a, hipStream_t stream);

// From zs_api.cpp: a status with its thread-local detail string ("" clears
// it), and the common end of a call that launched something.
zs_status api_fail(zs_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void api_clear();
zs_status api_after_launch(hipError_t e, hipStream_t stream, const char* what);

}  // namespace zs
