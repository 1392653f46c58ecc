// Internal interface of the gated feed-forward block: host checks are in
// zs_glu.cpp, kernels in zs_glu_gemm.hip (products) and zs_glu_rows.hip
// (elementwise gradients).  Not installed; not part of the ABI.
#pragma once

#include "zs_glu_choice.h"
#include "zs_internal.h"

namespace zs {

// Leading dimensions are in elements of their own array.
struct GluGemm {
  const void* a[2];
  int64_t lda;
  const void* b[2];
  int64_t ldb;
  const void* add[2];
  void* out[3];
  int64_t ldo[3];
  int64_t M, N, K;
  int32_t format;      // ZS_FORMAT_BF16 or ZS_FORMAT_FP16 of the operands
  int32_t out_format;  // kWeight: ZS_FORMAT_* of out and add; otherwise format
  int32_t act;         // kForward: ZS_ACT_*
};

struct GluRows {
  const void *dh, *gate, *up;
  void *dgate, *dup, *h;  // h: NULL for none
  int64_t ld_dh, ld_gu, ld_d, ld_h;
  int64_t rows, cols;
  int32_t format, act;
};

hipError_t launch_glu_gemm(GluOp op, const GluGemm& a, hipStream_t stream);
hipError_t launch_glu_rows(const GluRows& a, hipStream_t stream);

}  // namespace zs
