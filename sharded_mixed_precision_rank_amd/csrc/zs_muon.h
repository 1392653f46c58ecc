// Internal interface of the orthogonalised update: host checks are in
// zs_muon.cpp, kernels and the choice of tiles in zs_muon.hip.  Not installed;
// not part of the ABI.
#pragma once

#include <stddef.h>

#include "zs_internal.h"
#include "zs_muon_choice.h"

namespace zs {

constexpr int kMaxNsSteps = 32;
constexpr int64_t kMaxNsDim = 1 << 20;    // rows and columns
constexpr int64_t kMaxNsShort = 1 << 16;  // the shorter of the two
constexpr int64_t kMaxNsBatch = 65535;

// Where the matrices come from and go to.  Matrix i of the batch starts i *
// batch_ld elements on; `update` takes the place of x and out.
struct NsProblem {
  int64_t batch, rows, cols;
  int32_t steps;
  float coefs[3 * kMaxNsSteps];
  // orthogonalise: values in, values out
  const void* x;
  int32_t x_format;
  int64_t ld_x, batch_x;
  void* out;
  int32_t out_format;
  int64_t ld_out, batch_out;
  // update: replicas' mean and momentum in, master and working copy out (contiguous, rows * cols apart)
  bool update;
  const uint16_t* const* grads;  // host array of n_rep device pointers
  int32_t n_rep;
  int32_t nesterov;
  float mu, dk, ss;
  float* momentum;
  float* master;
  uint16_t* param;
};

size_t ns_workspace_bytes(int64_t rows, int64_t cols, int64_t batch);
hipError_t launch_ns(const NsProblem& p, void* workspace, hipStream_t stream);

// Matrices with sides of at most ns::kSmallSide, from values to values (zs_muon_small.hip).
hipError_t launch_ns_small(const NsProblem& p, hipStream_t stream);

}  // namespace zs
