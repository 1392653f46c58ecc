// C-ABI entry points of the orthogonalised update: argument checks and launches.
// The contract is in include/zshard.h; the kernels are in zs_muon.hip.
#include "zs_muon.h"

#include <cmath>

#include "zs_matrix_args.h"

namespace {

using namespace zs::args;
using zs::api_fail;

constexpr double kDefaultCoefs[3] = {3.4445, -4.7750, 2.0315};

zs_status check_shape(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || batch > zs::kMaxNsBatch)
    return api_fail(ZS_ERR_RANGE, "batch must be in [0, %lld] (got %lld)", (long long)zs::kMaxNsBatch, (long long)batch);
  for (const int64_t n : {rows, cols})
    if (n < 0 || n > zs::kMaxNsDim)
      return api_fail(ZS_ERR_RANGE, "rows and cols must be in [0, 2^20] (got %lld)", (long long)n);
  if (rows > zs::kMaxNsShort && cols > zs::kMaxNsShort)
    return api_fail(ZS_ERR_RANGE, "the smaller of rows and cols must be at most 2^16 (got %lld x %lld)", (long long)rows,
                    (long long)cols);
  return ZS_OK;
}

zs_status check_steps(int32_t steps, const double* coefs, float* to) {
  if (steps < 1 || steps > zs::kMaxNsSteps)
    return api_fail(ZS_ERR_RANGE, "steps must be in [1, %d] (got %d)", zs::kMaxNsSteps, steps);
  for (int i = 0; i < 3 * steps; ++i) {
    to[i] = (float)(coefs ? coefs[i] : kDefaultCoefs[i % 3]);
    if (!std::isfinite(to[i])) return api_fail(ZS_ERR_RANGE, "coefs[%d] is not a finite fp32 value", i);
  }
  return ZS_OK;
}

// Matrices of a batch as one region: the bytes between rows and between matrices count as theirs.
zs_status check_stack(const Region& flat, int64_t ld, int64_t batch_stride, int64_t batch, int64_t rows, int64_t cols, int align) {
  if (!flat.base) return api_fail(ZS_ERR_NULL, "%s is NULL", flat.name);
  if (flat.base % (uintptr_t)align) return api_fail(ZS_ERR_ALIGN, "%s must be %d-byte aligned", flat.name, align);
  if (rows > 1 && ld < cols)
    return api_fail(ZS_ERR_RANGE, "%s: the leading dimension must be at least the columns (got %lld for %lld)", flat.name,
                    (long long)ld, (long long)cols);
  if ((double)rows * (double)ld * 4.0 > kMaxBytes || (double)batch * (double)batch_stride * 4.0 > kMaxBytes)
    return api_fail(ZS_ERR_RANGE, "%s spans too many bytes (leading dimension %lld, batch stride %lld)", flat.name, (long long)ld,
                    (long long)batch_stride);
  if (batch > 1 && batch_stride < (rows - 1) * ld + cols)
    return api_fail(ZS_ERR_RANGE, "%s: the batch stride must hold a matrix (got %lld)", flat.name, (long long)batch_stride);
  return ZS_OK;
}
Region stack(const char* name, const void* p, int64_t ld, int64_t batch_stride, int64_t batch, int64_t rows, int64_t cols, int bytes) {
  const bool sane = (double)rows * (double)ld * 4.0 <= kMaxBytes && (double)batch * (double)batch_stride * 4.0 <= kMaxBytes;
  return Region{name, (uintptr_t)p, 1, sane ? ((batch - 1) * batch_stride + (rows - 1) * ld + cols) * bytes : 0, 0};
}

zs_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return api_fail(ZS_ERR_NULL, "workspace is NULL");
  if (bytes < need) return api_fail(ZS_ERR_RANGE, "workspace of %zu bytes is smaller than the %zu needed", bytes, need);
  return ZS_OK;
}

}  // namespace

extern "C" {

size_t zs_orthogonalize_workspace_bytes(int64_t rows, int64_t cols, int64_t batch) {
  zs::api_clear();
  if (check_shape(batch, rows, cols) != ZS_OK || batch == 0 || rows == 0 || cols == 0) return 0;
  return zs::ns_workspace_bytes(rows, cols, batch);
}

zs_status zs_orthogonalize(const void* x, int32_t x_format, int64_t ld_x, int64_t batch_stride_x, int64_t batch, int64_t rows,
                           int64_t cols, int32_t steps, const double* coefs, void* out, int32_t out_format, int64_t ld_out,
                           int64_t batch_stride_out, void* workspace, size_t workspace_bytes, zs_stream stream) {
  zs::api_clear();
  zs::NsProblem p{};
  ZS_TRY(check_shape(batch, rows, cols));
  ZS_TRY(check_format("x_format", x_format, true));
  ZS_TRY(check_format("out_format", out_format, true));
  ZS_TRY(check_steps(steps, coefs, p.coefs));
  if (batch == 0 || rows == 0 || cols == 0) return ZS_OK;
  if (rows == 1) ld_x = ld_out = cols;
  if (batch == 1) batch_stride_x = batch_stride_out = 0;
  const int xb = elem_bytes(x_format), ob = elem_bytes(out_format);
  const Region rx = stack("x", x, ld_x, batch_stride_x, batch, rows, cols, xb);
  const Region ro = stack("out", out, ld_out, batch_stride_out, batch, rows, cols, ob);
  ZS_TRY(check_stack(rx, ld_x, batch_stride_x, batch, rows, cols, xb));
  ZS_TRY(check_stack(ro, ld_out, batch_stride_out, batch, rows, cols, ob));
  const size_t need = zs::ns_workspace_bytes(rows, cols, batch);
  ZS_TRY(check_workspace(workspace, workspace_bytes, need));
  const Region rw{"workspace", (uintptr_t)workspace, 1, (int64_t)need, 0};
  ZS_TRY(check_disjoint(rw, rx));
  ZS_TRY(check_disjoint(rw, ro));
  // (x is read before out is written)
  if (!(x == out && xb == ob && ld_x == ld_out && batch_stride_x == batch_stride_out)) ZS_TRY(check_disjoint(ro, rx));
  p.batch = batch;
  p.rows = rows;
  p.cols = cols;
  p.steps = steps;
  p.x = x;
  p.x_format = x_format;
  p.ld_x = ld_x;
  p.batch_x = batch_stride_x;
  p.out = out;
  p.out_format = out_format;
  p.ld_out = ld_out;
  p.batch_out = batch_stride_out;
  return zs::api_after_launch(zs::launch_ns(p, workspace, (hipStream_t)stream), (hipStream_t)stream, "zs_orthogonalize");
}

zs_status zs_reduce_muon(const uint16_t* const* grad_chunks, int32_t N, int64_t batch, int64_t rows, int64_t cols, float* master,
                         float* momentum, uint16_t* param_bf16, const zs_muon_hp* hp, void* workspace, size_t workspace_bytes,
                         zs_stream stream) {
  zs::api_clear();
  zs::NsProblem p{};
  if (!hp) return api_fail(ZS_ERR_NULL, "hp is NULL");
  if (N < 1 || N > ZS_MAX_REPLICAS) return api_fail(ZS_ERR_RANGE, "N must be in [1, %d] (got %d)", ZS_MAX_REPLICAS, N);
  ZS_TRY(check_shape(batch, rows, cols));
  ZS_TRY(check_steps(hp->steps, hp->coefs, p.coefs));
  for (const double v : {hp->lr, hp->momentum, hp->weight_decay, hp->scale})
    if (!std::isfinite(v)) return api_fail(ZS_ERR_RANGE, "hyperparameters must be finite");
  if (hp->lr < 0 || hp->weight_decay < 0)
    return api_fail(ZS_ERR_RANGE, "lr and weight_decay must be >= 0 (got %g, %g)", hp->lr, hp->weight_decay);
  if (!(hp->momentum >= 0 && hp->momentum < 1)) return api_fail(ZS_ERR_RANGE, "momentum must be in [0, 1) (got %g)", hp->momentum);
  if (hp->nesterov != 0 && hp->nesterov != 1) return api_fail(ZS_ERR_RANGE, "nesterov must be 0 or 1 (got %d)", hp->nesterov);
  p.mu = (float)hp->momentum;
  p.dk = (float)(1.0 - hp->lr * hp->weight_decay);
  p.ss = (float)(hp->lr * hp->scale);
  // (an infinite factor would make NaN of an update of zeros)
  if (!std::isfinite(p.dk) || !std::isfinite(p.ss))
    return api_fail(ZS_ERR_RANGE, "lr * weight_decay and lr * scale must be fp32 values (got %g and %g)", hp->lr * hp->weight_decay,
                    hp->lr * hp->scale);
  if (batch == 0 || rows == 0 || cols == 0) return ZS_OK;
  const int64_t n = batch * rows * cols;
  if ((double)batch * (double)rows * (double)cols * 4.0 > kMaxBytes)
    return api_fail(ZS_ERR_RANGE, "batch * rows * cols is too large");
  if (!grad_chunks) return api_fail(ZS_ERR_NULL, "grad_chunks is NULL");
  const size_t need = zs::ns_workspace_bytes(rows, cols, batch);
  ZS_TRY(check_workspace(workspace, workspace_bytes, need));
  const Region written[4] = {{"master", (uintptr_t)master, 1, n * 4, 0},
                             {"momentum", (uintptr_t)momentum, 1, n * 4, 0},
                             {"param_bf16", (uintptr_t)param_bf16, 1, n * 2, 0},
                             {"workspace", (uintptr_t)workspace, 1, (int64_t)need, 0}};
  for (int i = 0; i < 3; ++i) {
    if (!written[i].base) return api_fail(ZS_ERR_NULL, "%s is NULL", written[i].name);
    if (written[i].base % (i < 2 ? 4 : 2)) return api_fail(ZS_ERR_ALIGN, "%s must be %d-byte aligned", written[i].name, i < 2 ? 4 : 2);
  }
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j) ZS_TRY(check_disjoint(written[i], written[j]));
  for (int r = 0; r < N; ++r) {
    const Region g{"a gradient", (uintptr_t)grad_chunks[r], 1, n * 2, 0};
    if (!g.base) return api_fail(ZS_ERR_NULL, "grad_chunks[%d] is NULL", r);
    if (g.base % 2) return api_fail(ZS_ERR_ALIGN, "grad_chunks[%d] must be 2-byte aligned", r);
    for (const Region& w : written) ZS_TRY(check_disjoint(w, g));
  }
  p.batch = batch;
  p.rows = rows;
  p.cols = cols;
  p.steps = hp->steps;
  p.update = true;
  p.grads = grad_chunks;
  p.n_rep = N;
  p.nesterov = hp->nesterov;
  p.momentum = momentum;
  p.master = master;
  p.param = param_bf16;
  return zs::api_after_launch(zs::launch_ns(p, workspace, (hipStream_t)stream), (hipStream_t)stream, "zs_reduce_muon");
}

}  // extern "C"
