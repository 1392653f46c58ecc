// C-ABI entry points of the gated feed-forward block: argument checks and
// launches.  The contract is in include/zshard.h; the kernels are in
// zs_glu_gemm.hip and zs_glu_rows.hip.
#include "zs_glu.h"
#include "zs_matrix_args.h"

namespace {

using namespace zs::args;
using zs::api_fail;

zs_status check_act(int32_t act) {
  if (act >= ZS_ACT_SILU && act <= ZS_ACT_RELU) return ZS_OK;
  return api_fail(ZS_ERR_RANGE, "act must be ZS_ACT_SILU, ZS_ACT_GELU, ZS_ACT_GELU_TANH or ZS_ACT_RELU (got %d)", act);
}
zs_status check_sizes(int64_t T, int64_t N, int64_t K) {
  ZS_TRY(check_dim("T", T));
  ZS_TRY(check_dim("N", N));
  return check_dim("K", K);
}
// An output on the input of the same place, which the elementwise kernel allows.
bool same(const Region& a, const Region& b) { return a.base == b.base && (a.pitch == b.pitch || a.rows == 1); }

}  // namespace

extern "C" {

zs_status zs_glu_forward(const void* x, int64_t ld_x, const void* w_gate, const void* w_up, int64_t ld_w, int32_t format,
                         int64_t T, int64_t N, int64_t K, int32_t act, void* h, int64_t ld_h, void* gate, void* up,
                         int64_t ld_gu, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_sizes(T, N, K));
  ZS_TRY(check_format("format", format, false));
  ZS_TRY(check_act(act));
  if (!gate != !up) return api_fail(ZS_ERR_NULL, "gate and up must be given together");
  if (T == 0 || N == 0) return ZS_OK;
  if (T == 1) ld_x = K, ld_h = ld_gu = N;
  if (N == 1) ld_w = K;
  const Region rx = matrix("x", x, T, K, ld_x, 2), rg = matrix("w_gate", w_gate, N, K, ld_w, 2);
  const Region ru = matrix("w_up", w_up, N, K, ld_w, 2), rh = matrix("h", h, T, N, ld_h, 2);
  const Region rkg = matrix("gate", gate, gate ? T : 0, N, ld_gu, 2), rku = matrix("up", up, up ? T : 0, N, ld_gu, 2);
  if (K > 0) {
    ZS_TRY(check_matrix(rx, ld_x, K, 2));
    ZS_TRY(check_matrix(rg, ld_w, K, 2));
    ZS_TRY(check_matrix(ru, ld_w, K, 2));
  }
  ZS_TRY(check_matrix(rh, ld_h, N, 2));
  if (gate) {
    ZS_TRY(check_matrix(rkg, ld_gu, N, 2));
    ZS_TRY(check_matrix(rku, ld_gu, N, 2));
  }
  for (const Region& o : {rh, rkg, rku})
    for (const Region& r : {rx, rg, ru}) ZS_TRY(check_disjoint(o, r));
  ZS_TRY(check_disjoint(rh, rkg));
  ZS_TRY(check_disjoint(rh, rku));
  ZS_TRY(check_disjoint(rkg, rku));
  zs::GluGemm a{};
  a.a[0] = x;
  a.lda = ld_x;
  a.b[0] = w_gate;
  a.b[1] = w_up;
  a.ldb = ld_w;
  a.out[0] = h;
  a.out[1] = gate;
  a.out[2] = up;
  a.ldo[0] = ld_h;
  a.ldo[1] = a.ldo[2] = ld_gu;
  a.M = T;
  a.N = N;
  a.K = K;
  a.format = a.out_format = format;
  a.act = act;
  return zs::api_after_launch(zs::launch_glu_gemm(zs::GluOp::kForward, a, (hipStream_t)stream), (hipStream_t)stream,
                              "zs_glu_forward");
}

zs_status zs_glu_backward(const void* dh, int64_t ld_dh, const void* gate, const void* up, int64_t ld_gu, int32_t format,
                          int64_t T, int64_t N, int32_t act, void* dgate, void* dup, int64_t ld_d, void* h, int64_t ld_h,
                          zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_sizes(T, N, 0));
  ZS_TRY(check_format("format", format, false));
  ZS_TRY(check_act(act));
  if (T == 0 || N == 0) return ZS_OK;
  if (T == 1) ld_dh = ld_gu = ld_d = ld_h = N;
  const Region rdh = matrix("dh", dh, T, N, ld_dh, 2), rg = matrix("gate", gate, T, N, ld_gu, 2);
  const Region ru = matrix("up", up, T, N, ld_gu, 2), rdg = matrix("dgate", dgate, T, N, ld_d, 2);
  const Region rdu = matrix("dup", dup, T, N, ld_d, 2), rh = matrix("h", h, h ? T : 0, N, ld_h, 2);
  ZS_TRY(check_matrix(rdh, ld_dh, N, 2));
  ZS_TRY(check_matrix(rg, ld_gu, N, 2));
  ZS_TRY(check_matrix(ru, ld_gu, N, 2));
  ZS_TRY(check_matrix(rdg, ld_d, N, 2));
  ZS_TRY(check_matrix(rdu, ld_d, N, 2));
  if (h) ZS_TRY(check_matrix(rh, ld_h, N, 2));
  if (!same(rdg, rg)) ZS_TRY(check_disjoint(rdg, rg));
  ZS_TRY(check_disjoint(rdg, rdh));
  ZS_TRY(check_disjoint(rdg, ru));
  if (!same(rdu, ru)) ZS_TRY(check_disjoint(rdu, ru));
  ZS_TRY(check_disjoint(rdu, rdh));
  ZS_TRY(check_disjoint(rdu, rg));
  if (!same(rh, rdh)) ZS_TRY(check_disjoint(rh, rdh));
  ZS_TRY(check_disjoint(rh, rg));
  ZS_TRY(check_disjoint(rh, ru));
  ZS_TRY(check_disjoint(rdg, rdu));
  ZS_TRY(check_disjoint(rh, rdg));
  ZS_TRY(check_disjoint(rh, rdu));
  const zs::GluRows a{dh, gate, up, dgate, dup, h, ld_dh, ld_gu, ld_d, ld_h, T, N, format, act};
  return zs::api_after_launch(zs::launch_glu_rows(a, (hipStream_t)stream), (hipStream_t)stream, "zs_glu_backward");
}

zs_status zs_glu_input_grad(const void* dgate, const void* dup, int64_t ld_d, const void* w_gate, const void* w_up, int64_t ld_w,
                            int32_t format, int64_t T, int64_t N, int64_t K, void* dx, int64_t ld_dx, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_sizes(T, N, K));
  ZS_TRY(check_format("format", format, false));
  if (T == 0 || K == 0) return ZS_OK;
  if (T == 1) ld_d = N, ld_dx = K;
  if (N == 1) ld_w = K;
  const Region rdg = matrix("dgate", dgate, T, N, ld_d, 2), rdu = matrix("dup", dup, T, N, ld_d, 2);
  const Region rg = matrix("w_gate", w_gate, N, K, ld_w, 2), ru = matrix("w_up", w_up, N, K, ld_w, 2);
  const Region rdx = matrix("dx", dx, T, K, ld_dx, 2);
  if (N > 0) {
    ZS_TRY(check_matrix(rdg, ld_d, N, 2));
    ZS_TRY(check_matrix(rdu, ld_d, N, 2));
    ZS_TRY(check_matrix(rg, ld_w, K, 2));
    ZS_TRY(check_matrix(ru, ld_w, K, 2));
  }
  ZS_TRY(check_matrix(rdx, ld_dx, K, 2));
  for (const Region& r : {rdg, rdu, rg, ru}) ZS_TRY(check_disjoint(rdx, r));
  zs::GluGemm a{};
  a.a[0] = dgate;
  a.a[1] = dup;
  a.lda = ld_d;
  a.b[0] = w_gate;
  a.b[1] = w_up;
  a.ldb = ld_w;
  a.out[0] = dx;
  a.ldo[0] = ld_dx;
  a.M = T;
  a.N = K;
  a.K = N;
  a.format = a.out_format = format;
  return zs::api_after_launch(zs::launch_glu_gemm(zs::GluOp::kInput, a, (hipStream_t)stream), (hipStream_t)stream,
                              "zs_glu_input_grad");
}

zs_status zs_glu_weight_grad(const void* dgate, const void* dup, int64_t ld_d, const void* x, int64_t ld_x, int32_t format,
                             int64_t T, int64_t N, int64_t K, const void* add_gate, const void* add_up, void* dw_gate,
                             void* dw_up, int32_t dw_format, int64_t ld_dw, zs_stream stream) {
  zs::api_clear();
  ZS_TRY(check_sizes(T, N, K));
  ZS_TRY(check_format("format", format, false));
  ZS_TRY(check_format("dw_format", dw_format, true));
  if (!add_gate != !add_up) return api_fail(ZS_ERR_NULL, "add_gate and add_up must be given together");
  if (N == 0 || K == 0) return ZS_OK;
  const int eb = elem_bytes(dw_format);
  if (T <= 1) ld_d = N, ld_x = K;
  if (N == 1) ld_dw = K;
  const Region rdg = matrix("dgate", dgate, T, N, ld_d, 2), rdu = matrix("dup", dup, T, N, ld_d, 2);
  const Region rx = matrix("x", x, T, K, ld_x, 2);
  const Region rog = matrix("dw_gate", dw_gate, N, K, ld_dw, eb), rou = matrix("dw_up", dw_up, N, K, ld_dw, eb);
  const Region rag = matrix("add_gate", add_gate, add_gate ? N : 0, K, ld_dw, eb);
  const Region rau = matrix("add_up", add_up, add_up ? N : 0, K, ld_dw, eb);
  if (T > 0) {
    ZS_TRY(check_matrix(rdg, ld_d, N, 2));
    ZS_TRY(check_matrix(rdu, ld_d, N, 2));
    ZS_TRY(check_matrix(rx, ld_x, K, 2));
  }
  ZS_TRY(check_matrix(rog, ld_dw, K, eb));
  ZS_TRY(check_matrix(rou, ld_dw, K, eb));
  if (add_gate) {
    ZS_TRY(check_matrix(rag, ld_dw, K, eb));
    ZS_TRY(check_matrix(rau, ld_dw, K, eb));
  }
  ZS_TRY(check_disjoint(rog, rou));
  for (const Region& o : {rog, rou})
    for (const Region& r : {rdg, rdu, rx}) ZS_TRY(check_disjoint(o, r));
  if (add_gate != dw_gate) ZS_TRY(check_disjoint(rog, rag));
  if (add_up != dw_up) ZS_TRY(check_disjoint(rou, rau));
  ZS_TRY(check_disjoint(rog, rau));
  ZS_TRY(check_disjoint(rou, rag));
  zs::GluGemm a{};
  a.a[0] = dgate;
  a.a[1] = dup;
  a.lda = ld_d;
  a.b[0] = x;
  a.ldb = ld_x;
  a.add[0] = add_gate;
  a.add[1] = add_up;
  a.out[0] = dw_gate;
  a.out[1] = dw_up;
  a.ldo[0] = a.ldo[1] = ld_dw;
  a.M = N;
  a.N = K;
  a.K = T;
  a.format = format;
  a.out_format = dw_format;
  return zs::api_after_launch(zs::launch_glu_gemm(zs::GluOp::kWeight, a, (hipStream_t)stream), (hipStream_t)stream,
                              "zs_glu_weight_grad");
}

}  // extern "C"
