// The elementwise half of the gated block's backward pass:
//   dgate = dh * up * act'(gate),  dup = dh * act(gate),  and h = act(gate) * up again where it is asked for
// (instead of keeping it).  Bound by memory: 10 bytes a value, 12 with h (8192 x
// 11008 in bf16: 142-151 us, 6.1 TB/s, as a plain copy), but for gelu, by its error
// function (among others 168-189 us, where the rest take 157-161).  A
// thread takes 8 consecutive columns; the hardware takes vector accesses at any
// address, so rows need no alignment, and an output may lie on the input of the
// same place: a thread has read its 8 values before it writes them.
#include "zs_act.h"
#include "zs_glu.h"
#include "zs_q8_dev.h"

namespace zs {
namespace {

using namespace dev;

template <int FMT, int ACT>
__device__ __forceinline__ void gate_grads(const float (&dh)[8], const float (&gate)[8], const float (&up)[8], float (&dg)[8],
                                           float (&du)[8], float (&h)[8]) {
  float value[8], slope[8];
  acts_of<ACT, true, 8>(gate, value, slope);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    dg[k] = dh[k] * up[k] * slope[k];
    du[k] = dh[k] * value[k];
    h[k] = value[k] * up[k];
  }
}

template <int FMT>
__device__ __forceinline__ void widen(u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[2 * k] = h_lo<FMT>(w[k]), v[2 * k + 1] = h_hi<FMT>(w[k]);
}
template <int FMT>
__device__ __forceinline__ u32x4 narrow(const float (&v)[8]) {
  return (u32x4){pack_two<FMT>(v[0], v[1]), pack_two<FMT>(v[2], v[3]), pack_two<FMT>(v[4], v[5]), pack_two<FMT>(v[6], v[7])};
}

template <int FMT, int ACT, class I>
__global__ __launch_bounds__(256) void glu_rows(const GluRows a, I per, I pieces) {
  const I stride = (I)gridDim.x * 256;
  for (I p = (I)blockIdx.x * 256 + threadIdx.x; p < pieces; p += stride) {
    const int64_t row = (int64_t)(p / per), col = (int64_t)(p % per) * 8;
    const int64_t at_dh = row * a.ld_dh + col, at_gu = row * a.ld_gu + col, at_d = row * a.ld_d + col;
    const int n = a.cols - col < 8 ? (int)(a.cols - col) : 8;
    float dh[8], gate[8], up[8], dg[8], du[8], h[8];
    if (n == 8) {
      widen<FMT>(ld_any<u32x4>((const uint16_t*)a.dh + at_dh), dh);
      widen<FMT>(ld_any<u32x4>((const uint16_t*)a.gate + at_gu), gate);
      widen<FMT>(ld_any<u32x4>((const uint16_t*)a.up + at_gu), up);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dh[k] = k < n ? ld_elem<FMT>(a.dh, at_dh + k) : 0.0f;
        gate[k] = k < n ? ld_elem<FMT>(a.gate, at_gu + k) : 0.0f;
        up[k] = k < n ? ld_elem<FMT>(a.up, at_gu + k) : 0.0f;
      }
    }
    gate_grads<FMT, ACT>(dh, gate, up, dg, du, h);
    if (n == 8) {
      st_any((uint16_t*)a.dgate + at_d, narrow<FMT>(dg));
      st_any((uint16_t*)a.dup + at_d, narrow<FMT>(du));
      if (a.h != nullptr) st_any((uint16_t*)a.h + row * a.ld_h + col, narrow<FMT>(h));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= n) continue;
        st_elem<FMT>(a.dgate, at_d + k, dg[k]);
        st_elem<FMT>(a.dup, at_d + k, du[k]);
        if (a.h != nullptr) st_elem<FMT>(a.h, row * a.ld_h + col + k, h[k]);
      }
    }
  }
}

template <int FMT, int ACT>
hipError_t rows_launch(const GluRows& given, hipStream_t stream) {
  GluRows a = given;
  // rows back to back are one long row
  if (a.ld_dh == a.cols && a.ld_gu == a.cols && a.ld_d == a.cols && (a.h == nullptr || a.ld_h == a.cols)) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  const int64_t per = (a.cols + 7) / 8, pieces = a.rows * per;
  const int64_t blocks = (pieces + 255) / 256;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  // (32-bit indices: a thread's last step must not pass 2^32)
  if (pieces < (int64_t(1) << 31))
    glu_rows<FMT, ACT, uint32_t><<<grid, 256, 0, stream>>>(a, (uint32_t)per, (uint32_t)pieces);
  else
    glu_rows<FMT, ACT, int64_t><<<grid, 256, 0, stream>>>(a, per, pieces);
  return hipGetLastError();
}

template <int FMT>
hipError_t by_act(const GluRows& a, hipStream_t stream) {
  switch (a.act) {
    case ZS_ACT_SILU: return rows_launch<FMT, ZS_ACT_SILU>(a, stream);
    case ZS_ACT_GELU: return rows_launch<FMT, ZS_ACT_GELU>(a, stream);
    case ZS_ACT_GELU_TANH: return rows_launch<FMT, ZS_ACT_GELU_TANH>(a, stream);
    default: return rows_launch<FMT, ZS_ACT_RELU>(a, stream);
  }
}

}  // namespace

hipError_t launch_glu_rows(const GluRows& a, hipStream_t stream) {
  return a.format == ZS_FORMAT_BF16 ? by_act<kBF16>(a, stream) : by_act<kFP16>(a, stream);
}

}  // namespace zs
