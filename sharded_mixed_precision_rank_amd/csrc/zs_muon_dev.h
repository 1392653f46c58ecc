// Device helpers of the orthogonalised update: matrices held as two fp16 parts,
// the momentum's step, where the last values go.
#pragma once

#include "zs_muon.h"
#include "zs_tile_dev.h"

namespace zs {
namespace ns {

using namespace dev;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kUnit = 4096.0f;           // held values are this times the matrix's
constexpr float kPerUnit = 1.0f / 4096.0f;
constexpr int kMostPartials = 1024;        // sums of squares of a matrix

struct MeanArgs {
  const uint16_t* g[ZS_MAX_REPLICAS];
  float* momentum;
  float* u;
  double* partials;
  int64_t n;  // values of a matrix
  int32_t n_rep, nesterov;
  float mu;
};

__device__ __forceinline__ float mean_step(float s, float m, const MeanArgs& a, float& m1) {
  const float g = s / (float)a.n_rep;
  m1 = a.mu * m + g;
  return a.nesterov ? g + a.mu * m1 : m1;
}

template <int FMT>
__device__ __forceinline__ void load8(const void* x, int64_t i, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (FMT == kFP32) {
      const f32x4 a = ld_any<f32x4>((const float*)x + i), b = ld_any<f32x4>((const float*)x + i + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
    } else {
      const u32x4 w = ld_any<u32x4>((const uint16_t*)x + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[2 * k] = h_lo<FMT>(w[k]), v[2 * k + 1] = h_hi<FMT>(w[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < left ? ld_elem<FMT>(x, i + k) : 0.0f;
  }
}
// v - h and by h + v, one instruction each that takes the fp16 value as it is (by a constant -1 it would be widened and
// subtracted).
__device__ __forceinline__ float less(float v, _Float16 h) {
  float minus = -1.0f;
  asm("" : "+s"(minus));
  return __builtin_fmaf((float)h, minus, v);
}
__device__ __forceinline__ float plus(float v, float by, _Float16 h) { return __builtin_fmaf((float)h, by, v); }
// Eight values as their parts.  (A product that the compiler folds into the conversion to hi is no matter: lo is what is
// left of the fp32 value.)
__device__ __forceinline__ void to_parts(const float* t, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f16x2 h = __builtin_convertvector((f32x2){t[2 * k], t[2 * k + 1]}, f16x2);
    const f16x2 l = __builtin_convertvector((f32x2){less(t[2 * k], h[0]), less(t[2 * k + 1], h[1])}, f16x2);
    hi[k] = __builtin_bit_cast(uint32_t, h);
    lo[k] = __builtin_bit_cast(uint32_t, l);
  }
}
// Eight held values from column col (a multiple of 8) of a row of parts.
__device__ __forceinline__ int64_t part_at(int64_t col) { return col / 32 * 128 + col % 32 * 2; }
__device__ __forceinline__ void store_parts(char* row, int64_t col, const float* t) {
  u32x4 hi, lo;
  to_parts(t, hi, lo);
  GLB char* p = (GLB char*)row + part_at(col);
  *(GLB u32x4*)p = hi;
  *(GLB u32x4*)(p + 64) = lo;
}
// t[k] += by times eight values held in parts, lo before hi.
__device__ __forceinline__ void add_parts(u32x4 hi, u32x4 lo, float by, float* t) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t two_hi = hi[k], two_lo = lo[k];  // (a bit cast of hi[k] itself takes hi[0])
    const f16x2 h = __builtin_bit_cast(f16x2, two_hi), l = __builtin_bit_cast(f16x2, two_lo);
#pragma unroll
    for (int r = 0; r < 2; ++r) t[2 * k + r] = plus(plus(t[2 * k + r], by, l[r]), by, h[r]);
  }
}

__device__ __forceinline__ f32x4 mfma_f16(i32x4 b, i32x4 a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}

// Where the last step's values go: out, or the update of master and param.
struct NsLast {
  int32_t turned, update;
  int64_t rows, cols;  // of the user's matrix
  void* out;
  int32_t out_format;
  int64_t ld_out, batch_out;
  float* master;
  uint16_t* param;
  float dk, ss;
};
// Eight held values of the last X, at row `row` from column `col` of the user's matrix.
template <int FMT>
__device__ __forceinline__ void store_values(const NsLast& a, int64_t batch, int64_t row, int64_t col, const float* t) {
  const int64_t i = batch * a.batch_out + row * a.ld_out + col;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = t[k] * kPerUnit;
  if (col + 8 <= a.cols) {
    st_four<FMT>(a.out, i, v);
    st_four<FMT>(a.out, i + 4, v + 4);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + k < a.cols) st_elem<FMT>(a.out, i + k, v[k]);
  }
}
__device__ __forceinline__ void store_update(const NsLast& a, int64_t batch, int64_t row, int64_t col, const float* t) {
  const int64_t i = batch * a.batch_out + row * a.ld_out + col;
  if (col + 8 <= a.cols) {
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4 p = ld_any<f32x4>(a.master + i + q);
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = a.dk * p[k] - a.ss * (t[q + k] * kPerUnit);
      st_four<kFP32>(a.master, i + q, v);
      st_four<kBF16>(a.param, i + q, v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (col + k >= a.cols) continue;
      const float v = a.dk * ((const GLB float*)a.master)[i + k] - a.ss * (t[k] * kPerUnit);
      st_elem<kFP32>(a.master, i + k, v);
      st_elem<kBF16>(a.param, i + k, v);
    }
  }
}
__device__ __forceinline__ void store_last(const NsLast& a, int64_t batch, int64_t row, int64_t col, const float* t) {
  if (row >= a.rows || col >= a.cols) return;
  if (a.update)
    store_update(a, batch, row, col, t);
  else if (a.out_format == ZS_FORMAT_FP32)
    store_values<kFP32>(a, batch, row, col, t);
  else if (a.out_format == ZS_FORMAT_BF16)
    store_values<kBF16>(a, batch, row, col, t);
  else
    store_values<kFP16>(a, batch, row, col, t);
}

// One of them.
__device__ __forceinline__ void store_one(const NsLast& a, int64_t batch, int64_t row, int64_t col, float t) {
  if (row >= a.rows || col >= a.cols) return;
  const int64_t i = batch * a.batch_out + row * a.ld_out + col;
  if (a.update) {
    const float v = a.dk * ((const GLB float*)a.master)[i] - a.ss * (t * kPerUnit);
    st_elem<kFP32>(a.master, i, v);
    st_elem<kBF16>(a.param, i, v);
  } else if (a.out_format == ZS_FORMAT_FP32) {
    st_elem<kFP32>(a.out, i, t * kPerUnit);
  } else if (a.out_format == ZS_FORMAT_BF16) {
    st_elem<kBF16>(a.out, i, t * kPerUnit);
  } else {
    st_elem<kFP16>(a.out, i, t * kPerUnit);
  }
}
// From a problem's description.
inline NsLast last_of(const NsProblem& p) {
  NsLast l{};
  l.turned = p.rows > p.cols;
  l.update = p.update;
  l.rows = p.rows;
  l.cols = p.cols;
  l.out = p.out;
  l.out_format = p.out_format;
  l.ld_out = p.update ? p.cols : p.ld_out;
  l.batch_out = p.update ? p.rows * p.cols : p.batch_out;
  l.master = p.master;
  l.param = p.param;
  l.dk = p.dk;
  l.ss = p.ss;
  return l;
}
inline MeanArgs mean_of(const NsProblem& p) {
  MeanArgs a{};
  for (int r = 0; r < p.n_rep; ++r) a.g[r] = p.grads[r];
  a.momentum = p.momentum;
  a.n = p.rows * p.cols;
  a.n_rep = p.n_rep;
  a.nesterov = p.nesterov;
  a.mu = p.mu;
  return a;
}

// The rest of a step of a matrix with at most kSlabSide rows, from its S (zs_muon_small.hip).
struct NsSlab {
  const char *s, *x;
  char* to;  // NULL: the last step
  int64_t pitch_x, batch_s, batch_x;
  int32_t m;
  int64_t n;  // padded
  float ca, cb, cc;
  NsLast last;
};
hipError_t launch_ns_slab(const NsSlab& a, int64_t batch, hipStream_t stream);

}  // namespace ns
}  // namespace zs
