// Small matrices (both sides at most 128) orthogonalised, or stepped, by one
// workgroup each in one kernel: X and S stay in LDS from the values to the
// values.  The products are those of zs_muon.hip (two fp16 parts an operand,
// three products of them, fp32 sums).
//
// A batch of them is bound by the matrix instructions and LDS reads of a
// workgroup, a single one by their latency: 15 products of 128 x 128 x 128 take
// about 2 us each, where a kernel for each product takes 5-6.
#include "zs_muon_dev.h"

namespace zs {
namespace {

using namespace dev;
using namespace ns;

struct SmallArgs {
  // values in
  const void* x;
  int64_t ld, batch_ld;
  MeanArgs mean;  // the update's
  int32_t m, n;   // short and long side, padded
  int32_t steps;
  float coefs[3 * kMaxNsSteps];
  NsLast last;
};

// A matrix of SIDE columns in LDS: rows of SIDE / 4 pieces of 16 bytes, in groups of 4 pieces of hi parts and 4 of lo
// parts of 32 columns; piece c of row r lies at place c ^ (r & 7) of its group, so that 8 rows' equal pieces lie in
// different banks.
template <int SIDE>
struct Small {
  static constexpr int kPitch = SIDE * 4, kBytes = SIDE * kPitch;
  static constexpr int WM = 2, WN = SIDE / 32, kThreads = WM * WN * 64;
  static constexpr int TM = SIDE / WM, FM = TM / 16, FN = 2;  // 32 columns a wave
  static __device__ __forceinline__ int at(int row, int piece) { return row * kPitch + (piece ^ (row & 7)) * 16; }
};

// acc += a b^T (TURNED: a b) over `groups` groups of 32 of the summed axis, for this wave's TM x 32 sums.
template <int SIDE, bool TURNED>
__device__ __forceinline__ void small_product(const LDS char* a, const LDS char* b, int groups, int wm, int wn,
                                              f32x4 (&acc)[Small<SIDE>::FM][2]) {
  typedef Small<SIDE> L;
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
#pragma unroll
  for (int i = 0; i < L::FM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  for (int k = 0; k < groups; ++k) {
    i32x4 fa[2][L::FM], fb[2][2];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
#pragma unroll
      for (int i = 0; i < L::FM; ++i) fa[part][i] = *(const LDS i32x4*)(a + L::at(wm + i * 16 + i16, k * 8 + part * 4 + g));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (TURNED) {
          // 8 rows (4 and 4) of the summed axis x 16 columns
          const int row = k * 32 + 8 * g + (i16 >> 2), piece = wn / 32 * 8 + part * 4 + j * 2 + (i16 >> 1 & 1);
          const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(LDS char*)(b + L::at(row, piece) + (i16 & 1) * 8));
          const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(LDS char*)(b + L::at(row + 4, piece) + (i16 & 1) * 8));
          fb[part][j] = __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
        } else {
          fb[part][j] = *(const LDS i32x4*)(b + L::at(wn + j * 16 + i16, k * 8 + part * 4 + g));
        }
      }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)  // lo hi, hi hi, hi lo
#pragma unroll
      for (int i = 0; i < L::FM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_f16(fb[p == 2][j], fa[p == 0][i], acc[i][j]);
  }
}

// f(row, column of the first, the 8 sums) for this wave's sums.
template <int SIDE, class F>
__device__ __forceinline__ void small_each(int wm, int wn, const f32x4 (&acc)[Small<SIDE>::FM][2], F f) {
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
#pragma unroll
  for (int i = 0; i < Small<SIDE>::FM; ++i) {
    float t[8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t lo, hi;
      trade(__float_as_uint(acc[i][0][r]), __float_as_uint(acc[i][1][r]), lo, hi);
      t[r] = __uint_as_float(lo) * kPerUnit;
      t[4 + r] = __uint_as_float(hi) * kPerUnit;
    }
    f(i, wm + i * 16 + i16, wn + eight_at(g), t);
  }
}
template <int SIDE>
__device__ __forceinline__ int small_piece(int col) { return col / 32 * 8 + col % 32 / 8; }
template <int SIDE>
__device__ __forceinline__ void small_put(LDS char* to, int row, int col, const float* t) {
  u32x4 hi, lo;
  to_parts(t, hi, lo);
  *(LDS u32x4*)(to + Small<SIDE>::at(row, small_piece<SIDE>(col))) = hi;
  *(LDS u32x4*)(to + Small<SIDE>::at(row, small_piece<SIDE>(col) + 4)) = lo;
}
template <int SIDE>
__device__ __forceinline__ void small_add(const LDS char* from, int row, int col, float by, float* t) {
  const u32x4 hi = *(const LDS u32x4*)(from + Small<SIDE>::at(row, small_piece<SIDE>(col)));
  const u32x4 lo = *(const LDS u32x4*)(from + Small<SIDE>::at(row, small_piece<SIDE>(col) + 4));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    t[2 * k] = by * (h_lo<kFP16>(hi[k]) + h_lo<kFP16>(lo[k])) + t[2 * k];
    t[2 * k + 1] = by * (h_hi<kFP16>(hi[k]) + h_hi<kFP16>(lo[k])) + t[2 * k + 1];
  }
}

template <int SIDE, int FMT, bool UPDATE>
__global__ __launch_bounds__(Small<SIDE>::kThreads) void ns_small(const SmallArgs a) {
  typedef Small<SIDE> L;
  constexpr int kPieces = SIDE * SIDE / 8 / L::kThreads;  // of 8 values a thread
  __shared__ __attribute__((aligned(1024))) char lds[2 * L::kBytes];
  __shared__ double sums[L::kThreads / 64];
  LDS char* const x = (LDS char*)lds;
  LDS char* const s = x + L::kBytes;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / L::WN * L::TM, wn = wave % L::WN * 32;
  const int rows = (int)a.last.rows, cols = (int)a.last.cols, per = (cols + 7) / 8;
  const int64_t batch = blockIdx.x;

  // u and its square sum
  float u[kPieces][8];
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int p = tid + c * L::kThreads, row = p / per, col = p % per * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) u[c][k] = 0.0f;
    if (row >= rows) continue;
    const int left = cols - col < 8 ? cols - col : 8;
    if constexpr (UPDATE) {
      const int64_t i = batch * a.mean.n + (int64_t)row * cols + col;
      float t[8], m[8], m1[8];
      load8<kBF16>(a.mean.g[0], i, left, t);
      for (int r = 1; r < a.mean.n_rep; ++r) {
        float v[8];
        load8<kBF16>(a.mean.g[r], i, left, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = t[k] + v[k];
      }
      load8<kFP32>(a.mean.momentum, i, left, m);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[c][k] = k < left ? mean_step(t[k], m[k], a.mean, m1[k]) : 0.0f;
      if (left == 8) {
        st_four<kFP32>(a.mean.momentum, i, m1);
        st_four<kFP32>(a.mean.momentum, i + 4, m1 + 4);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < left) st_elem<kFP32>(a.mean.momentum, i + k, m1[k]);
      }
    } else {
      load8<FMT>(a.x, batch * a.batch_ld + (int64_t)row * a.ld + col, left, u[c]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += (double)u[c][k] * (double)u[c][k];
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) sums[wave] = sum;
  // zeros, where X0 has padding
  for (int i = tid; i < L::kBytes / 16; i += L::kThreads) *(LDS u32x4*)(x + i * 16) = (u32x4){0, 0, 0, 0};
  __syncthreads();
  sum = sums[0];
#pragma unroll
  for (int w = 1; w < L::kThreads / 64; ++w) sum += sums[w];
  const double unit = sum == 0.0 ? 0.0 : (double)kUnit / __builtin_sqrt(sum);
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int p = tid + c * L::kThreads, row = p / per, col = p % per * 8;
    if (row >= rows) continue;
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = col + k < cols ? (float)((double)u[c][k] * unit) : 0.0f;  // (padding stays zero)
    if (!a.last.turned) {
      small_put<SIDE>(x, row, col, t);
    } else {
      u32x4 hi, lo;
      to_parts(t, hi, lo);
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // one value each of 8 rows of X
        if (col + k >= cols) continue;
        const int piece = small_piece<SIDE>(row);
        *(LDS uint16_t*)(x + L::at(col + k, piece) + row % 8 * 2) = (uint16_t)(hi[k / 2] >> (k % 2 * 16));
        *(LDS uint16_t*)(x + L::at(col + k, piece + 4) + row % 8 * 2) = (uint16_t)(lo[k / 2] >> (k % 2 * 16));
      }
    }
  }
  __syncthreads();

  const bool in_s = wm < a.m && wn < a.m, in_x = wm < a.m && wn < a.n;  // this wave's part is not all padding
  f32x4 acc[L::FM][2];
  for (int step = 0; step < a.steps; ++step) {
    const float ca = a.coefs[3 * step], cb = a.coefs[3 * step + 1], cc = a.coefs[3 * step + 2];
    if (in_s) {
      small_product<SIDE, false>(x, x, a.n / 32, wm, wn, acc);
      small_each<SIDE>(wm, wn, acc, [&](int, int row, int col, const float* t) { small_put<SIDE>(s, row, col, t); });
    }
    __syncthreads();
    float b[L::FM][8];
    if (in_s) {
      small_product<SIDE, false>(s, s, a.m / 32, wm, wn, acc);
      small_each<SIDE>(wm, wn, acc, [&](int i, int row, int col, const float* t) {
#pragma unroll
        for (int k = 0; k < 8; ++k) b[i][k] = cc * t[k];
        small_add<SIDE>(s, row, col, cb, b[i]);
      });
    }
    __syncthreads();  // S has been read
    if (in_s) {
      const int lane = tid & 63;
#pragma unroll
      for (int i = 0; i < L::FM; ++i) small_put<SIDE>(s, wm + i * 16 + (lane & 15), wn + eight_at(lane >> 4), b[i]);
    }
    __syncthreads();
    if (in_x) {
      small_product<SIDE, true>(s, x, a.m / 32, wm, wn, acc);
      small_each<SIDE>(wm, wn, acc, [&](int i, int row, int col, const float* t) {
#pragma unroll
        for (int k = 0; k < 8; ++k) b[i][k] = t[k];
        small_add<SIDE>(x, row, col, ca, b[i]);
      });
    }
    const int lane = tid & 63, col = wn + eight_at(lane >> 4);
    if (step == a.steps - 1) {
      if (!in_x) return;
#pragma unroll
      for (int i = 0; i < L::FM; ++i) {
        const int row = wm + i * 16 + (lane & 15);
        if (!a.last.turned) {
          store_last(a.last, batch, row, col, b[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) store_one(a.last, batch, col + k, row, b[i][k]);
        }
      }
      return;
    }
    __syncthreads();  // X has been read
    if (in_x) {
#pragma unroll
      for (int i = 0; i < L::FM; ++i) small_put<SIDE>(x, wm + i * 16 + (lane & 15), col, b[i]);
    }
    __syncthreads();
  }
}

template <int SIDE>
hipError_t small_launch(const NsProblem& p, hipStream_t stream) {
  SmallArgs a{};
  a.m = (int32_t)padded(p.rows < p.cols ? p.rows : p.cols);
  a.n = (int32_t)padded(p.rows < p.cols ? p.cols : p.rows);
  a.steps = p.steps;
  for (int i = 0; i < 3 * p.steps; ++i) a.coefs[i] = p.coefs[i];
  a.last = last_of(p);
  const dim3 grid((unsigned)p.batch);
  if (p.update) {
    a.mean = mean_of(p);
    ns_small<SIDE, kFP32, true><<<grid, Small<SIDE>::kThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.x = p.x;
  a.ld = p.ld_x;
  a.batch_ld = p.batch_x;
  if (p.x_format == ZS_FORMAT_FP32)
    ns_small<SIDE, kFP32, false><<<grid, Small<SIDE>::kThreads, 0, stream>>>(a);
  else if (p.x_format == ZS_FORMAT_BF16)
    ns_small<SIDE, kBF16, false><<<grid, Small<SIDE>::kThreads, 0, stream>>>(a);
  else
    ns_small<SIDE, kFP16, false><<<grid, Small<SIDE>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_small(const NsProblem& p, hipStream_t stream) {
  return p.rows <= 64 && p.cols <= 64 ? small_launch<64>(p, stream) : small_launch<kSmallSide>(p, stream);
}

}  // namespace zs
