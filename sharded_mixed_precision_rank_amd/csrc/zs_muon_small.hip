// Small matrices (both sides at most 128) orthogonalised, or stepped, by one
// workgroup each in one kernel: X and S stay in LDS from the values to the
// values.  The products are those of zs_muon.hip (two fp16 parts an operand,
// three products of them, fp32 sums).
//
// Bound by a workgroup's LDS reads and the trips between them: 15 products of 128 x
// 128 x 128, one behind the other, take 2.9 us each, 1.3 of them matrix instructions,
// whether one matrix or one for every compute unit (32 of them, fp32 to bf16: 46.6 us,
// where a kernel for each product took 96).
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
// A wave has ROWS rows of 32 columns.
template <int SIDE, int ROWS>
struct Small {
  static constexpr int kPitch = SIDE * 4, kBytes = SIDE * kPitch;
  static constexpr int WN = SIDE / 32, kThreads = SIDE / ROWS * WN * 64;
  static constexpr int TM = ROWS, FM = TM / 16;
};
template <int COLS>
__device__ __forceinline__ int small_at(int row, int piece) {
  return row * (COLS * 4) + (piece ^ (row & 7)) * 16;
}

// acc = a b^T (TURNED: a b) over `groups` groups of 32 of the summed axis, for a wave's 16 FM x 32 sums; a has CA columns in
// LDS, b CB.
template <int CA, int CB, bool TURNED, int FM>
__device__ __forceinline__ void small_product(const LDS char* a, const LDS char* b, int groups, int wm, int wn, f32x4 (&acc)[FM][2]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
  // A lane's places: the xor of a place is of the lane alone, groups and fragments lie at fixed distances from it.
  const LDS char *at_a[2], *at_b[2], *at_t[2][2][2];
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    at_a[part] = a + small_at<CA>(wm + i16, part * 4 + g);
    at_b[part] = b + small_at<CB>(wn + i16, part * 4 + g);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int four = 0; four < 2; ++four)  // 8 rows (4 and 4) of the summed axis x 16 columns
        at_t[part][j][four] = b + small_at<CB>(8 * g + (i16 >> 2) + 4 * four, part * 4 + j * 2 + (i16 >> 1 & 1)) + (i16 & 1) * 8 + wn * 4;
  }
  i32x4 fa[2][FM], fb[2][2];
  auto read_a = [&](int part, int k) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[part][i] = *(const LDS i32x4*)(at_a[part] + i * 16 * CA * 4 + k * 128);
  };
  auto read_b = [&](int part, int k) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (TURNED) {
        const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(LDS char*)(at_t[part][j][0] + k * 32 * CB * 4));
        const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(LDS char*)(at_t[part][j][1] + k * 32 * CB * 4));
        fb[part][j] = __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
      } else {
        fb[part][j] = *(const LDS i32x4*)(at_b[part] + j * 16 * CB * 4 + k * 128);
      }
    }
  };
  auto times = [&](int pa, int pb, auto first) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_f16(fb[pb][j], fa[pa][i], first ? (f32x4){0, 0, 0, 0} : acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // lo hi, hi hi, hi lo: the fragments of the next product, and of the next group's first, are read meanwhile (past the last
  // group: again, which is never used)
  read_a(1, 0);
  read_b(0, 0);
  auto group = [&](int k, auto first) {
    const int next = k + 1 < groups ? k + 1 : k;
    read_a(0, k);
    read_b(1, k);
    times(1, 0, first);
    read_a(1, next);
    times(0, 0, No{});
    read_b(0, next);
    times(0, 1, No{});
  };
  group(0, Yes{});
  for (int k = 1; k < groups; ++k) group(k, No{});
}

// f(fragment, row, column of the first, 8 held values) for a wave's sums times `by`.
template <int FM, class F>
__device__ __forceinline__ void small_each(int wm, int wn, const f32x4 (&acc)[FM][2], float by, F f) {
  const int lane = threadIdx.x & 63, g = lane >> 4, i16 = lane & 15;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    float t[8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t lo, hi;
      trade(__float_as_uint(acc[i][0][r]), __float_as_uint(acc[i][1][r]), lo, hi);
      t[r] = __uint_as_float(lo) * by;
      t[4 + r] = __uint_as_float(hi) * by;
    }
    f(i, wm + i * 16 + i16, wn + eight_at(g), t);
  }
}
__device__ __forceinline__ int small_piece(int col) { return col / 32 * 8 + col % 32 / 8; }
template <int COLS>
__device__ __forceinline__ void small_put(LDS char* to, int row, int col, const float* t) {
  u32x4 hi, lo;
  to_parts(t, hi, lo);
  *(LDS u32x4*)(to + small_at<COLS>(row, small_piece(col))) = hi;
  *(LDS u32x4*)(to + small_at<COLS>(row, small_piece(col) + 4)) = lo;
}
template <int COLS>
__device__ __forceinline__ void small_add(const LDS char* from, int row, int col, float by, float* t) {
  add_parts(*(const LDS u32x4*)(from + small_at<COLS>(row, small_piece(col))),
            *(const LDS u32x4*)(from + small_at<COLS>(row, small_piece(col) + 4)), by, t);
}
// b S + c S^2 of the S in LDS (m x m, padded), in its place; barriers in it.
template <int SIDE, int ROWS>
__device__ __forceinline__ void small_poly(LDS char* s, int m, int wm, int wn, float cb, float cc) {
  typedef Small<SIDE, ROWS> L;
  const bool in_s = wm < m && wn < m;
  f32x4 acc[L::FM][2];
  float b[L::FM][8];
  if (in_s) {
    small_product<SIDE, SIDE, false>(s, s, m / 32, wm, wn, acc);
    small_each(wm, wn, acc, cc * kPerUnit, [&](int i, int row, int col, const float* t) {
#pragma unroll
      for (int k = 0; k < 8; ++k) b[i][k] = t[k];
      small_add<SIDE>(s, row, col, cb, b[i]);
    });
  }
  __syncthreads();  // S has been read
  if (in_s) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < L::FM; ++i) small_put<SIDE>(s, wm + i * 16 + (lane & 15), wn + eight_at(lane >> 4), b[i]);
  }
  __syncthreads();
}
// The last step's values at (row, col .. col + 7) of X.
__device__ __forceinline__ void small_last(const NsLast& a, int64_t batch, int64_t row, int64_t col, const float* t) {
  if (!a.turned) {
    store_last(a, batch, row, col, t);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) store_one(a, batch, col + k, row, t[k]);
  }
}

template <int SIDE, int ROWS, int FMT, bool UPDATE>
__global__ __launch_bounds__((Small<SIDE, ROWS>::kThreads)) void ns_small(const SmallArgs a) {
  typedef Small<SIDE, ROWS> L;
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
        const int piece = small_piece(row);
        *(LDS uint16_t*)(x + small_at<SIDE>(col + k, piece) + row % 8 * 2) = (uint16_t)(hi[k / 2] >> (k % 2 * 16));
        *(LDS uint16_t*)(x + small_at<SIDE>(col + k, piece + 4) + row % 8 * 2) = (uint16_t)(lo[k / 2] >> (k % 2 * 16));
      }
    }
  }
  __syncthreads();

  const bool in_s = wm < a.m && wn < a.m, in_x = wm < a.m && wn < a.n;  // this wave's part is not all padding
  f32x4 acc[L::FM][2];
  for (int step = 0; step < a.steps; ++step) {
    const float ca = a.coefs[3 * step], cb = a.coefs[3 * step + 1], cc = a.coefs[3 * step + 2];
    if (in_s) {
      small_product<SIDE, SIDE, false>(x, x, a.n / 32, wm, wn, acc);
      small_each(wm, wn, acc, kPerUnit, [&](int, int row, int col, const float* t) { small_put<SIDE>(s, row, col, t); });
    }
    __syncthreads();
    small_poly<SIDE, ROWS>(s, a.m, wm, wn, cb, cc);
    float b[L::FM][8];
    if (in_x) {
      small_product<SIDE, SIDE, true>(s, x, a.m / 32, wm, wn, acc);
      small_each(wm, wn, acc, kPerUnit, [&](int i, int row, int col, const float* t) {
#pragma unroll
        for (int k = 0; k < 8; ++k) b[i][k] = t[k];
        small_add<SIDE>(x, row, col, ca, b[i]);
      });
    }
    const int lane = tid & 63, col = wn + eight_at(lane >> 4);
    if (step == a.steps - 1) {
      if (!in_x) return;
      int row_last = wm + (lane & 15), col_last = col;
      asm volatile("" : "+v"(row_last), "+v"(col_last));  // (so that the places in memory are not held through all steps)
#pragma unroll
      for (int i = 0; i < L::FM; ++i) small_last(a.last, batch, row_last + i * 16, col_last, b[i]);
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

// ---------------------------------------------------------------------------
// A long matrix with a short side of at most 64: the polynomial and X' = a X + B X in
// one kernel, instead of one each.  A workgroup has 64 columns of X; every one of
// them makes B = b S + c S^2 for itself, in LDS.  64 x 4096: 6.4 us, where the two
// kernels take 4.2 and 5 and a launch more.  (With 128 rows it took 12, as long as
// the two, and longer where there are more workgroups than compute units.)
// ---------------------------------------------------------------------------
template <int SIDE>
__global__ __launch_bounds__((Small<SIDE, 32>::kThreads)) void ns_slab(const NsSlab a) {
  typedef Small<SIDE, 32> L;
  constexpr int kCols = 64, FM = 2;
  static_assert(L::kThreads / 64 == SIDE / 32 * 2, "32 x 32 values a wave");
  __shared__ __attribute__((aligned(1024))) char lds[L::kBytes + SIDE * kCols * 4];
  LDS char* const s = (LDS char*)lds;
  LDS char* const x = s + L::kBytes;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kCols, batch = blockIdx.y;
  const int m = a.m, cols = a.n - n0 < kCols ? (int)(a.n - n0) : kCols;  // multiples of 32
  const char* const from_s = a.s + batch * a.batch_s;
  const char* const from_x = a.x + batch * a.batch_x + n0 * 4;
  for (int i = tid; i < m * (SIDE / 4); i += L::kThreads) {
    const int row = i / (SIDE / 4), piece = i % (SIDE / 4);
    if (piece * 4 < m)
      *(LDS u32x4*)(s + small_at<SIDE>(row, piece)) = *(const GLB u32x4*)(const GLB char*)(from_s + (int64_t)row * (m * 4) + piece * 16);
  }
  for (int i = tid; i < m * (kCols / 4); i += L::kThreads) {
    const int row = i / (kCols / 4), piece = i % (kCols / 4);
    if (piece * 4 < cols)
      *(LDS u32x4*)(x + small_at<kCols>(row, piece)) = *(const GLB u32x4*)(const GLB char*)(from_x + (int64_t)row * a.pitch_x + piece * 16);
  }
  __syncthreads();
  small_poly<SIDE, 32>(s, m, wave / L::WN * L::TM, wave % L::WN * 32, a.cb, a.cc);
  const int wm = wave / 2 * 32, wn = wave % 2 * 32;
  if (wm >= m || wn >= cols) return;
  f32x4 acc[FM][2];
  small_product<SIDE, kCols, true>(s, x, m / 32, wm, wn, acc);
  small_each(wm, wn, acc, kPerUnit, [&](int, int row, int col, const float* t) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = t[k];
    small_add<kCols>(x, row, col, a.ca, v);
    if (a.to != nullptr)
      store_parts(a.to + batch * a.batch_x + (int64_t)row * a.pitch_x, n0 + col, v);
    else
      small_last(a.last, batch, row, n0 + col, v);
  });
}

template <int SIDE, int ROWS>
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
    ns_small<SIDE, ROWS, kFP32, true><<<grid, Small<SIDE, ROWS>::kThreads, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.x = p.x;
  a.ld = p.ld_x;
  a.batch_ld = p.batch_x;
  if (p.x_format == ZS_FORMAT_FP32)
    ns_small<SIDE, ROWS, kFP32, false><<<grid, Small<SIDE, ROWS>::kThreads, 0, stream>>>(a);
  else if (p.x_format == ZS_FORMAT_BF16)
    ns_small<SIDE, ROWS, kBF16, false><<<grid, Small<SIDE, ROWS>::kThreads, 0, stream>>>(a);
  else
    ns_small<SIDE, ROWS, kFP16, false><<<grid, Small<SIDE, ROWS>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace ns {

hipError_t launch_ns_slab(const NsSlab& a, int64_t batch, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 63) / 64), (unsigned)batch);
  ns_slab<kSlabSide><<<grid, Small<kSlabSide, 32>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace ns

hipError_t launch_ns_small(const NsProblem& p, hipStream_t stream) {
  if (p.rows <= 64 && p.cols <= 64) return small_launch<64, 32>(p, stream);
  // 16 waves of 32 rows where some of them have nothing but padding (32 x 96 x 128: 35.1 us, 8 waves of 64 rows 40.5), 8 where
  // all have work (32 x 128 x 128: 46.6, 16 waves 51.8)
  return p.rows <= 96 || p.cols <= 96 ? small_launch<kSmallSide, 32>(p, stream) : small_launch<kSmallSide, 64>(p, stream);
}

}  // namespace zs
