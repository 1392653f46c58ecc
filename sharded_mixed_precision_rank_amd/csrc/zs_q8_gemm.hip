// The 8-bit matrix product and the weight gradient from a checkpoint.
//
//   kNT  y[t][n] = sx[t] sw[n] sum_k x[t][k] w[n][k]      a linear layer's output
//   kNN  y[t][k] = sg[t]       sum_n g[t][n] w[n][k]      its input gradient, from the same weight codes
//   kTN  dw[n][k] = (add +)    sum_t dy[t][n] (x[t][k] s[t])   its weight gradient, from the saved input
//
// The integer sums are exact in 32 bits (K <= 131071).  The weight gradient's
// operands are bf16: a code times a power of two is exact there, any other
// scale costs one rounding of half a bf16 step; fp16 gradients are taken as
// two bf16 parts, which hold them exactly.  Its sums are fp32.
#include "zs_q8_dev.h"

namespace zs {
namespace {

using namespace dev;

#define LDS __attribute__((address_space(3)))

// Sixteen bytes at `col` of a row of `bytes` bytes, zeros past its end.
template <int ELEM>
__device__ __forceinline__ u32x4 ld_piece(const char* row, int64_t col, int64_t bytes, bool live) {
  u32x4 v = {0, 0, 0, 0};
  if (!live || col >= bytes) return v;
  if (col + 16 <= bytes) {
    if constexpr (ELEM == 1)
      return ld_any<u32x4>((const uint8_t*)row + col);
    else
      return ld_any<u32x4>((const uint16_t*)(row + col));
  }
#pragma unroll
  for (int k = 0; k < 16 / ELEM; ++k) {
    if (col + k * ELEM < bytes) {
      if constexpr (ELEM == 1)
        v[k / 4] |= (uint32_t)((const GLB uint8_t*)(row + col))[k] << (8 * (k % 4));
      else
        v[k / 2] |= (uint32_t)((const GLB uint16_t*)(row + col))[k] << (16 * (k % 2));
    }
  }
  return v;
}

// Codes times their row's scale, as bf16: 16 codes to 32 bytes.
__device__ __forceinline__ void codes_to_bf16(u32x4 q, float s, u32x4& lo, u32x4& hi) {
  u32x4 o[2];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t w = q[k / 2] >> (16 * (k % 2));
    o[k / 4][k % 4] = pack_bf16((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s);
  }
  lo = o[0];
  hi = o[1];
}

// Eight fp16 values as two bf16 parts each: the nearest bf16 and the rest,
// which has at most 3 bits (0 where the value is not finite).
__device__ __forceinline__ void fp16_parts(u32x4 h, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = h_lo<kFP16>(h[k]), b = h_hi<kFP16>(h[k]);
    hi[k] = pack_bf16(a, b);
    const float ra = a - bf_lo(hi[k]), rb = b - bf_hi(hi[k]);
    lo[k] = pack_bf16(fabsf(a) <= 65504.0f ? ra : 0.0f, fabsf(b) <= 65504.0f ? rb : 0.0f);
  }
}

// One element's result from its sum, by op.
template <Q8Op OP>
struct Out {
  float rs;  // kNT, kNN: the row's scale
  __device__ __forceinline__ float of(int32_t acc, const float* cs, int64_t n) const {
    const float v = (float)acc * rs;
    return cs ? v * ((const GLB float*)cs)[n] : v;
  }
};

// Four results at row m, columns n .. n + 3 (those below N), any format.
template <int FMT>
__device__ __forceinline__ void store_row4(const Q8Gemm& a, int64_t m, int64_t n, float* v, bool adds) {
  const int64_t i = m * a.ldd + n;
  if (adds) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < a.N) v[r] = ld_elem<FMT>(a.add, i + r) + v[r];
  }
  if (n + 4 <= a.N) {
    st_four<FMT>(a.d, i, v);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < a.N) st_elem<FMT>(a.d, i + r, v[r]);
  }
}
__device__ __forceinline__ void store4(const Q8Gemm& a, int64_t m, int64_t n, float* v, bool adds) {
  if (a.format == ZS_FORMAT_BF16)
    store_row4<kBF16>(a, m, n, v, adds);
  else if (a.format == ZS_FORMAT_FP16)
    store_row4<kFP16>(a, m, n, v, adds);
  else
    store_row4<kFP32>(a, m, n, v, adds);
}

// ---------------------------------------------------------------------------
// Any layout: 64 x 64 outputs per workgroup of four waves (32 x 32 each), the
// operands staged through registers 16 bytes at a time, so that rows may start
// at any address and end anywhere.  The first operand of the matrix
// instruction is b's, so that a lane ends with four consecutive columns of a
// row.
// ---------------------------------------------------------------------------
constexpr int kAnyTile = 64;
constexpr int kAnyK = 128;   // codes along K per step (kNT, kNN)
constexpr int kAnyKT = 32;   // rows of K per step (kTN)

template <Q8Op OP, int AFMT>
__global__ __launch_bounds__(256) void q8_gemm_any(const Q8Gemm a, int64_t tiles_n, int64_t tiles) {
  constexpr bool kT = OP == Q8Op::kTN;
  constexpr bool kParts = kT && AFMT == kFP16;
  // a: kT [32 rows of K][64 columns], twice with two parts; else [64 rows][128 codes]
  // b: kNT [64 rows][128 codes]; kNN [128 rows of K][64 codes]; kTN [32 rows of K][64 bf16]
  __shared__ __attribute__((aligned(16))) char lds_a[8192];
  __shared__ __attribute__((aligned(16))) char lds_b[8192];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int g = lane >> 4, i16 = lane & 15;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / tiles_n * kAnyTile, n0 = tile % tiles_n * kAnyTile;
    i32x4 acci[2][2];
    f32x4 accf[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acci[i][j] = (i32x4){0, 0, 0, 0}, accf[i][j] = (f32x4){0, 0, 0, 0};
    constexpr int kStep = kT ? kAnyKT : kAnyK;
    for (int64_t k0 = 0; k0 < a.K; k0 += kStep) {
      u32x4 ra[2], rb[2];
      float rscale = 0.0f;
      if constexpr (!kT) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p = tid + 256 * c;  // 8 pieces a row
          const int64_t m = m0 + p / 8;
          ra[c] = ld_piece<1>((const char*)a.a + m * a.lda, k0 + p % 8 * 16, a.K, m < a.M);
          if constexpr (OP == Q8Op::kNT) {
            const int64_t n = n0 + p / 8;
            rb[c] = ld_piece<1>((const char*)a.b + n * a.ldb, k0 + p % 8 * 16, a.K, n < a.N);
          } else {
            const int64_t k = k0 + p / 4;  // 4 pieces a row
            rb[c] = ld_piece<1>((const char*)a.b + k * a.ldb, n0 + p % 4 * 16, a.N, k < a.K);
          }
        }
      } else {
        const int64_t k = k0 + tid / 8;  // 8 pieces a row of 64 values
        ra[0] = ld_piece<2>((const char*)a.a + k * a.lda * 2, m0 * 2 + tid % 8 * 16, a.M * 2, k < a.K);
        const int64_t kb = k0 + tid / 4;  // 4 pieces a row of 64 codes, 128 threads
        const bool live = tid < 128 && kb < a.K;
        rb[0] = ld_piece<1>((const char*)a.b + kb * a.ldb, n0 + tid % 4 * 16, a.N, live);
        rscale = live ? ((const GLB float*)a.rs)[kb] : 0.0f;
      }
      __syncthreads();  // the step before has been read
      if constexpr (!kT) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p = tid + 256 * c;
          *(u32x4*)(lds_a + p / 8 * 128 + ((p % 8) ^ (p / 8 % 8)) * 16) = ra[c];
          if constexpr (OP == Q8Op::kNT)
            *(u32x4*)(lds_b + p / 8 * 128 + ((p % 8) ^ (p / 8 % 8)) * 16) = rb[c];
          else
            *(u32x4*)(lds_b + p * 16) = rb[c];
        }
      } else {
        if constexpr (kParts) {
          u32x4 hi, lo;
          fp16_parts(ra[0], hi, lo);
          *(u32x4*)(lds_a + tid * 16) = hi;
          *(u32x4*)(lds_a + 4096 + tid * 16) = lo;
        } else {
          *(u32x4*)(lds_a + tid * 16) = ra[0];
        }
        if (tid < 128) {
          u32x4 lo, hi;
          codes_to_bf16(rb[0], rscale, lo, hi);
          *(u32x4*)(lds_b + tid * 32) = lo;
          *(u32x4*)(lds_b + tid * 32 + 16) = hi;
        }
      }
      __syncthreads();
      if constexpr (!kT) {
#pragma unroll
        for (int kk = 0; kk < 128; kk += 64) {
          i32x4 fa[2], fb[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = wm + i * 16 + i16;
            fa[i] = *(const i32x4*)(lds_a + r * 128 + ((kk / 16 + g) ^ (r % 8)) * 16);
            if constexpr (OP == Q8Op::kNT) {
              const int s = wn + i * 16 + i16;
              fb[i] = *(const i32x4*)(lds_b + s * 128 + ((kk / 16 + g) ^ (s % 8)) * 16);
            } else {
              // transposing read: 8 rows of K x 16 columns per 16 lanes
              const int row = kk + 16 * g + i16 / 2, off = wn + i * 16 + i16 % 2 * 8;
              const i32x2 p = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(lds_b + row * 64 + off));
              const i32x2 q = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(lds_b + (row + 8) * 64 + off));
              fb[i] = (i32x4){p[0], p[1], q[0], q[1]};
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acci[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acci[i][j], 0, 0, 0);
        }
      } else {
        auto tr = [&](const char* base, int col) {  // 8 rows of K (two reads of 4) x 16 columns
          const int row = 8 * g + i16 / 4, off = col * 2 + i16 % 4 * 8;
          const i16x4 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(base + row * 128 + off));
          const i16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(base + (row + 4) * 128 + off));
          return __builtin_bit_cast(bf16x8, (i16x8){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]});
        };
        bf16x8 fb[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[j] = tr(lds_b, wn + j * 16);
#pragma unroll
        for (int part = 0; part < (kParts ? 2 : 1); ++part)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bf16x8 fa = tr(lds_a + part * 4096, wm + i * 16);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              accf[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa, accf[i][j], 0, 0, 0);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + wm + i * 16 + i16;
      if (m >= a.M) continue;
      Out<OP> out{kT ? 0.0f : ((const GLB float*)a.rs)[m]};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wn + j * 16 + 4 * g;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = kT ? accf[i][j][r] : n + r < a.N ? out.of(acci[i][j][r], a.cs, n + r) : 0.0f;
        if (n < a.N) store4(a, m, n, v, kT && a.add != nullptr);
      }
    }
    __syncthreads();  // before the next tile's first pieces are written
  }
}

template <Q8Op OP, int AFMT>
hipError_t any_launch(const Q8Gemm& a, hipStream_t stream) {
  const int64_t tm = (a.M + kAnyTile - 1) / kAnyTile, tn = (a.N + kAnyTile - 1) / kAnyTile;
  const int64_t tiles = tm * tn;
  const dim3 grid((unsigned)(tiles < (1 << 20) ? tiles : (1 << 20)));
  q8_gemm_any<OP, AFMT><<<grid, 256, 0, stream>>>(a, tn, tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q8_gemm(Q8Op op, const Q8Gemm& a, hipStream_t stream) {
  switch (op) {
    case Q8Op::kNT: return any_launch<Q8Op::kNT, kBF16>(a, stream);
    case Q8Op::kNN: return any_launch<Q8Op::kNN, kBF16>(a, stream);
    default:
      return a.a_format == ZS_FORMAT_FP16 ? any_launch<Q8Op::kTN, kFP16>(a, stream)
                                          : any_launch<Q8Op::kTN, kBF16>(a, stream);
  }
}

}  // namespace zs
