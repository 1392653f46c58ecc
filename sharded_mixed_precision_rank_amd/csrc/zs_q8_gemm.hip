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
#include <utility>

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

// Eight codes times their row's scale, as bf16.
__device__ __forceinline__ u32x4 codes_to_bf16(uint32_t q0, uint32_t q1, float s) {
  u32x4 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = (k < 2 ? q0 : q1) >> (16 * (k % 2));
    o[k] = pack_bf16((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s);
  }
  return o;
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

// RUN (4 or 8) results at row m from column n on (those below N), plus what
// add holds there.  PAST: around the caches, for 16-bit formats.
template <int FMT, int RUN, bool PAST>
__device__ __forceinline__ void store_run_as(const Q8Gemm& a, int64_t m, int64_t n, float* v) {
  const int64_t i = m * a.ldd + n;
  if (n + RUN <= a.N) {
    if (a.add != nullptr) {
#pragma unroll
      for (int r = 0; r < RUN; r += 4) {
        if constexpr (FMT == kFP32) {
          const f32x4 x = ld_any<f32x4>((const float*)a.add + i + r);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[r + k] = x[k] + v[r + k];
        } else {
          const u32x2 x = ld_any<u32x2>((const uint16_t*)a.add + i + r);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[r + k] = (k % 2 ? h_hi<FMT>(x[k / 2]) : h_lo<FMT>(x[k / 2])) + v[r + k];
        }
      }
    }
    if constexpr (FMT == kFP32) {
#pragma unroll
      for (int r = 0; r < RUN; r += 4) st_four<FMT>(a.d, i + r, v + r);
    } else if constexpr (RUN == 8) {
      const u32x4 w = {pack_two<FMT>(v[0], v[1]), pack_two<FMT>(v[2], v[3]), pack_two<FMT>(v[4], v[5]),
                       pack_two<FMT>(v[6], v[7])};
      if constexpr (PAST)
        st_past((uint16_t*)a.d + i, w);
      else
        st_any((uint16_t*)a.d + i, w);
    } else {
      st_four<FMT>(a.d, i, v);
    }
  } else {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if (n + r < a.N) st_elem<FMT>(a.d, i + r, a.add != nullptr ? ld_elem<FMT>(a.add, i + r) + v[r] : v[r]);
    }
  }
}
template <int RUN, bool PAST = false>
__device__ __forceinline__ void store_run(const Q8Gemm& a, int64_t m, int64_t n, float* v) {
  if (a.format == ZS_FORMAT_BF16)
    store_run_as<kBF16, RUN, PAST>(a, m, n, v);
  else if (a.format == ZS_FORMAT_FP16)
    store_run_as<kFP16, RUN, PAST>(a, m, n, v);
  else
    store_run_as<kFP32, RUN, PAST>(a, m, n, v);
}

// Two accumulators side by side (columns 4 g + r of one 16-column fragment and
// of the next), traded between lane groups so that a lane has 8 consecutive
// columns: those from eight_at(g) on of the 32.
__device__ __forceinline__ int eight_at(int g) { return (g & 1) * 16 + (g >> 1) * 8; }
__device__ __forceinline__ void trade(uint32_t x, uint32_t y, uint32_t& lo, uint32_t& hi) {
  typedef uint32_t Two __attribute__((ext_vector_type(2)));
  const Two t = __builtin_bit_cast(Two, __builtin_amdgcn_permlane16_swap(x, y, false, false));
  lo = t[0];
  hi = t[1];
}

// ---------------------------------------------------------------------------
// Any layout: 64 x 64 outputs per workgroup of four waves (32 x 32 each), the
// operands staged through registers 16 bytes at a time, so that rows may start
// at any address and end anywhere.  The first operand of the matrix
// instruction is b's, so that a lane ends with four consecutive columns of a
// row.  8192 x 11008 x 4096 with rows one byte off 16-byte boundaries: 1172 us,
// kNN 2058 (on them, by the tiled kernels, 338 and 291): loads of 16 bytes that
// straddle lines, one buffer and two barriers a step.
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
          *(u32x4*)(lds_b + tid * 32) = codes_to_bf16(rb[0][0], rb[0][1], rscale);
          *(u32x4*)(lds_b + tid * 32 + 16) = codes_to_bf16(rb[0][2], rb[0][3], rscale);
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
      const float rs = kT ? 0.0f : ((const GLB float*)a.rs)[m];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wn + j * 16 + 4 * g;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = kT ? accf[i][j][r] : (float)acci[i][j][r] * rs;
          if (!kT && a.cs != nullptr && n + r < a.N) v[r] = v[r] * ((const GLB float*)a.cs)[n + r];
        }
        if (n < a.N) store_run<4>(a, m, n, v);
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

// ---------------------------------------------------------------------------
// Code rows on 16-byte boundaries: BM x BN outputs per workgroup of WM x WN
// waves, pieces of both operands moved from memory into LDS directly, 128
// codes of the summed axis a stage and NS stages in a ring.  A wave holds its
// fragments of the next 64 codes in registers while the matrix instructions
// take the current ones, so that LDS reads, memory loads and matrix
// instructions run side by side.  One barrier a stage: between its halves every
// wave has read all of the stage and its part of the next one has landed.
//
// 256 x 256 by eight waves (128 x 64 each, 245 registers, 128 KB of LDS):
// 8192 x 11008 x 4096 in 315-356 us (2070-2350 TOP/s), its input gradient in 275-297
// (2490-2690), where a library's int8 product takes 362 (2040).  Of 119 us at
// 8192 x 4096 x 4096, the matrix instructions alone take 79 (the clock falls
// under them, to about 1.7 GHz) and the loads alone 102.  Four waves of 128 x
// 128 spill or shuffle accumulators (309-909 us); stages of 64 codes in a ring of
// four or five load half lines and are slower (125 against 119, kNN 156 against
// 125).  Bank conflicts: none, by counter (SQ_LDS_BANK_CONFLICT, every tile shape).
// ---------------------------------------------------------------------------
typedef uint32_t Rsrc __attribute__((ext_vector_type(4)));

// A buffer descriptor over `rows` rows of `width` bytes, `pitch` apart, at p:
// loads past them give zeros.  The callers keep rows * pitch below 2^31; the
// last 4 bytes may lie partly past the end, within an aligned word.
__device__ __forceinline__ Rsrc make_rsrc(const void* p, int32_t rows, int32_t width, int32_t pitch) {
  const uint64_t b = (uint64_t)p;
  const int32_t n = max((rows - 1) * pitch + width + 3, 0) & ~3;  // width <= pitch: 0 without rows
  Rsrc r = {(uint32_t)b, (uint32_t)(b >> 32), (uint32_t)n, 0x00020000u};
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(r[i]);
  return r;
}
// What is left of `total` after `done`, at most `most`.
__device__ __forceinline__ int32_t left_of(int64_t total, int64_t done, int32_t most) {
  const int64_t n = total - done;
  return n < most ? (int32_t)n : most;
}

// 64 lanes' 16 bytes each, from rsrc + voff, to LDS at lds + 16 * lane.  The
// whole offset is in voff: the bounds check is against that.  The caller waits
// (vmcnt) before anyone reads them, and before the workgroup ends.  The LDS
// address is an operand in m0, so that the compiler knows of every write to
// that register; a load that follows the write needs one wait state.
// The descriptor has to come from scalar instructions, as it does (make_rsrc's
// readfirstlanes of scalar values fold away): after a vector instruction's write
// the load would need five wait states, which the compiler does not add in an
// asm statement and which, always there, cost 1-2% (333 x 4096 x 11008: 7%).
__device__ __forceinline__ void load_to_lds(Rsrc rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc), "{m0}"(lds) : "memory");
}

// The same with 4 bytes a lane.
__device__ __forceinline__ void load4_to_lds(Rsrc rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc), "{m0}"(lds) : "memory");
}

// Sixteen bytes of a buffer (zeros past its end).
__device__ __forceinline__ u32x4 ld_buffer16(Rsrc r, uint32_t voff) {
  const __amdgpu_buffer_rsrc_t b = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((uint64_t)r[0] | (uint64_t)r[1] << 32), 0, (int)r[2], 0x00020000);
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)voff, 0, 0));
}
__device__ __forceinline__ float ld_buffer4(Rsrc r, uint32_t voff) {
  const __amdgpu_buffer_rsrc_t b = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((uint64_t)r[0] | (uint64_t)r[1] << 32), 0, (int)r[2], 0x00020000);
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)voff, 0, 0));
}

// The tile of workgroup `bid`: workgroups go to the eight XCDs in turn, so
// each XCD takes a run of consecutive tiles, which go down groups of 8 tile
// rows: its L2 sees few rows and columns of operands at a time (groups of 4 or
// 16: the same or up to 5% slower).
__device__ __forceinline__ void tile_of(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t total = tiles_m * tiles_n;
  const uint32_t x = bid % 8, per = total / 8, more = total % 8;
  const uint32_t id = x * per + (x < more ? x : more) + bid / 8;
  const uint32_t group = id / (8 * tiles_n), first = group * 8;
  const uint32_t height = tiles_m - first < 8 ? tiles_m - first : 8;
  const uint32_t in = id % (8 * tiles_n);
  tm = first + in % height;
  tn = in / height;
}

constexpr int kStage = 128;  // codes of K per stage

// f of 0 .. N - 1, each a constant: unrolled whatever its size.
template <class F, int... I>
__device__ __forceinline__ void for_each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void for_each(F f) {
  for_each(f, std::make_integer_sequence<int, N>{});
}
typedef std::integral_constant<int, 0> First;
typedef std::integral_constant<int, 1> Second;
typedef std::true_type Yes;
typedef std::false_type No;
// Between a stage's halves: this wave has read all of its buffer, and all but
// its last LATER loads have landed (and what it wrote); then every wave's have.
template <int LATER>
__device__ __forceinline__ void meet() {
  static_assert(LATER >= 0 && LATER < 64, "a 6-bit count");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LATER) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The xor of a piece's place in row r of b's rows of K.
template <int BN>
__device__ __forceinline__ int place_nn(int r) {
  return BN > 64 ? r & 7 : (r >> 2 & 1) | (r >> 4 & 1) << 1;
}

template <Q8Op OP, int BM, int BN, int WM, int WN, int NS, bool PAST>
__global__ __launch_bounds__(WM* WN * 64, 2) void q8_gemm_tile(const Q8Gemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr bool kNT = OP == Q8Op::kNT;
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  // kNN: 16 rows of K of b, and 128 bytes that put the next 16 in the other half of the banks (rows of 4 pieces do
  // that by their places)
  constexpr int kGroup = 16 * BN + (BN > 64 ? 128 : 0);
  constexpr int kABytes = BM * kStage, kBBytes = kNT ? BN * kStage : kStage / 16 * kGroup, kBuf = kABytes + kBBytes;
  constexpr int kALoads = kABytes / 1024 / kWaves, kBLoads = BN * kStage / 1024 / kWaves;
  static_assert(FN % 2 == 0 && kBLoads % 2 == 0 && kALoads > 0 && kBLoads > 0 && (NS & (NS - 1)) == 0, "tile shape");
  __shared__ __attribute__((aligned(1024))) char lds[NS * kBuf];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int wm = wave / WN * TM, wn = wave % WN * TN;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const uint32_t lda = (uint32_t)a.lda, ldb = (uint32_t)a.ldb;
  const int32_t K = (int32_t)a.K;
  const Rsrc ra = make_rsrc((const char*)a.a + m0 * a.lda, left_of(a.M, m0, BM), K, (int32_t)lda);
  const int nk = (K + kStage - 1) / kStage;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS char*)lds;

  // Where a lane's piece of an operand comes from.  Rows of 128 codes are 8
  // pieces; piece c of row r lies at place c ^ s(r), s = the lane's row in a
  // fragment & 7, so that the 8 lanes that read one bank width at a time read
  // 8 different places.
  const uint32_t va = (uint32_t)(lane >> 3) * lda + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  uint32_t vb[2];
  if constexpr (kNT) {
    // a fragment's row i16 is column (i16 / 4) * 8 + 4 (j % 2) + i16 % 4 of the 32 of two fragments, which leaves each
    // lane 8 consecutive columns of the result; so s(r) = r % 4 + 4 (r / 8 % 2)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      vb[p] = (uint32_t)(lane >> 3) * ldb + (uint32_t)(((lane & 7) ^ ((lane >> 3 & 3) | p << 2)) * 16);
  } else {
    // rows of K, BN codes each; s(r) = r % 8, or with 4 pieces a row r / 4 % 2 + 2 (r / 16 % 2)
    constexpr int kPer = BN / 16, kRows = 64 / kPer;  // pieces a row, rows a load
    static_assert(kPer >= 4 && kRows >= 1, "tile width");
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = lane / kPer + p * kRows;
      vb[p] = (uint32_t)(lane / kPer) * ldb + (uint32_t)(((lane % kPer) ^ place_nn<BN>(row)) * 16);
    }
  }

  // A stage past the last lies past the end of every buffer: zeros, and no traffic (offsets in a tile are below 2^31).
  auto from = [&](int stage) { return stage < nk ? (uint32_t)(stage * kStage) : 0x7FFFFFF0u; };
  auto load_a = [&](int stage, int j) {
    const int t = wave * kALoads + j;  // 8 rows each
    load_to_lds(ra, va + (uint32_t)(t * 8) * lda + from(stage), lds0 + (stage & (NS - 1)) * kBuf + t * 1024);
  };
  const int32_t cols = left_of(a.N, n0, BN);
  const Rsrc rb_nt = make_rsrc((const char*)a.b + n0 * a.ldb, cols, K, (int32_t)ldb);
  auto load_b = [&](int stage, int j) {
    const int t = wave * kBLoads + j;
    const uint32_t to = lds0 + (stage & (NS - 1)) * kBuf + kABytes;
    if constexpr (kNT) {
      load_to_lds(rb_nt, vb[t & 1] + (uint32_t)(t * 8) * ldb + from(stage), to + t * 1024);
    } else {
      constexpr int kRows = 64 / (BN / 16);
      const int32_t k0 = stage * kStage;
      const Rsrc rb = make_rsrc((const char*)a.b + k0 * a.ldb + n0, max(min(K - k0, kStage), 0), cols, (int32_t)ldb);
      load_to_lds(rb, vb[t & 1] + (uint32_t)(t * kRows) * ldb, to + t * kRows / 16 * kGroup + t * kRows % 16 * BN);
    }
  };

  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  i32x4 fa[2][FM], fb[2][FN];

  const int s7 = i16 & 7;
  const int at_a = (wm + i16) * kStage;
  const int at_b_nt = kABytes + (wn + (i16 >> 2) * 8 + (i16 & 3)) * kStage;
  const int at_b_nn = kABytes + g * kGroup + (i16 >> 1) * BN + (i16 & 1) * 8;
  auto read_a = [&](int buf, int half, int i) {
    fa[half][i] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_a + i * 16 * kStage + ((4 * half + g) ^ s7) * 16);
  };
  auto read_b = [&](int buf, int half, int j) {
    if constexpr (kNT) {
      fb[half][j] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_b_nt + (j / 2 * 32 + j % 2 * 4) * kStage +
                                        ((4 * half + g) ^ s7) * 16);
    } else {
      // rows r and r + 8 share s
      LDS char* p = (LDS char*)lds + buf * kBuf + at_b_nn + half * 4 * kGroup +
                    (((wn >> 4) + j) ^ place_nn<BN>(16 * g + (i16 >> 1))) * 16;
      const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)p);
      const i32x2 y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(p + 8 * BN));
      fb[half][j] = (i32x4){x[0], x[1], y[0], y[1]};
    }
  };
  // The last stage's codes past K are whatever the rows go on with: zero them in one operand.  (kNN: rows of b
  // past K are read as zeros.)
  auto cut = [&](int stage, int half) {
    if constexpr (kNT) {
      if (K % kStage != 0) {
        const int left = K - stage * kStage - half * 64 - 16 * g;
        i32x4 mask;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int b = left - 4 * d;
          mask[d] = b >= 4 ? -1 : b <= 0 ? 0 : (1 << (8 * b)) - 1;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[half][i] &= mask;
      }
    }
  };
  // The matrix instructions of one half of a stage, with the fragment reads of the next half and, in the second, the
  // memory loads of stage `stage` + NS (into the buffer of the present one) spread between them.
  constexpr int kLoads = kALoads + kBLoads, kMfma = FM * FN;
  auto half_step = [&](auto half_c, int stage) {
    constexpr int half = decltype(half_c)::value;
    const int buf_next = (stage + half) & (NS - 1);
    if (stage == nk - 1) cut(stage, half);
    for_each<kMfma>([&](auto at_c) {
      constexpr int at = decltype(at_c)::value, i = at / FN, j = at % FN;
      // the next fragments of a as the present ones come to their last use, those of b in the first half
      if constexpr (j == 0) read_a(buf_next, half ^ 1, i);
      for_each<FN>([&](auto r) {
        if constexpr (r >= at * 2 * FN / kMfma && r < (at + 1) * 2 * FN / kMfma) read_b(buf_next, half ^ 1, r);
      });
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[half][j], fa[half][i], acc[i][j], 0, 0, 0);
      if constexpr (half == 1) {
        for_each<kLoads>([&](auto l) {
          if constexpr (l >= at * kLoads / kMfma && l < (at + 1) * kLoads / kMfma) {
            if constexpr (l < kALoads)
              load_a(stage + NS, l);
            else
              load_b(stage + NS, l - kALoads);
          }
        });
      }
      if constexpr (at % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    });
  };
  // The ring: stage s lies in buffer s % NS; stage s + NS is loaded into it once every wave has read the last of s.
  if (nk > 0) {
#pragma unroll
    for (int p = 0; p < NS; ++p) {
#pragma unroll
      for (int j = 0; j < kALoads; ++j) load_a(p, j);
#pragma unroll
      for (int j = 0; j < kBLoads; ++j) load_b(p, j);
    }
    meet<(NS - 1) * kLoads>();
#pragma unroll
    for (int j = 0; j < FN; ++j) read_b(0, 0, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) read_a(0, 0, i);
    for (int s = 0; s < nk; ++s) {
      half_step(First{}, s);
      meet<(NS - 2) * kLoads>();  // all but the stages after the next have landed
      half_step(Second{}, s);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS when the workgroup ends
  }

  // Results: lane i16 holds row i16 of a fragment, 8 consecutive columns from two accumulators (kNN: after a trade),
  // so that a store covers 64 bytes of each of 16 rows (with 4 columns a lane, kNN took 4-20% longer: 148 us against 120
  // at 8192 x 4096 x 4096).
  constexpr int kRun = 8;
  float rs[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + i16;
    rs[i] = m < a.M ? ((const GLB float*)a.rs)[m] : 0.0f;
  }
#pragma unroll
  for (int c = 0; c < FN * 4 / kRun; ++c) {
    const int64_t n = n0 + wn + c * 32 + (kNT ? g * 8 : eight_at(g));
    float cs[kRun];
    if (a.cs != nullptr) {
#pragma unroll
      for (int r = 0; r < kRun; ++r) cs[r] = n + r < a.N ? ((const GLB float*)a.cs)[n + r] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = m0 + wm + i * 16 + i16;
      int32_t sum[kRun];
      if constexpr (kNT) {
#pragma unroll
        for (int r = 0; r < kRun; ++r) sum[r] = acc[i][2 * c + r / 4][r % 4];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t lo, hi;
          trade((uint32_t)acc[i][2 * c][r], (uint32_t)acc[i][2 * c + 1][r], lo, hi);
          sum[r] = (int32_t)lo;
          sum[4 + r] = (int32_t)hi;
        }
      }
      float v[kRun];
#pragma unroll
      for (int r = 0; r < kRun; ++r) {
        v[r] = (float)sum[r] * rs[i];
        if (a.cs != nullptr) v[r] = v[r] * cs[r];
      }
      if (m < a.M && n < a.N) store_run<kRun, PAST>(a, m, n, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows of x: 16 x 16 NT outputs per workgroup, whose W waves each take
// every W-th 64 codes of the summed axis, so that the weight's bytes are
// spread over many waves although the outputs are few.  No wave needs
// another's operands: kNT reads fragments from memory straight into
// registers; kNN moves them through a part of LDS of the wave's own, to turn
// the weight's rows.  The waves' sums meet in LDS (integer additions, whose
// order does not matter).  Bound by the weight's bytes: one token, N = 4096: K =
// 4096 in 6.1 us, 11008 in 10.8 (4.2 TB/s).  kNN, 61 tokens, 4096 x 4096: 10.4 us.
// ---------------------------------------------------------------------------
template <Q8Op OP, int NT, int W>
__global__ __launch_bounds__(W * 64, 2) void q8_gemm_split(const Q8Gemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr bool kNT = OP == Q8Op::kNT;
  constexpr int BM = 16, BN = NT * 16;
  static_assert(kNT || NT == 4, "four pieces in a row of b");
  constexpr int kPitch = BN + 4;                       // of the sums in LDS: lanes of an instruction in 64 banks
  constexpr int kSums = BM * kPitch * 4;
  constexpr int kStageBytes = kNT ? 0 : (1 + NT) * 1024;  // a wave's operands of one step
  constexpr int kLds = 2 * W * kStageBytes > kSums ? 2 * W * kStageBytes : kSums;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int32_t K = (int32_t)a.K, steps = (K + 63) / 64;
  const int32_t lda = (int32_t)a.lda, ldb = (int32_t)a.ldb, cols = left_of(a.N, n0, BN);
  const Rsrc ra = make_rsrc((const char*)a.a + m0 * a.lda, left_of(a.M, m0, BM), K, lda);

  i32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = (i32x4){0, 0, 0, 0};
  // codes of a past K, in the step that holds its end
  auto cut = [&](int step, i32x4& fa) {
    if (step * 64 + 64 > K) {
      const int left = K - step * 64 - 16 * g;
      i32x4 mask;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int b = left - 4 * d;
        mask[d] = b >= 4 ? -1 : b <= 0 ? 0 : (1 << (8 * b)) - 1;
      }
      fa &= mask;
    }
  };
  if constexpr (kNT) {
    const Rsrc rb = make_rsrc((const char*)a.b + n0 * a.ldb, cols, K, ldb);
    const uint32_t va = (uint32_t)(i16 * lda + g * 16), vb = (uint32_t)(i16 * ldb + g * 16);
    constexpr int kAhead = 4;  // steps in flight
    i32x4 fa[kAhead], fb[kAhead][NT];
    auto fetch = [&](int step, int u) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[u][j] = __builtin_bit_cast(i32x4, ld_buffer16(rb, vb + j * 16 * ldb + step * 64));
      fa[u] = __builtin_bit_cast(i32x4, ld_buffer16(ra, va + step * 64));
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(wave + u * W, u);
    for (int step = wave; step < steps; step += kAhead * W) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int at = step + u * W;
        if (at < steps) {
          cut(at, fa[u]);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][j], fa[u], acc[j], 0, 0, 0);
        }
        fetch(at + kAhead * W, u);
      }
    }
  } else {
    // a step's rows of a: 64 codes, 4 pieces, piece c of row r at place c ^ (r / 2 % 4); its 64 rows of b: four
    // pieces, at place c ^ s(r)
    const uint32_t mine = (uint32_t)(uintptr_t)(LDS char*)lds + wave * 2 * kStageBytes;
    auto s_of = [](int r) { return (r >> 2 & 1) | (r >> 4 & 1) << 1; };
    const uint32_t va = (uint32_t)((lane >> 2) * lda + ((lane & 3) ^ (lane >> 3 & 3)) * 16);
    auto fetch = [&](int step, int buf) {
      const int32_t k0 = step * 64;
      const Rsrc rb = make_rsrc((const char*)a.b + (int64_t)k0 * a.ldb + n0, K - k0 < 64 ? K - k0 : 64, cols, ldb);
      load_to_lds(ra, va + k0, mine + buf * kStageBytes);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int row = j * (64 / NT) + lane / NT;
        load_to_lds(rb, (uint32_t)(row * ldb + ((lane % NT) ^ s_of(row)) * 16),
                    mine + buf * kStageBytes + 1024 + j * 1024);
      }
    };
    int buf = 0;
    if (wave < steps) fetch(wave, 0);
    for (int step = wave; step < steps; step += W, buf ^= 1) {
      // what was read from the other buffer has been used
      if (step + W < steps) {
        fetch(step + W, buf ^ 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(1 + NT) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      LDS char* p = (LDS char*)lds + wave * 2 * kStageBytes + buf * kStageBytes;
      const i32x4 fa = *(LDS i32x4*)(p + i16 * 64 + (g ^ (i16 >> 1 & 3)) * 16);
      i32x4 fb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int row = 16 * g + (i16 >> 1);
        LDS char* q = p + 1024 + row * BN + (i16 & 1) * 8;
        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(q + (j ^ s_of(row)) * 16));
        const i32x2 y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(q + 8 * BN + (j ^ s_of(row + 8)) * 16));
        fb[j] = (i32x4){x[0], x[1], y[0], y[1]};
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa, acc[j], 0, 0, 0);
    }
    __syncthreads();  // the operands' LDS is done with
  }
  int32_t* sums = (int32_t*)lds;
  for (int i = tid; i < BM * kPitch; i += W * 64) sums[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      __hip_atomic_fetch_add(&sums[i16 * kPitch + (j * 4 + r) * 4 + g], acc[j][r], __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_WORKGROUP);
  __syncthreads();
  for (int i = tid; i < BM * (BN / 4); i += W * 64) {
    const int row = i / (BN / 4), four = i % (BN / 4);  // columns 4 * four .. + 3: j = four / 4, g = four % 4
    const int64_t m = m0 + row, n = n0 + four * 4;
    if (m >= a.M || n >= a.N) continue;
    const float rs = ((const GLB float*)a.rs)[m];
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = (float)sums[row * kPitch + (four / 4 * 4 + r) * 4 + four % 4] * rs;
      if (a.cs != nullptr && n + r < a.N) v[r] = v[r] * ((const GLB float*)a.cs)[n + r];
    }
    store_run<4>(a, m, n, v);
  }
}

template <Q8Op OP, int NT, int W>
hipError_t split_launch(const Q8Gemm& a, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((a.M + 15) / 16), tn = (uint32_t)((a.N + NT * 16 - 1) / (NT * 16));
  q8_gemm_split<OP, NT, W><<<dim3(tm * tn), W * 64, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

template <Q8Op OP, int BM, int BN, int WM, int WN, int NS>
hipError_t tile_launch(const Q8Gemm& a, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN);
  // 16-bit outputs in whole pieces of 64 bytes go past the caches, whatever their size: large ones otherwise push the
  // operands out of them (8192 x 11008 x 4096: 314 us against 361 when this was chosen, 8192 x 4096 x 4096: 122 against
  // 136, kNN 115 against 125), and smaller ones gain too, alone (4096 x 4096 x 4096: 58.0 against 61.7, 1000: 22.5 against
  // 23.7).  With a call behind them that reads the output, elementwise, the two together: 4096 x 4096 x 4096 68.5 against
  // 70.1 us, 2000 41.7 both, 1000 (8 MB) 27.5 against 26.4.  Weight gradients, smaller beside their operands, gain 1% or
  // lose 2%.  Pieces that are not whole 64 bytes lose by it: 1000 x 5003 in fp32, 25.8 us against 18.7.
  if constexpr (BM >= 128) {
    if (a.format != ZS_FORMAT_FP32 && ((uintptr_t)a.d | (uintptr_t)(a.ldd * 2)) % 64 == 0) {
      q8_gemm_tile<OP, BM, BN, WM, WN, NS, true><<<dim3(tm * tn), WM * WN * 64, 0, stream>>>(a, tm, tn);
      return hipGetLastError();
    }
  }
  q8_gemm_tile<OP, BM, BN, WM, WN, NS, false><<<dim3(tm * tn), WM * WN * 64, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

// Code rows that the tiled kernels take: 16-byte rows (a single row at any
// distance from the next), offsets within a tile below 2^31, a grid that a
// launch can hold.
bool rows16(const void* p, int64_t rows, int64_t ld) {
  return (uintptr_t)p % 16 == 0 && (rows <= 1 || (ld % 16 == 0 && ld <= (1 << 22)));
}
int64_t tiles_of(const Q8Gemm& a, int64_t bm, int64_t bn) { return (a.M + bm - 1) / bm * ((a.N + bn - 1) / bn); }
constexpr int64_t kMostTiles = 1 << 22;

// The tile of a product with 16-byte rows, by the time of one stage of 128
// codes that its grid needs in all, measured at K = 4096 and 11008 (us).  The
// rounds are of the MI355X's 256 compute units, here and in the rules below:
//   256 x 256, one workgroup a unit: 1.15-1.45 for a first round of up to 256
//     tiles, 1.7-1.9 a round where there are more;
//   128 x 128: 0.45-0.7 up to 256 tiles with four stages, beyond that two
//     workgroups of two stages a unit, 0.8-1.15 for each 512;
//   96 x 64: 0.36-0.40 up to 256 tiles, less than any other where 64 x 64 need
//     a second round; beyond 256 one of the others is as good or better (640 x
//     4096: 19.5 us, 128 x 128 18.2);
//   64 x 64: 0.25-0.33 up to 256 tiles, 0.45-0.5 for each 512.
// For example 8192 x 11008 by 4096: 346 / 407 / 616 us; 2000 x 4096: 44.7 /
// 36.2 / 59.5; 1000 x 4096: 42.4 / 21.8 / 31.2; 333 x 4096: 41.5 / 16.5 /
// 15.2, in 96 x 64 13.6 (K = 11008: 37.4, in 96 x 64 31.4); 61 x 11008: 38.6 / 16.2 / 10.7.
enum class Tile { k64, k96, k128, k128Far, k256 };
Tile tile_for(const Q8Gemm& a) {
  const auto rounds = [](int64_t t, int64_t at_once) { return (double)((t + at_once - 1) / at_once); };
  const int64_t t64 = tiles_of(a, 64, 64), t96 = tiles_of(a, 96, 64), t128 = tiles_of(a, 128, 128), t256 = tiles_of(a, 256, 256);
  const double c64 = t64 <= 256 ? 0.30 : 0.475 * rounds(t64, 512);
  const double c128 = t128 <= 256 ? 0.50 + 0.18 * (double)t128 / 256 : t128 <= 512 ? 0.65 + 0.45 * (double)t128 / 512 : 1.1 * rounds(t128, 512);
  const double c256 = t256 <= 256 ? 1.40 : 1.8 * rounds(t256, 256);
  if (t64 > 256 && t96 <= 256) return Tile::k96;
  if (c64 <= c128 && c64 <= c256) return Tile::k64;
  if (c128 <= c256) return t128 <= 256 ? Tile::k128Far : Tile::k128;
  return Tile::k256;
}

template <Q8Op OP>
hipError_t product_launch(const Q8Gemm& given, hipStream_t stream) {
  Q8Gemm a = given;
  const int64_t rows_b = OP == Q8Op::kNT ? a.N : a.K;
  // (an empty sum goes there too: its operands may be NULL, and q8_gemm_split fetches before it looks at the length)
  if (a.K == 0 || !rows16(a.a, a.M, a.lda) || !rows16(a.b, rows_b, a.ldb) || tiles_of(a, 64, 64) >= kMostTiles)
    return any_launch<OP, kBF16>(a, stream);
  // a single row: any distance that holds what a tile reads of it
  if (a.M <= 1) a.lda = (a.K + 15) / 16 * 16;
  if (rows_b <= 1) a.ldb = OP == Q8Op::kNT ? (a.K + 15) / 16 * 16 : 256;
  // Few rows: their tiles of 64 columns may be too few to draw on all of the memory.  kNT, K = 4096: one token 6.2 us
  // against 9.2 in 64 x 64 tiles for N = 4096, 11.8 against 10.0 for N = 11008; 16 tokens 7.8 / 9.4 and 16.3 / 9.8.  From
  // 17 tokens on the split kernel's rows of tiles read the weight again: 17 and 61 tokens, 4096 x 4096: 11.3 and 20.0 us
  // against 10.1 and 10.3; 4096 x 11008: 23.4 and 44.0 against 21.5 and 21.8 (only a weight too narrow for that would
  // gain: 1024 x 11008, 12.9 and 13.0 against 21.2 and 21.4).
  // kNN, tiles of 16 x 64: 61 tokens 10.1 / 13.4 for 4096 columns (256 tiles), 21.0 / 14.2 for 11008 (688); 16 tokens
  // 11.2 / 12.3 for 11008 (172), 32 tokens 17.1 / 12.7 (344).
  if constexpr (OP == Q8Op::kNT) {
    if (a.M <= 16 && (a.N + 63) / 64 <= 96) return split_launch<OP, 1, 4>(a, stream);
  } else {
    if (tiles_of(a, 16, 64) <= 256) return split_launch<OP, 4, 8>(a, stream);
  }
  switch (tile_for(a)) {
    case Tile::k64: return tile_launch<OP, 64, 64, 4, 1, 4>(a, stream);
    case Tile::k96: return tile_launch<OP, 96, 64, 2, 2, 4>(a, stream);
    case Tile::k128Far: return tile_launch<OP, 128, 128, 4, 2, 4>(a, stream);
    case Tile::k128: return tile_launch<OP, 128, 128, 2, 2, 2>(a, stream);
    default: return tile_launch<OP, 256, 256, 2, 4, 2>(a, stream);
  }
}

// ---------------------------------------------------------------------------
// The weight gradient in tiles of BM x BN by WM x WN waves, 64 rows of tokens
// a stage and two stages, by the schedule of q8_gemm_tile.  Both operands lie
// as they do in memory, a token's values side by side, and are turned by the
// transposing LDS reads.  The codes go through registers, where they become
// bf16 once for the whole workgroup (in the fragments each wave would convert
// them again).  dy goes to LDS directly (kDirect), or through registers: as two
// bf16 parts of 32 tokens a stage when it is fp16 (kParts, kPartsAny), or as it
// is (kThrough).  kDirect and kParts want rows on 16-byte boundaries, the others
// take any.
//
// kDirect, 256 x 256: T, N, K = 8192, 11008, 4096 in 619-699 us (1060-1190
// TFLOP/s; a library's bf16 product of the same layout 795), 8192, 4096, 4096 in
// 224-269.  Of 236 for the latter, the matrix instructions took 136 and with the
// fragments' reads 181; the codes' fetch added 30, dy's loads 17, the conversion 8:
// a fetch waits on memory for more than the stage that it has.  Slower: 32-token
// stages in a ring of four with the codes loaded to LDS as they are (256); the
// waves in two groups half a stage apart (311); the codes fetched after dy's loads,
// with the same wait for all of them (284).  Bank conflicts of the transposing
// reads are 20-25% of the LDS cycles.  kParts (fp16) 1228-1288; rows one element
// off, 8192, 4096, 4096: kThrough 409-433, kPartsAny 669-692.
// ---------------------------------------------------------------------------
enum class DyPath { kDirect, kParts, kThrough, kPartsAny };

template <DyPath PATH, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void q8_grad_tile(const Q8Gemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr int kThreads = WM * WN * 64, kWaves = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool kTwo = PATH == DyPath::kParts || PATH == DyPath::kPartsAny;
  constexpr bool kAligned = PATH == DyPath::kDirect || PATH == DyPath::kParts;
  constexpr int kRows = kTwo ? 32 : 64;  // tokens a stage
  // 8 rows, and 128 bytes that put the next 8 in the other half of the banks
  constexpr int kGroup = 8 * BM * 2 + 128;
  constexpr int kABytes = 8 * kGroup, kBuf = 2 * kABytes;
  constexpr int kPer = BM / 8;                                   // pieces of 16 bytes in a row of dy
  constexpr int kALoads = 64 * BM * 2 / 1024 / kWaves;           // direct loads of a wave a stage
  constexpr int kAPieces = kRows * kPer / kThreads;              // pieces of dy of a thread a stage
  constexpr int kXPieces = kRows * (BN / 16) / kThreads;         // pieces of codes of a thread a stage
  constexpr int kARows = kThreads / kPer, kXRows = kThreads / (BN / 16);  // rows from a thread's piece to its next
  static_assert(kALoads > 0 && kAPieces > 0 && kXPieces > 0 && kPer >= 16 && kARows % 8 == 0 && kXRows % 8 == 0,
                "tile shape");
  __shared__ __attribute__((aligned(1024))) char lds[2 * kBuf];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int wm = wave / WN * TM, wn = wave % WN * TN;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int32_t T = (int32_t)a.K;
  const int nk = (int)(((int64_t)T + kRows - 1) / kRows);
  // tokens left at a stage (the difference is right even where stage * kRows passes 2^31)
  auto rows_at = [&](int stage) {
    const int32_t n = (int32_t)((uint32_t)T - (uint32_t)stage * (uint32_t)kRows);
    return n < kRows ? n : kRows;
  };
  const int32_t wide_a = left_of(a.M, m0, BM) * 2, wide_b = left_of(a.N, n0, BN);
  const int32_t pitch_a = (int32_t)a.lda * 2, pitch_b = (int32_t)a.ldb;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS char*)lds;

  // Piece c of row r lies at place c ^ s(r).  A transposing read takes 32
  // bytes of 4 consecutive rows, and of 4 that lie 8 rows on, per 32 lanes: s puts those 4 at different places.
  auto s_of = [](int row) { return (row & 3) << 1; };
  auto at_row = [](int row) { return row / 8 * kGroup + row % 8 * BM * 2; };

  auto rsrc_a = [&](int stage) {
    return make_rsrc((const char*)a.a + ((int64_t)stage * kRows * a.lda + m0) * 2, rows_at(stage), wide_a, pitch_a);
  };
  // dy, directly: a load is 64 / kPer rows; loads 4 rows apart share s
  constexpr int kApart = 4 / (64 / kPer);
  uint32_t va[kApart];
  if constexpr (PATH == DyPath::kDirect) {
#pragma unroll
    for (int j = 0; j < kApart; ++j) {
      const int row = (wave * kALoads + j) * (64 / kPer) + lane / kPer;
      va[j] = (uint32_t)row * (uint32_t)pitch_a + (uint32_t)(((lane % kPer) ^ s_of(row)) * 16);
    }
  }
  auto direct_a = [&](int stage, int j) {
    load_to_lds(rsrc_a(stage), va[j % kApart] + (uint32_t)(j / kApart * 4) * (uint32_t)pitch_a,
                lds0 + (stage & 1) * kBuf + at_row((wave * kALoads + j) * (64 / kPer)));
  };
  // dy, through registers: a thread's pieces lie kARows rows apart, at places that many groups apart
  u32x4 ar[PATH == DyPath::kDirect ? 1 : kAPieces];
  const int row_a = tid / kPer, row_x = tid / (BN / 16);
  auto fetch_a = [&](int stage, int c) {
    if constexpr (kAligned) {
      ar[c] = ld_buffer16(rsrc_a(stage), (uint32_t)(row_a * pitch_a + tid % kPer * 16) + (uint32_t)(c * kARows * pitch_a));
    } else {
      const int64_t t = (int64_t)stage * kRows + row_a + c * kARows;
      ar[c] = ld_piece<2>((const char*)a.a + t * a.lda * 2, m0 * 2 + tid % kPer * 16, a.M * 2, t < T);
    }
  };
  auto put_a = [&](int stage, int c) {
    LDS char* to = (LDS char*)lds + ((stage & 1) * kBuf + at_row(row_a) + ((tid % kPer) ^ s_of(row_a)) * 16) +
                   c * kARows / 8 * kGroup;
    if constexpr (kTwo) {
      u32x4 hi, lo;
      fp16_parts(ar[c], hi, lo);
      *(LDS u32x4*)to = hi;
      *(LDS u32x4*)(to + 4 * kGroup) = lo;  // 32 rows on: the same s
    } else {
      *(LDS u32x4*)to = ar[c];
    }
  };
  // codes, the same way
  u32x4 xr[kXPieces];
  float xs[kXPieces];
  auto fetch_x = [&](int stage, int c) {
    if constexpr (kAligned) {
      const int64_t t0 = (int64_t)stage * kRows;
      const int32_t rows = rows_at(stage);
      xr[c] = ld_buffer16(make_rsrc((const char*)a.b + t0 * a.ldb + n0, rows, wide_b, pitch_b),
                          (uint32_t)(row_x * pitch_b + tid % (BN / 16) * 16) + (uint32_t)(c * kXRows * pitch_b));
      xs[c] = ld_buffer4(make_rsrc(a.rs + t0, rows, 4, 4), (uint32_t)(row_x * 4) + c * kXRows * 4);
    } else {
      const int64_t t = (int64_t)stage * kRows + row_x + c * kXRows;
      xr[c] = ld_piece<1>((const char*)a.b + t * a.ldb, n0 + tid % (BN / 16) * 16, a.N, t < T);
      xs[c] = t < T ? ((const GLB float*)a.rs)[t] : 0.0f;
    }
  };
  auto put_x = [&](int stage, int c, int part) {  // part: 8 of a piece's 16 codes
    LDS char* to = (LDS char*)lds +
                   ((stage & 1) * kBuf + kABytes + at_row(row_x) + ((tid % (BN / 16) * 2) ^ s_of(row_x)) * 16) +
                   c * kXRows / 8 * kGroup;
    *(LDS u32x4*)(to + part * 16) = codes_to_bf16(xr[c][2 * part], xr[c][2 * part + 1], xs[c]);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  bf16x8 fa[2][FM], fb[2][FN];
  // A lane's place in the rows of a read, for each of the four values that s leaves of a fragment's first piece.
  // A and b have rows of one width, so these serve both.
  static_assert(BM == BN && TM % 64 == 0 && TN % 64 == 0, "one set of places");
  uint32_t place[4];
#pragma unroll
  for (int v = 0; v < 4; ++v)
    place[v] = (uint32_t)(g * kGroup + (i16 >> 2) * BM * 2 + ((2 * v + (i16 >> 1 & 1)) ^ (i16 >> 2) << 1) * 16 + (i16 & 1) * 8);
  auto turned = [&](uint32_t at, int col16) {  // 8 tokens (4 and 4) of the 16 columns from 16 * col16
    LDS char* p = (LDS char*)lds + (place[col16 & 3] + at) + (col16 >> 2) * 128;
    const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)p);
    const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(p + 4 * BM * 2));
    return __builtin_bit_cast(bf16x8, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
  };
  auto read_a = [&](int buf, int half, int i) {
    fa[half][i] = turned((uint32_t)(buf * kBuf + half * 4 * kGroup + wm * 2), i);
  };
  auto read_b = [&](int buf, int half, int j) {  // both parts of dy meet the same codes
    fb[half][j] = turned((uint32_t)(buf * kBuf + kABytes + (kTwo ? 0 : half * 4) * kGroup + wn * 2), j);
  };

  constexpr int kMfma = FM * FN;
  constexpr int kMoves = (PATH == DyPath::kDirect ? kALoads : kAPieces) + 2 * kXPieces;
  static_assert(kMoves <= kMfma && 2 * FN <= kMfma, "at most one move beside an instruction");
  auto half_step = [&](auto half_c, auto read_c, auto load_c, int buf_next, int stage) {
    constexpr int half = decltype(half_c)::value;
    for_each<kMfma>([&](auto at_c) {
      constexpr int at = decltype(at_c)::value, i = at / FN, j = at % FN;
      if constexpr (decltype(read_c)::value) {
        if constexpr (j == 0) read_a(buf_next, half ^ 1, i);
        // b's fragments in the second half of the instructions
        constexpr int lo = at * 2 * FN / kMfma - FN, hi = (at + 1) * 2 * FN / kMfma - FN;
        if constexpr (lo >= 0 && hi > lo) read_b(buf_next, half ^ 1, lo);
      }
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[half][j], fa[half][i], acc[i][j], 0, 0, 0);
      if constexpr (decltype(load_c)::value) {
        // what was fetched for `stage` goes to LDS and its place is fetched again for the stage after it
        constexpr int l = at * kMoves / kMfma;
        if constexpr ((at + 1) * kMoves / kMfma > l) {
          if constexpr (l < 2 * kXPieces) {
            put_x(stage, l / 2, l % 2);
            if constexpr (l % 2) fetch_x(stage + 1, l / 2);
          } else if constexpr (PATH == DyPath::kDirect) {
            direct_a(stage, l - 2 * kXPieces);
          } else {
            put_a(stage, l - 2 * kXPieces);
            fetch_a(stage + 1, l - 2 * kXPieces);
          }
        }
      }
      if constexpr (at % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto fetch = [&](int stage) {
#pragma unroll
    for (int c = 0; c < kXPieces; ++c) fetch_x(stage, c);
    if constexpr (PATH != DyPath::kDirect) {
#pragma unroll
      for (int c = 0; c < kAPieces; ++c) fetch_a(stage, c);
    }
  };
  auto put = [&](int stage) {
#pragma unroll
    for (int c = 0; c < 2 * kXPieces; ++c) put_x(stage, c / 2, c % 2);
    if constexpr (PATH == DyPath::kDirect) {
#pragma unroll
      for (int j = 0; j < kALoads; ++j) direct_a(stage, j);
    } else {
#pragma unroll
      for (int c = 0; c < kAPieces; ++c) put_a(stage, c);
    }
  };
  if (nk > 0) {
    fetch(0);
    put(0);
    fetch(1);
    meet<0>();
    if (nk > 1) put(1);
    fetch(2);
#pragma unroll
    for (int j = 0; j < FN; ++j) read_b(0, 0, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) read_a(0, 0, i);
    int k = 0;
    for (; k < nk - 2; ++k) {
      half_step(First{}, Yes{}, No{}, k & 1, 0);
      meet<0>();
      half_step(Second{}, Yes{}, Yes{}, (k + 1) & 1, k + 2);
    }
    if (k < nk - 1) {
      half_step(First{}, Yes{}, No{}, k & 1, 0);
      meet<0>();
      half_step(Second{}, Yes{}, No{}, (k + 1) & 1, 0);
      ++k;
    }
    half_step(First{}, Yes{}, No{}, k & 1, 0);
    half_step(Second{}, No{}, No{}, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + i16;
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t lo, hi;
        trade(__float_as_uint(acc[i][j][r]), __float_as_uint(acc[i][j + 1][r]), lo, hi);
        v[r] = __uint_as_float(lo);
        v[4 + r] = __uint_as_float(hi);
      }
      const int64_t n = n0 + wn + j * 16 + eight_at(g);
      if (m < a.M && n < a.N) store_run<8>(a, m, n, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Small weights, many tokens: 64 x 64 outputs per workgroup, whose eight waves
// each take every eighth 32 tokens, with a part of LDS of their own that they
// load three steps ahead and read through transposing reads: no wave waits for
// another until their sums are added, in the waves' order.  The codes become
// bf16 in the fragments: no other wave needs them.  T, N, K = 8192, 256, 256: 26
// us (in 128 x 128 tiles 105), bound by the loads' latency on the 16 compute
// units that 16 workgroups use.
// ---------------------------------------------------------------------------
template <bool TWO>
__global__ __launch_bounds__(512, 2) void q8_grad_split(const Q8Gemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr int kWaves = 8, kRows = 32, kAhead = 3, kOps = 7;
  constexpr int kAtX = kRows * 128, kAtS = kAtX + kRows * 64, kBuf = kAtS + 256;
  constexpr int kPitch = 68;  // floats from row to row of the sums
  constexpr int kLds = kWaves * kAhead * kBuf > kWaves * 64 * kPitch * 4 ? kWaves * kAhead * kBuf : kWaves * 64 * kPitch * 4;
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * 64, n0 = (int64_t)tn * 64;
  const int32_t T = (int32_t)a.K;
  const int steps = (int)(((int64_t)T + kRows - 1) / kRows);
  const int32_t wide_a = left_of(a.M, m0, 64) * 2, wide_b = left_of(a.N, n0, 64);
  const int32_t pitch_a = (int32_t)a.lda * 2, pitch_b = (int32_t)a.ldb;
  const uint32_t mine = (uint32_t)(uintptr_t)(LDS char*)lds + wave * kAhead * kBuf;
  // piece c of row r at place c ^ s(r): the rows that 32 lanes read at a time in different banks
  auto s_a = [](int r) { return (r >> 1 & 1) << 1 | (r >> 3 & 1) << 2; };
  auto s_x = [](int r) { return (r >> 2 & 1) | (r >> 3 & 1) << 1; };
  auto fetch = [&](int step, int buf) {
    const int64_t t0 = (int64_t)step * kRows;
    // the difference is right even where step * kRows passes 2^31
    const int32_t left = (int32_t)((uint32_t)T - (uint32_t)step * (uint32_t)kRows), rows = max(min(left, kRows), 0);
    const Rsrc ra = make_rsrc((const char*)a.a + (t0 * a.lda + m0) * 2, rows, wide_a, pitch_a);
    const Rsrc rx = make_rsrc((const char*)a.b + t0 * a.ldb + n0, rows, wide_b, pitch_b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = j * 8 + (lane >> 3);
      load_to_lds(ra, (uint32_t)(row * pitch_a + ((lane & 7) ^ s_a(row)) * 16), mine + buf * kBuf + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = j * 16 + (lane >> 2);
      load_to_lds(rx, (uint32_t)(row * pitch_b + ((lane & 3) ^ s_x(row)) * 16), mine + buf * kBuf + kAtX + j * 1024);
    }
    load4_to_lds(make_rsrc(a.rs + t0, rows, 4, 4), (uint32_t)lane * 4, mine + buf * kBuf + kAtS);
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < kAhead; ++p) fetch(wave + p * kWaves, p);
  int buf = 0;
  for (int step = wave; step < steps; step += kWaves) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * kOps) : "memory");
    LDS char* p = (LDS char*)lds + (wave * kAhead + buf) * kBuf;
    const f32x4 s0 = *(LDS f32x4*)(p + kAtS + g * 32), s1 = *(LDS f32x4*)(p + kAtS + g * 32 + 16);
    i32x2 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 8 * g + (i16 >> 1);
      q[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS i32x2*)(p + kAtX + row * 64 + (j ^ s_x(row)) * 16 + (i16 & 1) * 8));
    }
    bf16x8 fa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * g + (i16 >> 2);
      LDS char* r = p + row * 128 + ((2 * i + (i16 >> 1 & 1)) ^ s_a(row)) * 16 + (i16 & 1) * 8;
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)r);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(r + 4 * 128));
      fa[i] = __builtin_bit_cast(bf16x8, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // all of the buffer is read
    fetch(step + kAhead * kWaves, buf);
    bf16x8 fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c = (uint32_t)q[j][k / 2] >> (16 * (k % 2));
        const f32x4& sc = k < 2 ? s0 : s1;
        w[k] = pack_bf16((float)(int8_t)c * sc[k % 2 * 2], (float)(int8_t)(c >> 8) * sc[k % 2 * 2 + 1]);
      }
      fb[j] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TWO) {
        u32x4 hi, lo;
        fp16_parts(__builtin_bit_cast(u32x4, fa[i]), hi, lo);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], __builtin_bit_cast(bf16x8, hi), acc[i][j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], __builtin_bit_cast(bf16x8, lo), acc[i][j], 0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
    buf = buf == kAhead - 1 ? 0 : buf + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS
  __syncthreads();
  float* sums = (float*)lds;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *(f32x4*)(sums + (wave * 64 + i * 16 + i16) * kPitch + j * 16 + g * 4) = acc[i][j];
  __syncthreads();
  const int row = tid / 8, col = tid % 8 * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int w = 0; w < kWaves; ++w) {
    const f32x4 x = *(const f32x4*)(sums + (w * 64 + row) * kPitch + col);
    const f32x4 y = *(const f32x4*)(sums + (w * 64 + row) * kPitch + col + 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = v[r] + x[r], v[4 + r] = v[4 + r] + y[r];
  }
  if (m0 + row < a.M && n0 + col < a.N) store_run<8>(a, m0 + row, n0 + col, v);
}

hipError_t grad_split_launch(const Q8Gemm& a, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((a.M + 63) / 64), tn = (uint32_t)((a.N + 63) / 64);
  if (a.a_format == ZS_FORMAT_FP16)
    q8_grad_split<true><<<dim3(tm * tn), 512, 0, stream>>>(a, tm, tn);
  else
    q8_grad_split<false><<<dim3(tm * tn), 512, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

template <DyPath PATH, int BM, int BN, int WM, int WN>
hipError_t grad_tile_launch(const Q8Gemm& a, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN);
  q8_grad_tile<PATH, BM, BN, WM, WN><<<dim3(tm * tn), WM * WN * 64, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

// The weight gradient's kernel, by the time its grid needs for T tokens, in
// stages of 64 (us, measured on 256 compute units at T = 1 to 16384; fp16, whose
// stages are 32 tokens, takes 1.7 to 2 times as long in each):
//   64 x 64, tokens split over eight waves: 3.5 and 0.25 a stage for each 256
//   128 x 128: 4.5 and 0.85 a stage up to 256 tiles, 1.12 for each 512
//   256 x 256: 8 and 1.4 a stage up to 128 tiles, 1.85 for each 256
// For example (T, N, K) = 8192, 1024, 1024: 33 / 111 / 171 us; 1025, 1376, 4096:
// 42 / 24.5 / 31; 2000, 4096, 4096: 153 / 85 / 63; 100, 4096, 4096: 60 / 14.5 /
// 13.1; 77, 1001, 517: 5.3 / 5.7 / 11.8.
enum class GradTile { kSplit, k128, k256 };
GradTile grad_tile_for(const Q8Gemm& a) {
  const auto rounds = [](int64_t t, int64_t at_once) { return (double)((t + at_once - 1) / at_once); };
  const int64_t t64 = tiles_of(a, 64, 64), t128 = tiles_of(a, 128, 128), t256 = tiles_of(a, 256, 256);
  const double stages = (double)((a.K + 63) / 64);
  const double split = (3.5 + 0.25 * stages) * rounds(t64, 256);
  const double c128 = (4.5 + (t128 <= 256 ? 0.85 : 1.12) * stages) * rounds(t128, 512);
  const double c256 = (8.0 + (t256 <= 128 ? 1.4 : 1.85) * stages) * rounds(t256, 256);
  if (split <= c128 && split <= c256) return GradTile::kSplit;
  return c128 <= c256 ? GradTile::k128 : GradTile::k256;
}

hipError_t grad_launch(const Q8Gemm& given, hipStream_t stream) {
  Q8Gemm a = given;
  const bool two = a.a_format == ZS_FORMAT_FP16;
  const int64_t tiles = tiles_of(a, 128, 128);
  if (!rows16(a.a, a.K, a.lda * 2) || !rows16(a.b, a.K, a.ldb) || tiles_of(a, 64, 64) >= kMostTiles) {
    // rows at any address: the kernel of 64 x 64 tiles spreads a small weight over more compute units
    if (tiles < 64 || tiles >= kMostTiles)
      return two ? any_launch<Q8Op::kTN, kFP16>(a, stream) : any_launch<Q8Op::kTN, kBF16>(a, stream);
    return two ? grad_tile_launch<DyPath::kPartsAny, 128, 128, 2, 2>(a, stream)
               : grad_tile_launch<DyPath::kThrough, 128, 128, 2, 2>(a, stream);
  }
  if (a.K <= 1) a.lda = a.ldb = 256;  // a single row: any distance that holds what a tile reads of it
  switch (grad_tile_for(a)) {
    case GradTile::kSplit: return grad_split_launch(a, stream);
    case GradTile::k128:
      return two ? grad_tile_launch<DyPath::kParts, 128, 128, 2, 2>(a, stream)
                 : grad_tile_launch<DyPath::kDirect, 128, 128, 2, 2>(a, stream);
    default:
      return two ? grad_tile_launch<DyPath::kParts, 256, 256, 2, 4>(a, stream)
                 : grad_tile_launch<DyPath::kDirect, 256, 256, 2, 4>(a, stream);
  }
}

}  // namespace

hipError_t launch_q8_gemm(Q8Op op, const Q8Gemm& a, hipStream_t stream) {
  switch (op) {
    case Q8Op::kNT: return product_launch<Q8Op::kNT>(a, stream);
    case Q8Op::kNN: return product_launch<Q8Op::kNN>(a, stream);
    default: return grad_launch(a, stream);
  }
}

}  // namespace zs
