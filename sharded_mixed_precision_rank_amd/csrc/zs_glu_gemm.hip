// The products of the gated feed-forward block.
//
//   kForward  h = act(x Wg^T) * (x Wu^T)          both projections in one kernel, gate and up kept where asked for
//   kInput    dx = dgate Wg + dup Wu              one sum over both
//   kWeight   dWg = dgate^T x, dWu = dup^T x      (+ earlier micro-batches' sums), two products in one launch
//
// Operands are bf16 or fp16, sums fp32, each output rounded once.
#include "zs_act.h"
#include "zs_glu.h"
#include "zs_tile_dev.h"

namespace zs {
namespace {

using namespace dev;
using namespace glu;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// c[r] += sum over 32 k of b's row 4 g + r and a's row i16, of two 16 x 32
// fragments: lane (g, i16) holds row i16, k = 8 g .. 8 g + 7 of each.
template <int FMT>
__device__ __forceinline__ f32x4 mfma16(i32x4 b, i32x4 a, f32x4 c) {
  if constexpr (FMT == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}

// RUN (4 or 8) results from element i on, of which the first `left` exist, plus
// what add holds there.  PAST: around the caches, for 16-bit formats.
template <int FMT, int RUN, bool PAST>
__device__ __forceinline__ void store_run_as(void* d, const void* add, int64_t i, int64_t left, const float* x) {
  float v[RUN];
#pragma unroll
  for (int r = 0; r < RUN; ++r) v[r] = x[r];
  if (left >= RUN) {
    if (add != nullptr) {
#pragma unroll
      for (int r = 0; r < RUN; r += 4) {
        if constexpr (FMT == kFP32) {
          const f32x4 w = ld_any<f32x4>((const float*)add + i + r);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[r + k] = w[k] + v[r + k];
        } else {
          const u32x2 w = ld_any<u32x2>((const uint16_t*)add + i + r);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[r + k] = (k % 2 ? h_hi<FMT>(w[k / 2]) : h_lo<FMT>(w[k / 2])) + v[r + k];
        }
      }
    }
    if constexpr (FMT == kFP32) {
#pragma unroll
      for (int r = 0; r < RUN; r += 4) st_four<FMT>(d, i + r, v + r);
    } else if constexpr (RUN == 8) {
      const u32x4 w = {pack_two<FMT>(v[0], v[1]), pack_two<FMT>(v[2], v[3]), pack_two<FMT>(v[4], v[5]),
                       pack_two<FMT>(v[6], v[7])};
      if constexpr (PAST)
        st_past((uint16_t*)d + i, w);
      else
        st_any((uint16_t*)d + i, w);
    } else {
      st_four<FMT>(d, i, v);
    }
  } else {
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      if (r < left) st_elem<FMT>(d, i + r, add != nullptr ? ld_elem<FMT>(add, i + r) + v[r] : v[r]);
    }
  }
}
// The same in the weight gradient's output format, which need not be the operands'.
template <int FMT, int RUN>
__device__ __forceinline__ void store_grad(const GluGemm& a, int p, int64_t i, int64_t left, const float* v) {
  if (a.out_format == ZS_FORMAT_FP32)
    store_run_as<kFP32, RUN, false>(a.out[p], a.add[p], i, left, v);
  else if (a.out_format == ZS_FORMAT_BF16)
    store_run_as<kBF16, RUN, false>(a.out[p], a.add[p], i, left, v);
  else
    store_run_as<kFP16, RUN, false>(a.out[p], a.add[p], i, left, v);
}
// h, and gate and up where they are kept, at row m from column n on.
template <int FMT, int RUN, bool PAST>
__device__ __forceinline__ void store_gated(const GluGemm& a, int64_t m, int64_t n, const float* gate, const float* up) {
  if (m >= a.M || n >= a.N) return;
  float h[RUN], none[RUN];
  switch (a.act) {
    case ZS_ACT_SILU: acts_of<ZS_ACT_SILU, false, RUN>(gate, h, none); break;
    case ZS_ACT_GELU: acts_of<ZS_ACT_GELU, false, RUN>(gate, h, none); break;
    case ZS_ACT_GELU_TANH: acts_of<ZS_ACT_GELU_TANH, false, RUN>(gate, h, none); break;
    default: acts_of<ZS_ACT_RELU, false, RUN>(gate, h, none);
  }
#pragma unroll
  for (int r = 0; r < RUN; ++r) h[r] = h[r] * up[r];
  store_run_as<FMT, RUN, PAST>(a.out[0], nullptr, m * a.ldo[0] + n, a.N - n, h);
  if (a.out[1] != nullptr) {
    store_run_as<FMT, RUN, PAST>(a.out[1], nullptr, m * a.ldo[1] + n, a.N - n, gate);
    store_run_as<FMT, RUN, PAST>(a.out[2], nullptr, m * a.ldo[2] + n, a.N - n, up);
  }
}

// Values of a fragment's dwords past the end of the summed axis: `left` of the lane's 8 are inside.
__device__ __forceinline__ i32x4 inside(int left) {
  i32x4 mask;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int n = left - 2 * d;
    mask[d] = n >= 2 ? -1 : n == 1 ? 0xFFFF : 0;
  }
  return mask;
}

// ---------------------------------------------------------------------------
// Rows at any address, few tiles: 64 x 64 sums per workgroup of four waves (32 x 32 each),
// operands staged through registers 16 bytes at a time, 64 of the summed axis a
// stage, four stages ahead of the matrix instructions; two buffers in LDS and
// one barrier a stage.  Forward: 32 columns of gate beside the same 32 of up.
// (Addresses and bounds of four stages are more scalar values than there are
// registers: 64 of them forward, 106 in the input gradient lie in lanes of vector
// registers, none in memory.)
// ---------------------------------------------------------------------------
constexpr int kAnyTile = 64;

template <GluOp OP, int FMT>
__global__ __launch_bounds__(256) void glu_any(const GluGemm a, int64_t tiles_n, int64_t tiles) {
  constexpr bool kForward = OP == GluOp::kForward, kInput = OP == GluOp::kInput, kWeight = OP == GluOp::kWeight;
  constexpr bool kARow = !kWeight, kBRow = kForward;
  constexpr int kOutN = kForward ? 32 : 64, kAhead = 4;
  __shared__ __attribute__((aligned(16))) char lds[2][2][8192];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int g = lane >> 4, i16 = lane & 15;
  const int64_t nk = (a.K + kStage - 1) / kStage, stages = kInput ? 2 * nk : nk;
  const int64_t all = kWeight ? 2 * tiles : tiles;
  for (int64_t at = blockIdx.x; at < all; at += gridDim.x) {
    const int out = at >= tiles ? 1 : 0;
    const int64_t tile = at - out * tiles;
    const int64_t m0 = tile / tiles_n * kAnyTile, n0 = tile % tiles_n * kOutN;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
    u32x4 ra[kAhead][2], rb[kAhead][2];
    // A thread's pieces: rows tid / 8 and 32 on, bytes tid % 8 * 16
    const int row = tid / 8, col = tid % 8 * 16;
    // Forward, inside the summed axis: no bounds to look at (490 x 752 x 7392, rows one element off: 50 us, was 126; the
    // others lost by a second path).  Rows behind the last, whose sums are not stored, are the last one again.
    const char* fast_a[2] = {};
    const char* fast_b[2] = {};
    if constexpr (kForward) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t m = m0 + row + 32 * c, n = n0 + row;  // (rows 0 .. 31 of gate, then of up)
        fast_a[c] = (const char*)a.a[0] + (m < a.M ? m : a.M - 1) * a.lda * 2 + col;
        fast_b[c] = (const char*)a.b[c] + (n < a.N ? n : a.N - 1) * a.ldb * 2 + col;
      }
    }
    auto fetch = [&](int64_t stage, int u) {
      const bool second = kInput && stage >= nk, live = stage < stages;
      const int64_t k0 = (second ? stage - nk : stage) * kStage;
      if constexpr (kForward) {
        if (k0 + kStage <= a.K) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            ra[u][c] = ld_any<u32x4>((const uint16_t*)(fast_a[c] + k0 * 2));
            rb[u][c] = ld_any<u32x4>((const uint16_t*)(fast_b[c] + k0 * 2));
          }
          return;
        }
      }
      const char* base_a = (const char*)a.a[kForward ? 0 : kWeight ? out : second];
      const char* base_b = (const char*)a.b[kInput ? second : 0];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t k = k0 + row + 32 * c;
        if constexpr (kARow) {
          const int64_t m = m0 + row + 32 * c;
          ra[u][c] = ld_piece<2>(base_a + m * a.lda * 2, k0 * 2 + col, a.K * 2, live && m < a.M);
        } else {
          ra[u][c] = ld_piece<2>(base_a + k * a.lda * 2, m0 * 2 + col, a.M * 2, live && k < a.K);
        }
        if constexpr (kBRow) {
          const int64_t n = n0 + row;
          rb[u][c] = ld_piece<2>((const char*)a.b[c] + n * a.ldb * 2, k0 * 2 + col, a.K * 2, live && n < a.N);
        } else {
          rb[u][c] = ld_piece<2>(base_b + k * a.ldb * 2, n0 * 2 + col, a.N * 2, live && k < a.K);
        }
      }
    };
    auto place = [](int row, int piece, bool by_row) { return row * 128 + (piece ^ (by_row ? row & 7 : (row & 3) << 1)) * 16; };
    auto by_row = [&](const char* base, int r, int half) {
      return *(const i32x4*)(base + r * 128 + ((4 * half + g) ^ (r & 7)) * 16);
    };
    auto turned = [&](const char* base, int col, int half) {  // 8 rows of the summed axis x 16 columns
      const int row = 32 * half + 8 * g + (i16 >> 2);
      const char* q = base + row * 128 + ((col / 8 + (i16 >> 1 & 1)) ^ (row & 3) << 1) * 16 + (i16 & 1) * 8;
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)q);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(q + 4 * 128));
      return __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(u, u);
    for (int64_t s0 = 0; s0 < stages; s0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // (stages past the last are zeros)
        char* const lds_a = lds[u & 1][0];
        char* const lds_b = lds[u & 1][1];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p = tid + 256 * c;
          *(u32x4*)(lds_a + place(p / 8, p % 8, kARow)) = ra[u][c];
          *(u32x4*)(lds_b + place(p / 8, p % 8, kBRow)) = rb[u][c];
        }
        fetch(s0 + u + kAhead, u);
        // what is written here was read two stages ago, before the barrier in between
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          i32x4 fa[2], fb[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (kARow)
              fa[i] = by_row(lds_a, wm + i * 16 + i16, half);
            else
              fa[i] = turned(lds_a, wm + i * 16, half);
            if constexpr (kBRow)  // 16 columns of gate, then of up
              fb[i] = by_row(lds_b, i * 32 + wn / 2 + i16, half);
            else
              fb[i] = turned(lds_b, wn + i * 16, half);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<FMT>(fb[j], fa[i], acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + wm + i * 16 + i16;
      if constexpr (kForward) {
        float gate[4], up[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) gate[r] = acc[i][0][r], up[r] = acc[i][1][r];
        store_gated<FMT, 4, false>(a, m, n0 + wn / 2 + 4 * g, gate, up);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = n0 + wn + j * 16 + 4 * g;
          if (m >= a.M || n >= a.N) continue;
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r];
          if constexpr (kInput)
            store_run_as<FMT, 4, false>(a.out[0], nullptr, m * a.ldo[0] + n, a.N - n, v);
          else
            store_grad<FMT, 4>(a, out, m * a.ldo[out] + n, a.N - n, v);
        }
      }
    }
    __syncthreads();  // before the next tile's first pieces are written
  }
}

template <GluOp OP, int FMT>
hipError_t any_launch(const GluGemm& a, hipStream_t stream) {
  const int64_t tm = (a.M + kAnyTile - 1) / kAnyTile;
  const int64_t wide = OP == GluOp::kForward ? 32 : 64, tn = (a.N + wide - 1) / wide;
  const int64_t tiles = tm * tn, all = OP == GluOp::kWeight ? 2 * tiles : tiles;
  const dim3 grid((unsigned)(all < (1 << 20) ? all : (1 << 20)));
  glu_any<OP, FMT><<<grid, 256, 0, stream>>>(a, tn, tiles);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Rows on 4-byte boundaries (16-byte ones fastest): BM x BN sums per workgroup of WM x WN
// waves, pieces of both operands moved from memory into LDS directly, 64 of the summed
// axis a stage and NS stages in a ring.  A wave holds its fragments of the next
// 32 in registers while the matrix instructions take the current ones, so that
// LDS reads, memory loads and matrix instructions run side by side.  One barrier
// a stage: between its halves every wave has read all of the stage and its part
// of the next one has landed.  THROUGH: rows at any address, which the direct loads
// do not take, through registers (8192 x 11008 x 4096, rows one element off: 2054-2312 us).
//
// Bound, where there are many tiles, by the matrix instructions and the clock that they
// leave: 8192 x 11008 x 4096 in bf16, 256 x 256 tiles, 1103-1249 us forward (1180-1340
// TFLOP/s), 1192-1300 with gate and up kept, 1099-1173 input gradient, 1132-1257 weight
// gradients, matrix pipes 65-74% busy at 1.48-1.67 GHz; 32 x 32 x 16 instructions on the same
// fragments, in one process with these, took 1221-1344 / 1169-1184 / 1169 where these
// took 1155-1257 / 1110-1172 / 1122-1143.  With few tiles by what a compute unit takes
// in: 333 x 11008 x 4096 86 us in 192 x 128.
//
// An operand whose rows run along the summed axis lies in rows of 128 bytes,
// read 16 bytes a lane; one whose rows lie across it (both weights in kInput,
// everything in kWeight) lies as in memory and is turned by the transposing LDS
// reads.  Forward: b's tile holds, for each wave's 64 columns, 32 rows of gate and
// the same 32 of up, so that a lane ends with 8 columns of both.
// ---------------------------------------------------------------------------
template <GluOp OP, int FMT, int BM, int BN, int WM, int WN, int NS, bool PAST, bool THROUGH>
__global__ __launch_bounds__(WM* WN * 64, NS*(BM + BN) * 128 > 81920 && WM * WN == 4 ? 1 : 2) void glu_tile(const GluGemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr bool kForward = OP == GluOp::kForward, kInput = OP == GluOp::kInput, kWeight = OP == GluOp::kWeight;
  constexpr bool kARow = !kWeight, kBRow = kForward;
  constexpr int kWaves = WM * WN, kOutN = kForward ? BN / 2 : BN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  // across the summed axis: 8 rows, and 128 bytes that put the next 8 in the other half of the banks
  constexpr int kAGroup = 8 * BM * 2 + 128, kBGroup = 8 * BN * 2 + 128;
  constexpr int kABytes = kARow ? BM * 128 : 8 * kAGroup, kBBytes = kBRow ? BN * 128 : 8 * kBGroup;
  constexpr int kBuf = kABytes + kBBytes;
  constexpr int kALoads = BM / 8 / kWaves, kBLoads = BN / 8 / kWaves;
  // Forward: a wave's 64 columns are 32 of gate and 32 of up; a narrow tile's 32 are 16 and 16
  constexpr bool kNarrow = kForward && TN == 32;
  constexpr int kUpAt = TN / 16;  // b's loads of 8 rows: so many, half of gate and half of up
  static_assert(FN % 2 == 0 && kALoads > 0 && kBLoads > 0 && (NS & (NS - 1)) == 0 && (!kForward || TN == 64 || TN == 32) &&
                    (!kForward || kUpAt % kBLoads == 0),
                "tile shape");
  __shared__ __attribute__((aligned(1024))) char lds[NS * kBuf];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int wm = wave / WN * TM, wn = wave % WN * TN;
  const int out = kWeight ? (int)blockIdx.y : 0;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  tm = scalar(tm), tn = scalar(tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * kOutN;
  const int32_t K = (int32_t)a.K;
  const int nk = (int)(((int64_t)K + kStage - 1) / kStage), stages = kInput ? 2 * nk : nk;
  const int32_t pitch_a = (int32_t)a.lda * 2, pitch_b = (int32_t)a.ldb * 2;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS char*)lds;
  const char* const a0 = (const char*)a.a[kWeight ? out : 0];
  const char* const b0 = (const char*)a.b[0];
  // kInput: the second half of the stages are of the second pair of operands
  auto a_of = [&](int stage) { return kInput && stage >= nk ? (const char*)a.a[1] : a0; };
  auto b_of = [&](int stage) { return kInput && stage >= nk ? (const char*)a.b[1] : b0; };
  auto k_of = [&](int stage) { return (int64_t)(kInput && stage >= nk ? stage - nk : stage) * kStage; };
  // rows of the summed axis that a stage has (none past the last stage)
  auto rows_at = [&](int stage) {
    if (stage >= stages) return 0;
    const int64_t left = K - k_of(stage);
    return (int)(left < kStage ? left : kStage);
  };

  // Along the summed axis: piece c of row r lies at place c ^ s(r), s = the lane's row in a fragment & 7, so that the 8
  // lanes that read one bank width at a time read 8 different places.  b's fragment rows i16 are columns
  // (i16 / 4) * 8 + 4 (j % 2) + i16 % 4 of the 32 of two fragments, which leaves each lane 8 consecutive columns.
  const int32_t rows_a = left_of(a.M, m0, BM), cols_b = left_of(a.N, n0, kOutN);
  const uint32_t va_row = (uint32_t)(lane >> 3) * (uint32_t)pitch_a + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  uint32_t vb_row[2];
#pragma unroll
  for (int p = 0; p < 2; ++p)
    vb_row[p] = (uint32_t)(lane >> 3) * (uint32_t)pitch_b + (uint32_t)(((lane & 7) ^ (kNarrow ? lane >> 3 : (lane >> 3 & 3) | p << 2)) * 16);
  // A stage past the last lies past the end of every buffer: zeros, and no traffic.
  auto from = [&](int stage) { return stage < stages ? (uint32_t)(k_of(stage) * 2) : 0x7FFFFFF0u; };
  // Across it: piece c of row r at place c ^ s(r).  A transposing read takes 32 bytes of 4 consecutive rows, and of 4
  // that lie 8 rows on, per 32 lanes: s puts those 4 at different places.
  auto s_of = [](int row) { return (row & 3) << 1; };
  constexpr int kAPer = BM / 8, kBPer = BN / 8;            // pieces in a row
  constexpr int kARows = 64 / kAPer, kBRows = 64 / kBPer;  // rows a load (across the axis)
  static_assert((kARow || 64 % kAPer == 0) && (kBRow || 64 % kBPer == 0), "whole rows a load");
  constexpr int kAApart = kARows >= 4 ? 1 : 4 / kARows, kBApart = kBRows >= 4 ? 1 : 4 / kBRows;  // loads to the same s
  uint32_t va_col[kAApart], vb_col[kBApart];
#pragma unroll
  for (int j = 0; j < kAApart; ++j) {
    const int row = (wave * kALoads + j) * kARows + lane / kAPer;
    va_col[j] = (uint32_t)row * (uint32_t)pitch_a + (uint32_t)(((lane % kAPer) ^ s_of(row)) * 16);
  }
#pragma unroll
  for (int j = 0; j < kBApart; ++j) {
    const int row = (wave * kBLoads + j) * kBRows + lane / kBPer;
    vb_col[j] = (uint32_t)row * (uint32_t)pitch_b + (uint32_t)(((lane % kBPer) ^ s_of(row)) * 16);
  }

  // Forward: this wave's loads of b are all of gate or all of up.
  const int up = kForward ? wave * kBLoads / kUpAt % 2 : 0;
  const Rsrc ra_row = make_rsrc(a0 + m0 * a.lda * 2, rows_a, K * 2, pitch_a);
  const Rsrc ra_next = make_rsrc((const char*)a.a[kInput ? 1 : 0] + m0 * a.lda * 2, rows_a, K * 2, pitch_a);
  const Rsrc rb_row = make_rsrc((const char*)a.b[up] + n0 * a.ldb * 2, cols_b, K * 2, pitch_b);
  // THROUGH: rows at any address, in registers on their way: what a thread's loads would have put into LDS
  u32x4 ta[THROUGH ? kALoads : 1], tb[THROUGH ? kBLoads : 1];
  auto fetch_a = [&](int stage, int j) {
    const int t = wave * kALoads + j;
    const bool live = stage < stages;
    if constexpr (kARow) {
      const int64_t m = m0 + t * 8 + (lane >> 3);
      ta[j] = ld_piece<2>(a_of(stage) + m * a.lda * 2, k_of(stage) * 2 + ((lane & 7) ^ (lane >> 3)) * 16, a.K * 2, live && m < a.M);
    } else {
      const int row = t * kARows + lane / kAPer;
      const int64_t k = k_of(stage) + row;
      ta[j] = ld_piece<2>(a_of(stage) + k * a.lda * 2, m0 * 2 + ((lane % kAPer) ^ s_of(row)) * 16, a.M * 2, live && k < a.K);
    }
  };
  auto fetch_b = [&](int stage, int j) {
    const int t = wave * kBLoads + j;
    const bool live = stage < stages;
    if constexpr (kBRow) {
      const int64_t n = n0 + t / (2 * kUpAt) * (TN / 2) + t % kUpAt * 8 + (lane >> 3);
      tb[j] = ld_piece<2>((const char*)a.b[up] + n * a.ldb * 2,
                          k_of(stage) * 2 + ((lane & 7) ^ (kNarrow ? lane >> 3 : (lane >> 3 & 3) | (t & 1) << 2)) * 16, a.K * 2, live && n < a.N);
    } else {
      const int row = t * kBRows + lane / kBPer;
      const int64_t k = k_of(stage) + row;
      tb[j] = ld_piece<2>(b_of(stage) + k * a.ldb * 2, n0 * 2 + ((lane % kBPer) ^ s_of(row)) * 16, a.N * 2, live && k < a.K);
    }
  };
  auto put_a = [&](int stage, int j) {
    const int t = wave * kALoads + j;
    const int at = kARow ? t * 1024 : t * kARows / 8 * kAGroup + t * kARows % 8 * BM * 2;
    *(LDS u32x4*)((LDS char*)lds + (stage & (NS - 1)) * kBuf + at + lane * 16) = ta[j];
  };
  auto put_b = [&](int stage, int j) {
    const int t = wave * kBLoads + j;
    const int at = kBRow ? t * 1024 : t * kBRows / 8 * kBGroup + t * kBRows % 8 * BN * 2;
    *(LDS u32x4*)((LDS char*)lds + (stage & (NS - 1)) * kBuf + kABytes + at + lane * 16) = tb[j];
  };
  auto load_a = [&](int stage, int j) {
    const int t = wave * kALoads + j;
    const uint32_t to = lds0 + (stage & (NS - 1)) * kBuf;
    if constexpr (THROUGH) {  // what was fetched for the stage, and its place is fetched again for the one after it
      put_a(stage, j);
      fetch_a(stage + 1, j);
    } else if constexpr (kARow) {
      const bool next = kInput && stage >= nk;
      const Rsrc r = {next ? ra_next[0] : ra_row[0], next ? ra_next[1] : ra_row[1], ra_row[2], ra_row[3]};
      load_to_lds(r, va_row + (uint32_t)(t * 8) * (uint32_t)pitch_a + from(stage), to + t * 1024);
    } else {
      const Rsrc r = make_rsrc(a_of(stage) + (k_of(stage) * a.lda + m0) * 2, rows_at(stage), rows_a * 2, pitch_a);
      load_to_lds(r, va_col[j % kAApart] + (uint32_t)(j / kAApart * kAApart * kARows) * (uint32_t)pitch_a,
                  to + t * kARows / 8 * kAGroup + t * kARows % 8 * BM * 2);
    }
  };
  auto load_b = [&](int stage, int j) {
    const int t = wave * kBLoads + j;
    const uint32_t to = lds0 + (stage & (NS - 1)) * kBuf + kABytes;
    if constexpr (THROUGH) {
      put_b(stage, j);
      fetch_b(stage + 1, j);
    } else if constexpr (kBRow) {
      const int row = t / (2 * kUpAt) * (TN / 2) + t % kUpAt * 8;  // of gate or up
      load_to_lds(rb_row, vb_row[t & 1] + (uint32_t)row * (uint32_t)pitch_b + from(stage), to + t * 1024);
    } else {
      const Rsrc r = make_rsrc(b_of(stage) + (k_of(stage) * a.ldb + n0) * 2, rows_at(stage), cols_b * 2, pitch_b);
      load_to_lds(r, vb_col[j % kBApart] + (uint32_t)(j / kBApart * kBApart * kBRows) * (uint32_t)pitch_b,
                  to + t * kBRows / 8 * kBGroup + t * kBRows % 8 * BN * 2);
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  i32x4 fa[2][FM], fb[2][FN];

  const int s7 = i16 & 7;
  const int at_a_row = (wm + i16) * 128;
  const int at_b_row = kABytes + (wn + (kNarrow ? i16 : (i16 >> 2) * 8 + (i16 & 3))) * 128;
  // A lane's place in the rows of a transposing read of 16 columns from 16 c on.
  auto place_of = [&](int group, int pitch, int c) {
    return (uint32_t)(g * group + (i16 >> 2) * pitch + ((2 * (c & 3) + (i16 >> 1 & 1)) ^ (i16 >> 2) << 1) * 16 + (i16 & 1) * 8 +
                      (c >> 2) * 128);
  };
  constexpr int kAPlaces = FM < 4 ? FM : 4, kBPlaces = FN < 4 ? FN : 4;
  static_assert((FM <= 4 || TM % 64 == 0) && (FN <= 4 || TN % 64 == 0), "places repeat");
  uint32_t place_a[kAPlaces], place_b[kBPlaces];
#pragma unroll
  for (int v = 0; v < kAPlaces; ++v) place_a[v] = place_of(kAGroup, BM * 2, (wm >> 4) + v);
#pragma unroll
  for (int v = 0; v < kBPlaces; ++v) place_b[v] = kABytes + place_of(kBGroup, BN * 2, (wn >> 4) + v);
  auto turned = [&](uint32_t at, int pitch4) {  // 8 rows (4 and 4)
    LDS char* p = (LDS char*)lds + at;
    const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)p);
    const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(p + pitch4));
    return __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
  };
  auto read_a = [&](int buf, int half, int i) {
    if constexpr (kARow)
      fa[half][i] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_a_row + i * 16 * 128 + ((4 * half + g) ^ s7) * 16);
    else
      fa[half][i] = turned(place_a[i % kAPlaces] + (uint32_t)(buf * kBuf + half * 4 * kAGroup + i / 4 * 128), 4 * BM * 2);
  };
  auto read_b = [&](int buf, int half, int j) {
    if constexpr (kBRow)
      fb[half][j] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_b_row +
                                        (kNarrow ? j * 16 : j / 2 * 32 + j % 2 * 4) * 128 + ((4 * half + g) ^ s7) * 16);
    else
      fb[half][j] = turned(place_b[j % kBPlaces] + (uint32_t)(buf * kBuf + half * 4 * kBGroup + j / 4 * 128), 4 * BN * 2);
  };
  // The last stage's values past K are whatever the rows go on with: zero them (in both operands, for they may not be
  // finite).  Rows across the summed axis are read as zeros past its end.
  auto cut = [&](int stage, int half) {
    if constexpr (kARow) {
      if (K % kStage != 0 && (stage == stages - 1 || (kInput && stage == nk - 1))) {
        const i32x4 mask = inside(K - (nk - 1) * kStage - half * 32 - 8 * g);
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[half][i] &= mask;
        if constexpr (kBRow) {
#pragma unroll
          for (int j = 0; j < FN; ++j) fb[half][j] &= mask;
        }
      }
    }
  };
  // The matrix instructions of one half of a stage, with the fragment reads of the next half and, in the second, the
  // memory loads of stage `stage` + NS (into the buffer of the present one) spread between them.
  constexpr int kLoads = kALoads + kBLoads, kMfma = FM * FN;
  auto half_step = [&](auto half_c, int stage) {
    constexpr int half = decltype(half_c)::value;
    const int buf_next = (stage + half) & (NS - 1);
    cut(stage, half);
    for_each<kMfma>([&](auto at_c) {
      constexpr int at = decltype(at_c)::value, i = at / FN, j = at % FN;
      // the next fragments of a as the present ones come to their last use, those of b in the first half
      if constexpr (j == 0) read_a(buf_next, half ^ 1, i);
      for_each<FN>([&](auto r) {
        if constexpr (r >= at * 2 * FN / kMfma && r < (at + 1) * 2 * FN / kMfma) read_b(buf_next, half ^ 1, r);
      });
      acc[i][j] = mfma16<FMT>(fb[half][j], fa[half][i], acc[i][j]);
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
  if (stages > 0) {
    if constexpr (THROUGH) {
#pragma unroll
      for (int j = 0; j < kALoads; ++j) fetch_a(0, j);
#pragma unroll
      for (int j = 0; j < kBLoads; ++j) fetch_b(0, j);
    }
#pragma unroll
    for (int p = 0; p < NS; ++p) {
#pragma unroll
      for (int j = 0; j < kALoads; ++j) load_a(p, j);
#pragma unroll
      for (int j = 0; j < kBLoads; ++j) load_b(p, j);
    }
    // (THROUGH: the compiler waits for what a put needs; all puts are done where the waves meet)
    meet < THROUGH ? 63 : (NS - 1) * kLoads > ();
#pragma unroll
    for (int j = 0; j < FN; ++j) read_b(0, 0, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) read_a(0, 0, i);
    for (int s = 0; s < stages; ++s) {
      half_step(First{}, s);
      meet < THROUGH ? 63 : (NS - 2) * kLoads > ();  // all but the stages after the next have landed
      half_step(Second{}, s);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS when the workgroup ends
  }

  // Results: lane i16 holds row i16 of a fragment, 8 consecutive columns from two accumulators (after a trade where b
  // was turned), so that a store covers 64 bytes of each of 16 rows.
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + i * 16 + i16;
    if constexpr (kNarrow) {
      float v[2][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[0][r] = acc[i][0][r], v[1][r] = acc[i][1][r];
      store_gated<FMT, 4, false>(a, m, n0 + wn / 2 + g * 4, v[0], v[1]);
    } else if constexpr (kForward) {
      float v[2][8];
#pragma unroll
      for (int r = 0; r < 8; ++r) v[0][r] = acc[i][r / 4][r % 4], v[1][r] = acc[i][2 + r / 4][r % 4];
      store_gated<FMT, 8, PAST>(a, m, n0 + wn / 2 + g * 8, v[0], v[1]);
    } else {
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
        if (m >= a.M || n >= a.N) continue;
        if constexpr (kInput)
          store_run_as<FMT, 8, PAST>(a.out[0], nullptr, m * a.ldo[0] + n, a.N - n, v);
        else
          store_grad<FMT, 8>(a, out, m * a.ldo[out] + n, a.N - n, v);
      }
    }
  }
}

template <GluOp OP, int FMT, int BM, int BN, int WM, int WN, int NS, bool THROUGH = false>
hipError_t tile_launch(const GluGemm& a, hipStream_t stream) {
  constexpr int kOutN = OP == GluOp::kForward ? BN / 2 : BN;
  const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + kOutN - 1) / kOutN);
  const dim3 grid(tm * tn, OP == GluOp::kWeight ? 2 : 1);
  if constexpr (BM >= 128 && OP != GluOp::kWeight && !THROUGH) {
    bool whole = true;  // 16-bit outputs in whole pieces of 64 bytes: written past the caches, which keep the operands
    for (int p = 0; p < 3; ++p) whole = whole && (a.out[p] == nullptr || ((uintptr_t)a.out[p] | (uintptr_t)(a.ldo[p] * 2)) % 64 == 0);
    if (whole) {
      glu_tile<OP, FMT, BM, BN, WM, WN, NS, true, THROUGH><<<grid, WM * WN * 64, 0, stream>>>(a, tm, tn);
      return hipGetLastError();
    }
  }
  glu_tile<OP, FMT, BM, BN, WM, WN, NS, false, THROUGH><<<grid, WM * WN * 64, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few tokens, forward: 16 rows, and 16 columns of gate and the same 16 of up,
// per workgroup, whose W waves take every W-th 32 of the summed axis.  Fragments
// go from memory straight into registers, eight steps ahead, and no wave waits
// for another until their sums meet in LDS, where they are added in the waves'
// order: a stage of the tiled kernels takes at least 0.2 us, whatever its size,
// for its barrier and two rounds of LDS reads.  With 32 or 64 rows a workgroup it
// lost to the tiles (61 x 4096 x 4096: 32 and 24 us, 18 in 64 x 32).  One token, N =
// 11008, K = 4096: 41 us, 40-44 in tiles of up to 128, the weights' 180 MB at 4.1-4.5 TB/s.
// ---------------------------------------------------------------------------
template <int FMT, int W>
__global__ __launch_bounds__(W * 64, 2) void glu_few(const GluGemm a, uint32_t tiles_n) {
  constexpr int kAhead = 8, kPitch = 20;
  __shared__ __attribute__((aligned(16))) float lds[W][2][16 * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 16, m0 = (int64_t)(blockIdx.x / tiles_n) * 16;
  const int32_t K = (int32_t)a.K, steps = (K + 31) / 32;
  const int32_t pitch_a = (int32_t)a.lda * 2, pitch_b = (int32_t)a.ldb * 2, cols = left_of(a.N, n0, 16);
  const Rsrc ra = make_rsrc((const char*)a.a[0] + m0 * a.lda * 2, left_of(a.M, m0, 16), K * 2, pitch_a);
  const Rsrc rg = make_rsrc((const char*)a.b[0] + n0 * a.ldb * 2, cols, K * 2, pitch_b);
  const Rsrc ru = make_rsrc((const char*)a.b[1] + n0 * a.ldb * 2, cols, K * 2, pitch_b);
  const uint32_t va = (uint32_t)(i16 * pitch_a + g * 16), vb = (uint32_t)(i16 * pitch_b + g * 16);
  f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  i32x4 fa[kAhead], fb[kAhead][2];
  // (a step past the last is not fetched: its offset could lie in the next row)
  auto fetch = [&](int step, int u) {
    const uint32_t off = step < steps ? (uint32_t)step * 64u : 0x7FFFFFF0u;
    fb[u][0] = __builtin_bit_cast(i32x4, ld_buffer16(rg, vb + off));
    fb[u][1] = __builtin_bit_cast(i32x4, ld_buffer16(ru, vb + off));
    fa[u] = __builtin_bit_cast(i32x4, ld_buffer16(ra, va + off));
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(wave + u * W, u);
  for (int step = wave; step < steps; step += kAhead * W) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = step + u * W;
      if (at * 32 + 32 > K) {  // the end of the axis, or past it: what the rows go on with may not be finite
        const i32x4 mask = inside(K - at * 32 - 8 * g);
        fa[u] &= mask;
        fb[u][0] &= mask;
        fb[u][1] &= mask;
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) acc[p] = mfma16<FMT>(fb[u][p], fa[u], acc[p]);
      fetch(at + kAhead * W, u);
    }
  }
  // sums: row i16, columns 4 g .. 4 g + 3
#pragma unroll
  for (int p = 0; p < 2; ++p) *(f32x4*)(&lds[wave][p][i16 * kPitch + 4 * g]) = acc[p];
  __syncthreads();
  if (tid >= 64) return;
  const int row = tid / 4, four = tid % 4 * 4;
  float v[2][4];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    f32x4 sum = *(const f32x4*)(&lds[0][p][row * kPitch + four]);
#pragma unroll
    for (int w = 1; w < W; ++w) sum = sum + *(const f32x4*)(&lds[w][p][row * kPitch + four]);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[p][r] = sum[r];
  }
  store_gated<FMT, 4, false>(a, m0 + row, n0 + four, v[0], v[1]);
}

template <int FMT>
hipError_t few_launch(const GluGemm& a, hipStream_t stream) {
  const uint32_t tn = (uint32_t)((a.N + 15) / 16), tm = (uint32_t)((a.M + 15) / 16);
  glu_few<FMT, 4><<<dim3(tm * tn), 256, 0, stream>>>(a, tn);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few tokens, input gradient: 16 x 64 sums per workgroup, whose eight waves take
// every eighth 32 of the summed axis (both pairs of operands one behind the
// other), loaded into a part of LDS of the wave's own, three steps ahead, where
// the weights' rows are turned.  The waves' sums are added in their order.
// ---------------------------------------------------------------------------
template <int FMT>
__global__ __launch_bounds__(512, 2) void glu_input_split(const GluGemm a, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr int kWaves = 8, kAhead = 3, kOps = 5;
  constexpr int kAtB = 1024, kBuf = kAtB + 32 * 128;  // 16 rows of 32 values; 32 rows of 64 columns
  constexpr int kPitch = 68;                          // floats from row to row of the sums
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * kAhead * kBuf];
  static_assert(sizeof(lds) >= kWaves * 16 * kPitch * 4, "sums");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  tm = scalar(tm), tn = scalar(tn);
  const int64_t m0 = (int64_t)tm * 16, n0 = (int64_t)tn * 64;
  const int32_t K = (int32_t)a.K, half = (K + 31) / 32, steps = 2 * half;
  const int32_t pitch_a = (int32_t)a.lda * 2, pitch_b = (int32_t)a.ldb * 2;
  const int32_t rows = left_of(a.M, m0, 16), cols = left_of(a.N, n0, 64);
  const uint32_t mine = (uint32_t)(uintptr_t)(LDS char*)lds + wave * kAhead * kBuf;
  // a: 4 pieces a row, piece c of row r at place c ^ (r / 2 % 4); b: 8 pieces a row, at place c ^ s(r)
  auto s_of = [](int r) { return (r & 3) << 1; };
  const uint32_t va = (uint32_t)((lane >> 2) * pitch_a + ((lane & 3) ^ (lane >> 3 & 3)) * 16);
  auto fetch = [&](int step, int buf) {
    const bool second = step >= half;
    const int32_t k0 = (second ? step - half : step) * 32;
    const int32_t left = step < steps ? (K - k0 < 32 ? K - k0 : 32) : 0;
    const Rsrc ra = make_rsrc((const char*)(second ? a.a[1] : a.a[0]) + m0 * a.lda * 2, rows, K * 2, pitch_a);
    const Rsrc rb = make_rsrc((const char*)(second ? a.b[1] : a.b[0]) + ((int64_t)k0 * a.ldb + n0) * 2, left, cols * 2, pitch_b);
    load_to_lds(ra, va + (step < steps ? (uint32_t)k0 * 2u : 0x7FFFFFF0u), mine + buf * kBuf);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = j * 8 + (lane >> 3);
      load_to_lds(rb, (uint32_t)(row * pitch_b + ((lane & 7) ^ s_of(row)) * 16), mine + buf * kBuf + kAtB + j * 1024);
    }
  };
  f32x4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < kAhead; ++p) fetch(wave + p * kWaves, p);
  int buf = 0;
  for (int step = wave; step < steps; step += kWaves) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * kOps) : "memory");
    LDS char* p = (LDS char*)lds + (wave * kAhead + buf) * kBuf;
    i32x4 fa = *(LDS i32x4*)(p + i16 * 64 + (g ^ (i16 >> 1 & 3)) * 16);
    i32x4 fb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 8 * g + (i16 >> 2);
      LDS char* q = p + kAtB + row * 128 + ((2 * j + (i16 >> 1 & 1)) ^ s_of(row)) * 16 + (i16 & 1) * 8;
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)q);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(q + 4 * 128));
      fb[j] = __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // all of the buffer is read
    fetch(step + kAhead * kWaves, buf);
    const int left = K - (step >= half ? step - half : step) * 32;
    if (left < 32) fa &= inside(left - 8 * g);  // rows of b past the end are zeros
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = mfma16<FMT>(fb[j], fa, acc[j]);
    buf = buf == kAhead - 1 ? 0 : buf + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS
  __syncthreads();
  float* sums = (float*)lds;
#pragma unroll
  for (int j = 0; j < 4; ++j) *(f32x4*)(sums + (wave * 16 + i16) * kPitch + j * 16 + g * 4) = acc[j];
  __syncthreads();
  if (tid >= 256) return;
  const int row = tid / 16, col = tid % 16 * 4;
  f32x4 v = *(const f32x4*)(sums + row * kPitch + col);
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = v + *(const f32x4*)(sums + (w * 16 + row) * kPitch + col);
  const int64_t m = m0 + row, n = n0 + col;
  const float out[4] = {v[0], v[1], v[2], v[3]};
  if (m < a.M && n < a.N) store_run_as<FMT, 4, false>(a.out[0], nullptr, m * a.ldo[0] + n, a.N - n, out);
}

template <int FMT>
hipError_t input_split_launch(const GluGemm& a, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((a.M + 15) / 16), tn = (uint32_t)((a.N + 63) / 64);
  glu_input_split<FMT><<<dim3(tm * tn), 512, 0, stream>>>(a, tm, tn);
  return hipGetLastError();
}

// Rows that the direct loads take: on 4-byte boundaries (a single row at any
// distance from the next), offsets within a tile below 2^31.
bool rows4(const void* p, int64_t rows, int64_t ld) {
  return (uintptr_t)p % 4 == 0 && (rows <= 1 || (ld % 2 == 0 && ld <= (1 << 21)));
}

template <GluOp OP, int FMT>
hipError_t gemm_launch(const GluGemm& given, hipStream_t stream) {
  GluGemm a = given;
  const bool weight = OP == GluOp::kWeight, forward = OP == GluOp::kForward;
  const int64_t rows_a = weight ? a.K : a.M, rows_b = forward ? a.N : a.K;
  bool direct = rows4(a.a[0], rows_a, a.lda) && rows4(a.b[0], rows_b, a.ldb);
  if (!forward) direct = direct && rows4(a.a[1], rows_a, a.lda);
  if (!weight) direct = direct && rows4(a.b[1], rows_b, a.ldb);
  if (!weight) direct = direct && a.K <= (1 << 21);  // (a single row may be longer)
  const GluTile tile = choose(OP, a.M, a.N, a.K, direct);
  if (tile == GluTile::kAny) return any_launch<OP, FMT>(a, stream);
  if (tile == GluTile::kThrough) return tile_launch<OP, FMT, 128, 128, 2, 2, 2, true>(a, stream);
  // a single row: any distance that holds what a tile reads of it
  const int64_t wide_a = weight ? 256 : a.K, wide_b = forward ? a.K : 256;
  if (rows_a <= 1) a.lda = (wide_a + 255) / 256 * 256;
  if (rows_b <= 1) a.ldb = (wide_b + 255) / 256 * 256;
  if constexpr (OP == GluOp::kForward) {
    switch (tile) {
      case GluTile::kFew: return few_launch<FMT>(a, stream);
      case GluTile::k64x32: return tile_launch<OP, FMT, 64, 32, 4, 1, 8>(a, stream);
      case GluTile::k64: return tile_launch<OP, FMT, 64, 64, 4, 1, 4>(a, stream);
      case GluTile::k128: return tile_launch<OP, FMT, 128, 128, 4, 2, 4>(a, stream);
      case GluTile::k192: return tile_launch<OP, FMT, 192, 128, 4, 2, 2>(a, stream);
      default: return tile_launch<OP, FMT, 256, 256, 2, 4, 2>(a, stream);
    }
  } else if constexpr (OP == GluOp::kInput) {
    switch (tile) {
      case GluTile::kSplit: return input_split_launch<FMT>(a, stream);
      case GluTile::k32: return tile_launch<OP, FMT, 32, 64, 2, 2, 4>(a, stream);
      case GluTile::k64x128: return tile_launch<OP, FMT, 64, 128, 2, 2, 4>(a, stream);
      case GluTile::k128: return tile_launch<OP, FMT, 128, 128, 4, 2, 4>(a, stream);
      case GluTile::k128Near: return tile_launch<OP, FMT, 128, 128, 2, 2, 2>(a, stream);
      default: return tile_launch<OP, FMT, 256, 256, 2, 4, 2>(a, stream);
    }
  } else {
    switch (tile) {
      case GluTile::k64: return tile_launch<OP, FMT, 64, 64, 4, 1, 2>(a, stream);
      case GluTile::k128: return tile_launch<OP, FMT, 128, 128, 4, 2, 4>(a, stream);
      case GluTile::k128Near: return tile_launch<OP, FMT, 128, 128, 2, 2, 2>(a, stream);
      default: return tile_launch<OP, FMT, 256, 256, 2, 4, 2>(a, stream);
    }
  }
}

template <GluOp OP>
hipError_t by_format(const GluGemm& a, hipStream_t stream) {
  return a.format == ZS_FORMAT_BF16 ? gemm_launch<OP, kBF16>(a, stream) : gemm_launch<OP, kFP16>(a, stream);
}

}  // namespace

hipError_t launch_glu_gemm(GluOp op, const GluGemm& a, hipStream_t stream) {
  switch (op) {
    case GluOp::kForward: return by_format<GluOp::kForward>(a, stream);
    case GluOp::kInput: return by_format<GluOp::kInput>(a, stream);
    default: return by_format<GluOp::kWeight>(a, stream);
  }
}

}  // namespace zs
