// Orthogonalising a matrix by Newton-Schulz products, and the step that uses it.
//
//   X0 = U / |U|_F;  X <- a X + (b S + c S^2) X,  S = X X^T,  once a step
//
// X has no more rows than columns (a taller U goes by its transpose), so S is
// the smaller of the two squares.  The polynomial lifts small singular values by
// a = 3.4 each step, and a rounding of X with them: with X, S and b S + c S^2
// kept in one fp16 (11 bits) results were 0.1-1% off, in bf16 1-9%.  They are
// kept as two fp16 parts, hi + lo (22 bits), which leaves 1e-6 (128 x 128) to 4.5e-6
// (11008 x 4096), where fp32 products are 1.4e-6 to 8e-6 off.  A product is then three of the parts, hi hi + hi lo +
// lo hi (lo lo is below the last bit), at the fp16 rate with fp32 sums.
//
// Values are held times 2^12: the largest entry of X, S and b S + c S^2 is about
// 3 and may reach 15, a typical one of X0 is 1 / sqrt(rows columns), whose lo part
// stays above fp16's smallest numbers that way.
//
// Matrices lie in rows of groups of 128 bytes: 32 hi parts, then the 32 lo parts.
// Rows and columns are padded with zeros to multiples of 32, which the products
// keep at zero.
#include "zs_muon_dev.h"

namespace zs {
namespace {

using namespace dev;
using namespace ns;

// ---------------------------------------------------------------------------
// The update's first pass: the replicas' mean (fixed order, one rounding an
// operation), the momentum, and u, whose squares are summed in 64 bits, a
// workgroup's part in its own place.  Bound by memory: 2 N + 12 bytes a value (8
// replicas of 11008 x 4096: 230 us, 5.5 TB/s).
// ---------------------------------------------------------------------------
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  const double t = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  __syncthreads();
  return t;
}

__global__ __launch_bounds__(256) void ns_mean(const MeanArgs a) {
  __shared__ double lds[4];
  const int64_t base = (int64_t)blockIdx.y * a.n, pieces = (a.n + 7) / 8;
  double sum = 0.0;
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += (int64_t)gridDim.x * 256) {
    const int64_t i = base + p * 8;
    if (p * 8 + 8 <= a.n) {
      float s[8];
      widen_first<kBF16>(s, ld_any<u32x4>(a.g[0] + i));
      for (int r = 1; r < a.n_rep; ++r) accumulate<kBF16>(s, ld_any<u32x4>(a.g[r] + i));
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        const f32x4 m = ld_any<f32x4>(a.momentum + i + q);
        f32x4 m1, u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float t;
          u[k] = mean_step(s[q + k], m[k], a, t);
          m1[k] = t;
          sum += (double)u[k] * (double)u[k];
        }
        st_any(a.momentum + i + q, m1);
        st_any(a.u + i + q, u);
      }
    } else {
      for (int64_t k = i; k < base + a.n; ++k) {
        float s = bf_one(a.g[0][k]);
        for (int r = 1; r < a.n_rep; ++r) s = s + bf_one(a.g[r][k]);
        float m1;
        const float u = mean_step(s, a.momentum[k], a, m1);
        a.momentum[k] = m1;
        a.u[k] = u;
        sum += (double)u * (double)u;
      }
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) a.partials[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// The squares of given matrices, summed the same way.
struct NormArgs {
  const void* x;
  int64_t ld, batch_ld, rows, cols;
  double* partials;
};
template <int FMT>
__global__ __launch_bounds__(256) void ns_norm(const NormArgs a) {
  __shared__ double lds[4];
  const uint32_t per = (uint32_t)((a.cols + 7) / 8);
  const uint64_t pieces = (uint64_t)a.rows * per;
  double sum = 0.0;
  for (uint64_t p = (uint64_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += (uint64_t)gridDim.x * 256) {
    const int64_t row = pieces >> 32 ? (int64_t)(p / per) : (int64_t)((uint32_t)p / per), col = (int64_t)(p - (uint64_t)row * per) * 8;
    float v[8];
    load8<FMT>(a.x, (int64_t)blockIdx.y * a.batch_ld + row * a.ld + col, a.cols - col, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += (double)v[k] * (double)v[k];
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) a.partials[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// ---------------------------------------------------------------------------
// X0: values over their matrix's norm, as parts, turned where the matrix has
// more rows than columns.  64 x 64 values a workgroup, through LDS.  Each
// workgroup adds up the matrix's partial sums itself, in one order.  A matrix
// of zeros stays one.
// ---------------------------------------------------------------------------
struct PackArgs {
  const void* x;
  int64_t ld, batch_ld, rows, cols;
  const double* partials;
  int32_t n_partials;
  int32_t turned;
  char* to;
  int64_t pitch, batch_bytes;    // of X0
  uint32_t tiles_n;              // 64-column tiles of X0
  int64_t rows_to, cols_to;      // padded
  uint32_t* counters;            // zeroed here
  int32_t n_counters;            // of a matrix
};

template <int FMT>
__global__ __launch_bounds__(256) void ns_pack(const PackArgs a) {
  __shared__ double sums[4];
  __shared__ float tile[64 * 65];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    for (int i = tid; i < a.n_counters; i += 256) a.counters[(int64_t)blockIdx.y * a.n_counters + i] = 0;
  }
  double sum = 0.0;
  for (int i = tid; i < a.n_partials; i += 256) sum += a.partials[(int64_t)blockIdx.y * a.n_partials + i];
  sum = block_sum(sum, sums);
  const double per = sum == 0.0 ? 0.0 : (double)kUnit / __builtin_sqrt(sum);
  const int64_t r0 = (int64_t)(blockIdx.x / a.tiles_n) * 64, c0 = (int64_t)(blockIdx.x % a.tiles_n) * 64;  // in X0
  const int64_t sr0 = a.turned ? c0 : r0, sc0 = a.turned ? r0 : c0;                                        // in x
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int p = tid + 256 * c, row = p / 8, col = p % 8 * 8;
    float v[8];
    const int64_t sr = sr0 + row, sc = sc0 + col;
    if (sr < a.rows && sc < a.cols) {
      load8<FMT>(a.x, (int64_t)blockIdx.y * a.batch_ld + sr * a.ld + sc, a.cols - sc, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // (padding stays zero whatever the norm is)
      const float t = sr < a.rows && sc + k < a.cols ? (float)((double)v[k] * per) : 0.0f;
      tile[a.turned ? (col + k) * 65 + row : row * 65 + col + k] = t;
    }
  }
  __syncthreads();
  char* to = a.to + (int64_t)blockIdx.y * a.batch_bytes;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int p = tid + 256 * c, row = p / 8, col = p % 8 * 8;
    if (r0 + row >= a.rows_to || c0 + col >= a.cols_to) continue;
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = tile[row * 65 + col + k];
    store_parts(to + (r0 + row) * a.pitch, c0 + col, t);
  }
}

// ---------------------------------------------------------------------------
// The products, on parts: BM x BN sums per workgroup of WM x WN waves.
//
//   kGram   S = X X^T                symmetric: tiles on and below the diagonal, the others by turning them
//   kPoly   B = b S + c S S^T        the same
//   kApply  X' = a X + B X           the right operand's rows lie across the sum: transposing LDS reads
//
// A stage is 32 of the summed axis: rows of 128 bytes, hi and lo parts, moved
// into LDS directly, NS stages in a ring.  A wave's matrix instructions of a
// stage go lo hi, hi hi, hi lo; while one group runs, the fragments that are
// free are read for the next: hi of a and lo of b in the first group, lo of a of
// the next stage in the second, hi of b in the third.  So two sets of fragments
// serve three products, and 8 + 4 reads stand beside 96 instructions.
//
// Few tiles: the summed axis is split over `splits` workgroups.  Each leaves its
// sums in the workspace; the last to arrive (a counter a tile) adds them in
// their order, so the result does not depend on who that is.
//
// Large products are bound by the matrix instructions and the clock under them: 4096
// x 4096, S and the polynomial 175-178 us each in 192 x 192 tiles (matrix pipes busy 65% at
// 1.9 GHz), B X 290 in 256 x 256 (76% at 1.8 GHz; 1420 TFLOP/s of the parts' three
// products); S of 4096 x 11008 442-458, B X 821-828.  Small ones by a launch's start and end, 4 us, and
// what a compute unit takes in.
// ---------------------------------------------------------------------------
enum class NsOp : int32_t { kGram = 0, kPoly = 1, kApply = 2 };
struct NsGemm {
  const char* a;      // rows of the left operand
  const char* b;      // right operand: rows (kGram, kPoly), or rows of the summed axis (kApply)
  const char* add;    // kPoly: S; kApply: X
  char* d;            // parts out; NULL: the last step, values out
  int64_t pitch_a, pitch_b, pitch_d;  // bytes (add: pitch_d)
  int64_t batch_a, batch_b, batch_d;
  int64_t M, N, K;    // padded
  float by_add, by_sum;
  int32_t splits;
  float* sums;        // of split tiles
  uint32_t* counters;
  int32_t n_counters;
  NsLast last;
};

// Tile `id` of a triangle of tiles, row by row.
__device__ __forceinline__ void triangle(uint32_t id, uint32_t& i, uint32_t& j) {
  uint32_t r = (uint32_t)((__builtin_sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
  while (r * (r + 1) / 2 > id) --r;
  while ((r + 1) * (r + 2) / 2 <= id) ++r;
  i = r;
  j = id - r * (r + 1) / 2;
}

template <NsOp OP, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(WM* WN * 64, 2) void ns_tile(const NsGemm a, uint32_t tiles_m, uint32_t tiles_n, uint32_t tiles) {
  constexpr bool kTurned = OP == NsOp::kApply;  // b
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  // kApply: 8 rows of the summed axis, and 128 bytes that put the next 8 in the other half of the banks
  constexpr int kRowB = BN * 4, kGroup = 8 * kRowB + 128;
  constexpr int kABytes = BM * 128, kBBytes = kTurned ? 4 * kGroup : BN * 128, kBuf = kABytes + kBBytes;
  constexpr int kALoads = BM / 8 / kWaves, kBLoads = BN / 8 / kWaves;
  // values turned through LDS: up to 64 rows of a wave's part at a time
  constexpr int CM = TM < 64 ? TM : TM % 64 == 0 ? 64 : 32, kPitch = CM + 2, kTurn = TN * kPitch * 4;
  constexpr int kLds = NS * kBuf > kWaves * kTurn ? NS * kBuf : kWaves * kTurn;
  static_assert(FN % 2 == 0 && TN % 32 == 0 && TM % CM == 0 && CM % 16 == 0 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 &&
                    (NS & (NS - 1)) == 0,
                "tile shape");
  __shared__ __attribute__((aligned(1024))) char lds[kLds];
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int wm = wave / WN * TM, wn = wave % WN * TN;
  uint32_t tm, tn, id = 0;
  const uint32_t split = blockIdx.x / tiles;
  if constexpr (OP == NsOp::kApply) {
    tile_of(blockIdx.x % tiles, tiles_m, tiles_n, tm, tn);
    id = tm * tiles_n + tn;
  } else {
    // XCDs take runs of consecutive tiles
    const uint32_t bid = blockIdx.x % tiles, x = bid % 8, per = tiles / 8, more = tiles % 8;
    id = x * per + (x < more ? x : more) + bid / 8;
    triangle(id, tm, tn);
  }
  tm = scalar(tm), tn = scalar(tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int all = (int)(a.K / 32);
  const int first = (int)((int64_t)all * split / (uint32_t)a.splits), last = (int)((int64_t)all * (split + 1) / (uint32_t)a.splits);
  const int32_t pitch_a = (int32_t)a.pitch_a, pitch_b = (int32_t)a.pitch_b;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS char*)lds;
  const int32_t rows_a = left_of(a.M, m0, BM), cols_b = left_of(a.N, n0, BN);
  const char* const base_a = a.a + (int64_t)blockIdx.y * a.batch_a + m0 * a.pitch_a;
  const char* const base_b = a.b + (int64_t)blockIdx.y * a.batch_b + (kTurned ? n0 * 4 : n0 * a.pitch_b);
  const Rsrc ra = make_rsrc(base_a, rows_a, (int32_t)a.K * 4, pitch_a);
  const Rsrc rb = make_rsrc(base_b, cols_b, (int32_t)a.K * 4, pitch_b);  // (not kApply)

  // Rows of 8 pieces: piece c of row r at place c ^ s(r), s = the lane's row in a fragment & 7.  b's fragment rows i16
  // are columns (i16 / 4) * 8 + 4 (j % 2) + i16 % 4 of the 32 of two fragments.
  const uint32_t va = (uint32_t)(lane >> 3) * (uint32_t)pitch_a + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  uint32_t vb[kTurned ? kBLoads : 2];
  auto s_of = [](int row) { return (row & 3) << 1; };
  if constexpr (kTurned) {
#pragma unroll
    for (int j = 0; j < kBLoads; ++j) {
      const int at = (wave * kBLoads + j) * 1024 + lane * 16, row = at / kRowB, piece = at % kRowB / 16;
      vb[j] = (uint32_t)row * (uint32_t)pitch_b + (uint32_t)((piece ^ s_of(row)) * 16);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      vb[p] = (uint32_t)(lane >> 3) * (uint32_t)pitch_b + (uint32_t)(((lane & 7) ^ ((lane >> 3 & 3) | p << 2)) * 16);
  }
  // A stage past the last lies past the end of every buffer: zeros, and no traffic.
  auto from = [&](int stage) { return stage < last ? (uint32_t)stage * 128u : 0x7FFFFFF0u; };
  auto load_a = [&](int stage, int j) {
    const int t = wave * kALoads + j;
    load_to_lds(ra, va + (uint32_t)(t * 8) * (uint32_t)pitch_a + from(stage), lds0 + ((stage - first) & (NS - 1)) * kBuf + t * 1024);
  };
  auto load_b = [&](int stage, int j) {
    const int t = wave * kBLoads + j;
    const uint32_t to = lds0 + ((stage - first) & (NS - 1)) * kBuf + kABytes;
    if constexpr (kTurned) {
      const Rsrc r = make_rsrc(base_b + (int64_t)stage * 32 * a.pitch_b, stage < last ? 32 : 0, cols_b * 4, pitch_b);
      load_to_lds(r, vb[j], to + t * 1024 + t * 1024 / (8 * kRowB) * 128);
    } else {
      load_to_lds(rb, vb[t & 1] + (uint32_t)(t * 8) * (uint32_t)pitch_b + from(stage), to + t * 1024);
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  i32x4 fa[2][FM], fb[2][FN];  // hi, lo

  const int s7 = i16 & 7;
  const int at_a = (wm + i16) * 128;
  const int at_b = kABytes + (wn + (i16 >> 2) * 8 + (i16 & 3)) * 128;
  uint32_t place[4];
#pragma unroll
  for (int v = 0; v < 4; ++v)  // part v / 2, column fragment v % 2 of a group of 32
    place[v] = (uint32_t)(kABytes + g * kGroup + (i16 >> 2) * kRowB + ((2 * v + (i16 >> 1 & 1)) ^ (i16 >> 2) << 1) * 16 +
                          (i16 & 1) * 8 + (wn >> 5) * 128);
  auto read_a = [&](int buf, int part, int i) {
    fa[part][i] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_a + i * 16 * 128 + ((4 * part + g) ^ s7) * 16);
  };
  auto read_b = [&](int buf, int part, int j) {
    if constexpr (kTurned) {
      LDS char* p = (LDS char*)lds + (place[part * 2 + j % 2] + (uint32_t)(buf * kBuf + j / 2 * 128));
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)p);
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS i16x4*)(p + 4 * kRowB));
      fb[part][j] = __builtin_bit_cast(i32x4, (i16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    } else {
      fb[part][j] = *(const LDS i32x4*)((LDS char*)lds + buf * kBuf + at_b + (j / 2 * 32 + j % 2 * 4) * 128 +
                                        ((4 * part + g) ^ s7) * 16);
    }
  };
  constexpr int kLoads = kALoads + kBLoads, kMfma = FM * FN;
  // One group of a stage's matrix instructions: GROUP 0 lo hi, 1 hi hi, 2 hi lo.
  auto group = [&](auto group_c, int stage) {
    constexpr int G = decltype(group_c)::value, pa = G == 0 ? 1 : 0, pb = G == 2 ? 1 : 0;
    const int buf = (stage - first) & (NS - 1), next = (stage + 1 - first) & (NS - 1);
    for_each<kMfma>([&](auto at_c) {
      constexpr int at = decltype(at_c)::value, i = at / FN, j = at % FN;
      // reads, spread over the group
      constexpr int kReads = G == 0 ? FM + FN : G == 1 ? FM : FN;
      for_each<kReads>([&](auto r) {
        if constexpr (r >= at * kReads / kMfma && r < (at + 1) * kReads / kMfma) {
          if constexpr (G == 0) {
            if constexpr (r < FM)
              read_a(buf, 0, r);
            else
              read_b(buf, 1, r - FM);
          } else if constexpr (G == 1) {
            read_a(next, 1, r);
          } else {
            read_b(next, 0, r);
          }
        }
      });
      acc[i][j] = mfma_f16(fb[pb][j], fa[pa][i], acc[i][j]);
      if constexpr (G > 0) {
        for_each<kLoads>([&](auto l) {
          constexpr int w = at + (G - 1) * kMfma;
          if constexpr (l >= w * kLoads / (2 * kMfma) && l < (w + 1) * kLoads / (2 * kMfma)) {
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
#pragma unroll
  for (int p = 0; p < NS; ++p) {
#pragma unroll
    for (int j = 0; j < kALoads; ++j) load_a(first + p, j);
#pragma unroll
    for (int j = 0; j < kBLoads; ++j) load_b(first + p, j);
  }
  meet<(NS - 1) * kLoads>();
#pragma unroll
  for (int j = 0; j < FN; ++j) read_b(0, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) read_a(0, 1, i);
  for (int s = first; s < last; ++s) {
    group(First{}, s);
    meet<(NS - 2) * kLoads>();  // every wave has read all of the stage; all but the stages after the next have landed
    group(Second{}, s);
    group(std::integral_constant<int, 2>{}, s);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS
  __syncthreads();                                  // and its space is free

  if (a.splits > 1) {
    // The sums go past the XCD's own cache and are read the same way, by loads and stores of the whole device's scope: no
    // cache is written back or emptied for them (fences of that scope, which do both, took 35 us a kernel).
    const int64_t tile = (int64_t)blockIdx.y * tiles + id;
    uint64_t* const all_sums = (uint64_t*)(a.sums + tile * a.splits * (BM * BN));
    uint64_t* mine = all_sums + (int64_t)split * (BM * BN / 2);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          __hip_atomic_store((GLB uint64_t*)mine + ((wave * FM + i) * FN + j) * 128 + q * 64 + lane,
                             (uint64_t)__float_as_uint(acc[i][j][2 * q]) | (uint64_t)__float_as_uint(acc[i][j][2 * q + 1]) << 32,
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are there for every other
    __syncthreads();
    if (tid == 0) {
      uint32_t* counter = a.counters + (int64_t)blockIdx.y * a.n_counters + id;
      arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // the last leaves the counter as it was found
      if (arrived == (uint32_t)a.splits - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != (uint32_t)a.splits - 1) return;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
    for (int s = 0; s < a.splits; ++s) {
      const GLB uint64_t* from_split = (const GLB uint64_t*)all_sums + (int64_t)s * (BM * BN / 2);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint64_t w = __hip_atomic_load(from_split + ((wave * FM + i) * FN + j) * 128 + q * 64 + lane, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
            acc[i][j][2 * q] = acc[i][j][2 * q] + __uint_as_float((uint32_t)w);
            acc[i][j][2 * q + 1] = acc[i][j][2 * q + 1] + __uint_as_float((uint32_t)(w >> 32));
          }
    }
  }

  // Results, 8 consecutive columns a lane.  Symmetric ones go to their mirrored place too, and the last step of a taller
  // matrix only there: through LDS, a part of it for each wave.
  const bool final_step = a.d == nullptr;
  const bool direct = !final_step || !a.last.turned;
  const bool mirrored = kTurned ? final_step && a.last.turned : tm != tn;
  char* const d = a.d + (int64_t)blockIdx.y * a.batch_d;
  const char* const add = OP == NsOp::kGram ? nullptr : a.add + (int64_t)blockIdx.y * a.batch_d;
  LDS float* const turn = (LDS float*)((LDS char*)lds + wave * kTurn);
  for_each<TM / CM>([&](auto h_c) {
    constexpr int h = decltype(h_c)::value;
    for_each<CM / 16>([&](auto ii_c) {
      constexpr int ii = decltype(ii_c)::value, i = h * (CM / 16) + ii;
      const int64_t m = m0 + wm + i * 16 + i16;
#pragma unroll
      for (int c = 0; c < FN / 2; ++c) {
        float t[8];
        int col;
        if constexpr (kTurned) {
          col = c * 32 + eight_at(g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t lo, hi;
            trade(__float_as_uint(acc[i][2 * c][r]), __float_as_uint(acc[i][2 * c + 1][r]), lo, hi);
            t[r] = __uint_as_float(lo);
            t[4 + r] = __uint_as_float(hi);
          }
        } else {
          col = c * 32 + g * 8;
#pragma unroll
          for (int r = 0; r < 8; ++r) t[r] = acc[i][2 * c + r / 4][r % 4];
        }
        const int64_t n = n0 + wn + col;
        const bool live = m < a.M && n < a.N;
#pragma unroll
        for (int r = 0; r < 8; ++r) t[r] = t[r] * (a.by_sum * kPerUnit);
        if (OP != NsOp::kGram && live) {
          const GLB char* p = (const GLB char*)add + m * a.pitch_d + part_at(n);
          add_parts(*(const GLB u32x4*)p, *(const GLB u32x4*)(p + 64), a.by_add, t);
        }
        if (direct && live) {
          if (final_step)
            store_last(a.last, blockIdx.y, m, n, t);
          else
            store_parts(d + m * a.pitch_d, n, t);
        }
        if (mirrored) {
#pragma unroll
          for (int r = 0; r < 8; ++r) turn[(col + r) * kPitch + ii * 16 + i16] = t[r];
        }
      }
    });
    if (mirrored) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's values are there
      constexpr int kPer = CM / 8, kRows = 64 / kPer;
#pragma unroll
      for (int r0 = 0; r0 < TN; r0 += kRows) {
        const int r = r0 + lane / kPer, c = lane % kPer * 8;
        if (lane >= kPer * kRows || r >= TN) continue;
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = turn[r * kPitch + c + k];
        const int64_t row = n0 + wn + r, col = m0 + wm + h * CM + c;
        if (row >= a.N || col >= a.M) continue;
        if (final_step)
          store_last(a.last, blockIdx.y, row, col, t);
        else
          store_parts(d + row * a.pitch_d, col, t);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next are written
    }
  });
}

// ---------------------------------------------------------------------------
// The workspace, and the launches (the choice of tiles is in zs_muon_choice.h).
// ---------------------------------------------------------------------------
struct NsLayout {
  int64_t m, n;          // short and long side, padded
  Choice gram, poly, apply;
  int64_t n_partials, n_counters;  // of a matrix
  size_t at_partials, at_counters, at_x[2], at_s, at_b, at_sums, bytes;
};
size_t sums_bytes(const Choice& c, int64_t batch) {
  const size_t side = (size_t)kTileSide[(int)c.tile];
  return c.splits > 1 ? (size_t)c.tiles * (size_t)batch * (size_t)c.splits * side * side * 4 : 0;
}
NsLayout layout_of(int64_t rows, int64_t cols, int64_t batch) {
  NsLayout l{};
  l.m = padded(rows < cols ? rows : cols);
  l.n = padded(rows < cols ? cols : rows);
  const bool slab = l.m <= kSlabSide;  // no polynomial in memory, no product after it
  l.gram = choose(l.m, l.m, l.n, batch, true);
  l.poly = slab ? Choice{} : choose(l.m, l.m, l.m, batch, true);
  l.apply = slab ? Choice{} : choose(l.m, l.n, l.m, batch, false);
  const int64_t want = (rows * cols + 8 * 256 - 1) / (8 * 256);
  l.n_partials = want < kMostPartials ? want : kMostPartials;
  l.n_counters = 1;
  size_t sums = 0;
  for (const Choice& c : {l.gram, l.poly, l.apply}) {
    if (c.splits > 1 && c.tiles > l.n_counters) l.n_counters = c.tiles;
    if (sums_bytes(c, batch) > sums) sums = sums_bytes(c, batch);
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.at_partials = take((size_t)batch * (size_t)l.n_partials * 8);
  l.at_counters = take((size_t)batch * (size_t)l.n_counters * 4);
  for (int i = 0; i < 2; ++i) l.at_x[i] = take((size_t)batch * (size_t)l.m * (size_t)l.n * 4);
  l.at_s = take((size_t)batch * (size_t)l.m * (size_t)l.m * 4);
  l.at_b = take(slab ? 0 : (size_t)batch * (size_t)l.m * (size_t)l.m * 4);
  l.at_sums = take(sums);
  l.bytes = at;
  return l;
}

template <NsOp OP>
hipError_t gemm_launch(const NsGemm& given, const Choice& c, int64_t batch, hipStream_t stream) {
  NsGemm a = given;
  a.splits = c.splits;
  const int64_t side = kTileSide[(int)c.tile];
  const uint32_t tm = (uint32_t)((a.M + side - 1) / side), tn = (uint32_t)((a.N + side - 1) / side);
  const dim3 grid((unsigned)(c.tiles * c.splits), (unsigned)batch);
  const uint32_t tiles = (uint32_t)c.tiles;
  switch (c.tile) {
    case NsTile::k32: ns_tile<OP, 32, 32, 2, 1, 4><<<grid, 128, 0, stream>>>(a, tm, tn, tiles); break;
    case NsTile::k64: ns_tile<OP, 64, 64, 2, 2, 4><<<grid, 256, 0, stream>>>(a, tm, tn, tiles); break;
    case NsTile::k128: ns_tile<OP, 128, 128, 2, 2, 2><<<grid, 256, 0, stream>>>(a, tm, tn, tiles); break;
    case NsTile::k192: ns_tile<OP, 192, 192, 4, 2, 2><<<grid, 512, 0, stream>>>(a, tm, tn, tiles); break;
    default: ns_tile<OP, 256, 256, 2, 4, 2><<<grid, 512, 0, stream>>>(a, tm, tn, tiles);
  }
  return hipGetLastError();
}

}  // namespace

size_t ns_workspace_bytes(int64_t rows, int64_t cols, int64_t batch) {
  if (one_workgroup(rows, cols)) {
    // not touched: asked for as for the others, X twice, S and the polynomial, so that what a call accepts does not hang on
    // where a matrix is kept
    const int64_t side = rows < cols ? rows : cols;
    return (size_t)(batch * 8 * side * (rows + cols)) + 256;
  }
  return layout_of(rows, cols, batch).bytes + 256;  // and the way to a 256-byte boundary
}

hipError_t launch_ns(const NsProblem& p, void* workspace, hipStream_t stream) {
  if (one_workgroup(p.rows, p.cols)) return launch_ns_small(p, stream);
  const NsLayout l = layout_of(p.rows, p.cols, p.batch);
  char* const ws = (char*)(((uintptr_t)workspace + 255) / 256 * 256);
  const int64_t n = p.rows * p.cols;
  const int32_t parts = (int32_t)l.n_partials;
  double* const partials = (double*)(ws + l.at_partials);
  const dim3 first_grid((unsigned)parts, (unsigned)p.batch);
  PackArgs k{};
  k.rows = p.rows;
  k.cols = p.cols;
  if (p.update) {
    MeanArgs a = mean_of(p);
    a.u = (float*)(ws + l.at_x[1]);  // until the first product writes there
    a.partials = partials;
    ns_mean<<<first_grid, 256, 0, stream>>>(a);
    k.x = a.u;
    k.ld = p.cols;
    k.batch_ld = n;
  } else {
    const NormArgs a{p.x, p.ld_x, p.batch_x, p.rows, p.cols, partials};
    if (p.x_format == ZS_FORMAT_FP32)
      ns_norm<kFP32><<<first_grid, 256, 0, stream>>>(a);
    else if (p.x_format == ZS_FORMAT_BF16)
      ns_norm<kBF16><<<first_grid, 256, 0, stream>>>(a);
    else
      ns_norm<kFP16><<<first_grid, 256, 0, stream>>>(a);
    k.x = p.x;
    k.ld = p.ld_x;
    k.batch_ld = p.batch_x;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t pitch_x = l.n * 4, pitch_s = l.m * 4;
  k.partials = partials;
  k.n_partials = parts;
  k.turned = p.rows > p.cols;
  k.to = ws + l.at_x[0];
  k.pitch = pitch_x;
  k.batch_bytes = l.m * pitch_x;
  k.tiles_n = (uint32_t)((l.n + 63) / 64);
  k.rows_to = l.m;
  k.cols_to = l.n;
  k.counters = (uint32_t*)(ws + l.at_counters);
  k.n_counters = (int32_t)l.n_counters;
  const dim3 pack_grid((unsigned)((l.m + 63) / 64 * k.tiles_n), (unsigned)p.batch);
  if (p.update || p.x_format == ZS_FORMAT_FP32)
    ns_pack<kFP32><<<pack_grid, 256, 0, stream>>>(k);
  else if (p.x_format == ZS_FORMAT_BF16)
    ns_pack<kBF16><<<pack_grid, 256, 0, stream>>>(k);
  else
    ns_pack<kFP16><<<pack_grid, 256, 0, stream>>>(k);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  for (int s = 0; s < p.steps; ++s) {
    const char* const x = ws + l.at_x[s % 2];
    char* const s_at = ws + l.at_s;
    char* const b_at = ws + l.at_b;
    NsGemm a{};
    a.sums = (float*)(ws + l.at_sums);
    a.counters = (uint32_t*)(ws + l.at_counters);
    a.n_counters = (int32_t)l.n_counters;
    a.a = a.b = x;
    a.pitch_a = a.pitch_b = pitch_x;
    a.batch_a = a.batch_b = l.m * pitch_x;
    a.d = s_at;
    a.pitch_d = pitch_s;
    a.batch_d = l.m * pitch_s;
    a.M = a.N = l.m;
    a.K = l.n;
    a.by_sum = 1.0f;
    if ((e = gemm_launch<NsOp::kGram>(a, l.gram, p.batch, stream)) != hipSuccess) return e;
    if (l.m <= kSlabSide) {
      NsSlab b{s_at, x, s == p.steps - 1 ? nullptr : ws + l.at_x[(s + 1) % 2], pitch_x, l.m * pitch_s, l.m * pitch_x, (int32_t)l.m, l.n,
               p.coefs[3 * s], p.coefs[3 * s + 1], p.coefs[3 * s + 2], last_of(p)};
      if ((e = launch_ns_slab(b, p.batch, stream)) != hipSuccess) return e;
      continue;
    }
    a.a = a.b = a.add = s_at;
    a.pitch_a = a.pitch_b = pitch_s;
    a.batch_a = a.batch_b = l.m * pitch_s;
    a.d = b_at;
    a.K = l.m;
    a.by_add = p.coefs[3 * s + 1];
    a.by_sum = p.coefs[3 * s + 2];
    if ((e = gemm_launch<NsOp::kPoly>(a, l.poly, p.batch, stream)) != hipSuccess) return e;
    a.a = b_at;
    a.b = a.add = x;
    a.pitch_b = a.pitch_d = pitch_x;
    a.batch_b = a.batch_d = l.m * pitch_x;
    a.d = ws + l.at_x[(s + 1) % 2];
    a.N = l.n;
    a.by_add = p.coefs[3 * s];
    a.by_sum = 1.0f;
    if (s == p.steps - 1) {
      a.d = nullptr;
      a.last = last_of(p);
    }
    if ((e = gemm_launch<NsOp::kApply>(a, l.apply, p.batch, stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace zs
