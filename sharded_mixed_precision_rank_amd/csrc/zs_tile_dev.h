// Device helpers shared by the tiled matrix products: buffer descriptors, direct
// loads to LDS, the mapping of workgroups to tiles, loops unrolled by constants,
// trades of accumulators between lane groups.
#pragma once

#include <utility>

#include "zs_q8_dev.h"

namespace zs {
namespace dev {

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

// A value that is the same in every lane, in a scalar register from here on: what descriptors are made of inside a loop
// must not be read back from vector registers there (see load_to_lds).
__device__ __forceinline__ uint32_t scalar(uint32_t v) {
  uint32_t s = __builtin_amdgcn_readfirstlane(v);
  asm volatile("" : "+s"(s));
  return s;
}

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

}  // namespace dev
}  // namespace zs
