// Row codes in 8 bits: zs_q8_save and zs_q8_load.
//
// Save, for each row t: a = max |x c|; s = max(f32(a / 127), 2^-126), or the
// least power of two that keeps a <= 127 s; q = rint(x c / s) of the exact
// quotient, ties to even.  A row with a NaN or an infinity gets s = NaN and
// codes 0.  Load: x^ = q s.
//
// Both are bound by memory: save reads each value once and writes a byte,
// load reads a byte and writes a value.  A row is taken by 8 to 64 lanes of a
// wave, or by a workgroup, that keep it in registers, as it was stored,
// between the maximum and the codes (rows of more than 16,384 columns are read
// twice).  16384 x 11008 bf16, other rows at each call: save 123-131 us (4.1-4.4
// TB/s), load 86-90 (6.0-6.3); a large copy moves 6.3.  The same rows again, part of
// them in the caches: save 103-110, with column factors 127-153.  The save waits for
// a whole row, then for its maximum, before it stores: that is what it has over
// the load.  Holding the unpacked values took 264 registers and 225-327 us.
#include "zs_q8_dev.h"

namespace zs {
namespace {

using namespace dev;

constexpr int kRowBlock = 256;

// Eight consecutive values as stored.
template <int FMT>
struct Raw8 {
  uint32_t w[FMT == kFP32 ? 8 : 4];
};

template <int FMT>
__device__ __forceinline__ void ld_raw(Raw8<FMT>& r, const void* row, int64_t col) {
  if constexpr (FMT == kFP32) {
    const u32x4 a = ld_any<u32x4>((const float*)row + col), b = ld_any<u32x4>((const float*)row + col + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[k] = a[k], r.w[4 + k] = b[k];
  } else {
    const u32x4 a = ld_any<u32x4>((const uint16_t*)row + col);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[k] = a[k];
  }
}
// Forgets what was made of the words: they are taken apart again where they
// are needed next, instead of held in twice the registers.
template <int FMT>
__device__ __forceinline__ void keep_raw(Raw8<FMT>& r) {
#pragma unroll
  for (uint32_t& w : r.w) asm volatile("" : "+v"(w));
}

template <int FMT>
__device__ __forceinline__ float raw_value(const Raw8<FMT>& r, int k) {
  if constexpr (FMT == kFP32)
    return __uint_as_float(r.w[k]);
  else
    return k % 2 ? h_hi<FMT>(r.w[k / 2]) : h_lo<FMT>(r.w[k / 2]);
}

// The eight values of a chunk, times their columns' factors (one fp32
// rounding each).
template <int FMT, bool COL>
__device__ __forceinline__ void values(const Raw8<FMT>& r, const float* col_scale, int64_t col, float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = raw_value<FMT>(r, k);
  if constexpr (COL) {
    const f32x4 a = ld_any<f32x4>(col_scale + col), b = ld_any<f32x4>(col_scale + col + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = v[k] * a[k], v[4 + k] = v[4 + k] * b[k];
  }
}

// |v| as bits: ordered as unsigned numbers, a NaN above an infinity above
// every finite value, so a plain integer maximum also finds those.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The largest magnitude met so far, as bits: two 16-bit ones side by side
// where the values are 16-bit and have no factors, else one of fp32.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <int FMT, bool COL>
__device__ __forceinline__ uint32_t larger(uint32_t top, const Raw8<FMT>& r, const float* col_scale, int64_t col) {
  if constexpr (FMT != kFP32 && !COL) {
    u16x2 t = __builtin_bit_cast(u16x2, top);
#pragma unroll
    for (int k = 0; k < 4; ++k) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, r.w[k] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, t);
  } else {
    float v[8];
    values<FMT, COL>(r, col_scale, col, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, mag(v[k]));
    return top;
  }
}
template <int FMT, bool COL>
__device__ __forceinline__ uint32_t largest(uint32_t top) {
  if constexpr (FMT != kFP32 && !COL) return mag(h_one<FMT>((uint16_t)max(top & 0xFFFFu, top >> 16)));
  return top;
}

struct Scale {
  float s, inv;  // the scale, and 1 / s
  bool bad;      // the row holds a NaN or an infinity
};

template <bool POW2>
__device__ __forceinline__ Scale scale_of(uint32_t top) {
  Scale r;
  r.bad = top >= 0x7F800000u;
  if constexpr (POW2) {
    // 127 = 1.984375 * 2^6: one power of two more when the mantissa is above that
    const int32_t e = (int32_t)(top >> 23) - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    const int32_t b = r.bad || e < 1 ? 1 : e;
    r.s = __uint_as_float((uint32_t)b << 23);
    r.inv = __uint_as_float((uint32_t)(254 - b) << 23);  // exact
  } else {
    r.s = fmaxf(__uint_as_float(r.bad ? 0u : top) / 127.0f, 0x1p-126f);
    r.inv = 1.0f / r.s;
  }
  if (r.bad) r.s = __uint_as_float(0x7FC00000u);
  return r;
}

// The codes of eight values, packed.  v * inv is within 127 * 2^-23 < 1.6e-5
// of the exact quotient, so adding 1.5 * 2^23 rounds it to the right integer
// (to even at ties) unless its distance from that integer is within 1.6e-5 of
// a half.  Those values, about one in 30,000, are decided by the
// remainder v - q s, which a fused multiply-add gives exactly.  With a power of
// two the product is exact and nothing needs deciding.
template <bool POW2>
__device__ __forceinline__ u32x2 codes8(const float* v, const Scale& sc) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  float m[8];
  float far = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = v[k] * sc.inv;
    m[k] = t + kMagic;
    if constexpr (!POW2) far = fmaxf(far, fabsf(t - (m[k] - kMagic)));
  }
  if constexpr (!POW2) {
    if (far > 0.49998f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float r = __builtin_fmaf(-(m[k] - kMagic), sc.s, v[k]);
        const float two = 2.0f * fabsf(r);
        const bool odd = (__float_as_uint(m[k]) & 1u) != 0;
        m[k] = m[k] + (two > sc.s || (two == sc.s && odd) ? __builtin_copysignf(1.0f, r) : 0.0f);
      }
    }
  }
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m[4 * h + 1]), __float_as_uint(m[4 * h]), 0x0C0C0400u);
    const uint32_t hi =
        __builtin_amdgcn_perm(__float_as_uint(m[4 * h + 3]), __float_as_uint(m[4 * h + 2]), 0x04000C0Cu);
    w[h] = sc.bad ? 0u : lo | hi;
  }
  return w;
}

// Rows of at least 8 columns.  lanes: lanes per row, a power of two from 8 to
// 64, or kRowBlock (one row per workgroup).  HELD: chunks of 8 values a lane
// keeps (lanes * HELD * 8 >= cols), or 0 to read the row twice.  The last chunk
// of a row ends with it and may take some of the one before again, and lanes
// past the last row take that again: the same codes to the same places.
template <int FMT, bool COL, bool POW2, int HELD>
__global__ __launch_bounds__(kRowBlock) void q8_save_kernel(const Q8Save a, int lanes) {
  __shared__ uint32_t wave_top[kRowBlock / 64];
  const int lane = threadIdx.x & (lanes - 1);
  const int sub = threadIdx.x / lanes, per = kRowBlock / lanes;
  const int64_t cols = a.cols;
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.rows; r0 += (int64_t)gridDim.x * per) {
    const int64_t row = r0 + sub < a.rows ? r0 + sub : a.rows - 1;
    constexpr int kBytes = FMT == kFP32 ? 4 : 2;
    const char* x = (const char*)a.x + row * a.ld_x * kBytes;
    int8_t* q = a.codes + row * a.ld_codes;
    uint32_t top = 0;
    Raw8<FMT> held[HELD > 0 ? HELD : 1];
    const auto at = [&](int64_t chunk) { return chunk * 8 + 8 <= cols ? chunk * 8 : cols - 8; };
    // with factors: the products, so that the factors are read once
    Raw8<kFP32> products[COL && HELD > 0 ? HELD : 1];
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if ((int64_t)(lane + i * lanes) * 8 < cols) ld_raw<FMT>(held[i], x, at(lane + i * lanes));
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if ((int64_t)(lane + i * lanes) * 8 < cols) {
          if constexpr (COL) {
            float v[8];
            values<FMT, true>(held[i], a.col_scale, at(lane + i * lanes), v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              products[i].w[k] = __float_as_uint(v[k]);
              top = max(top, mag(v[k]));
            }
          } else {
            top = larger<FMT, false>(top, held[i], nullptr, 0);
          }
        }
      }
    } else {
      for (int64_t c = lane; c * 8 < cols; c += lanes) {
        ld_raw<FMT>(held[0], x, at(c));
        top = larger<FMT, COL>(top, held[0], a.col_scale, at(c));
      }
    }
    top = largest<FMT, COL>(top);
    for (int off = (lanes < 64 ? lanes : 64) / 2; off >= 1; off >>= 1)
      top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if (lanes == kRowBlock) {
      if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = top;
      __syncthreads();
      top = max(max(wave_top[0], wave_top[1]), max(wave_top[2], wave_top[3]));
      __syncthreads();
    }
    const Scale sc = scale_of<POW2>(top);
    if (lane == 0) ((GLB float*)a.scales)[row] = sc.s;
    float v[8];
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if ((int64_t)(lane + i * lanes) * 8 < cols) {
          const int64_t col = at(lane + i * lanes);
          if constexpr (COL) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(products[i].w[k]);
          } else {
            keep_raw<FMT>(held[i]);
            values<FMT, false>(held[i], nullptr, col, v);
          }
          st_any<u32x2>(q + col, codes8<POW2>(v, sc));
        }
      }
    } else {
      for (int64_t c = lane; c * 8 < cols; c += lanes) {
        ld_raw<FMT>(held[0], x, at(c));
        values<FMT, COL>(held[0], a.col_scale, at(c), v);
        st_any<u32x2>(q + at(c), codes8<POW2>(v, sc));
      }
    }
  }
}

// Rows of fewer than 8 columns: a thread each.
template <int FMT, bool POW2>
__global__ __launch_bounds__(kRowBlock) void q8_save_narrow_kernel(const Q8Save a) {
  for (int64_t row = (int64_t)blockIdx.x * kRowBlock + threadIdx.x; row < a.rows; row += (int64_t)gridDim.x * kRowBlock) {
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = 0.0f;
      if (k < a.cols) {
        v[k] = ld_elem<FMT>(a.x, row * a.ld_x + k);
        if (a.col_scale != nullptr) v[k] = v[k] * ((const GLB float*)a.col_scale)[k];
      }
      top = max(top, mag(v[k]));
    }
    const Scale sc = scale_of<POW2>(top);
    ((GLB float*)a.scales)[row] = sc.s;
    const u32x2 w = codes8<POW2>(v, sc);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < a.cols) ((GLB int8_t*)a.codes)[row * a.ld_codes + k] = (int8_t)(w[k / 4] >> (8 * (k % 4)));
  }
}

// A lane takes 8 codes at a time; lanes (a power of two up to kRowBlock) share
// a row.
template <int FMT>
__global__ __launch_bounds__(kRowBlock) void q8_load_kernel(const Q8Load a, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int sub = threadIdx.x / lanes, per = kRowBlock / lanes;
  constexpr int kBytes = FMT == kFP32 ? 4 : 2;
  for (int64_t row = (int64_t)blockIdx.x * per + sub; row < a.rows; row += (int64_t)gridDim.x * per) {
    const float s = ((const GLB float*)a.scales)[row];
    const int8_t* q = a.codes + row * a.ld_codes;
    char* out = (char*)a.out + row * a.ld_out * kBytes;
    for (int64_t col = (int64_t)lane * 8; col < a.cols; col += (int64_t)lanes * 8) {
      if (col + 8 <= a.cols) {
        const u32x2 w = ld_any<u32x2>(q + col);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)(w[k / 4] >> (8 * (k % 4))) * s;
        if constexpr (FMT == kFP32) {
          st_four<FMT>(out, col, v);
          st_four<FMT>(out, col + 4, v + 4);
        } else {
          st_any<u32x4>((uint16_t*)out + col, (u32x4){pack_two<FMT>(v[0], v[1]), pack_two<FMT>(v[2], v[3]),
                                                      pack_two<FMT>(v[4], v[5]), pack_two<FMT>(v[6], v[7])});
        }
      } else {
        for (int64_t c = col; c < a.cols; ++c) st_elem<FMT>(out, c, (float)((const GLB int8_t*)q)[c] * s);
      }
    }
  }
}

dim3 row_grid(int64_t rows, int64_t per) {
  const int64_t groups = (rows + per - 1) / per;
  return dim3((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
}

template <int FMT, bool COL, bool POW2>
hipError_t save_launch(const Q8Save& a, hipStream_t stream) {
  const int64_t chunks = (a.cols + 7) / 8;
  int lanes = 8;
  while (lanes < 64 && chunks > lanes * 4) lanes *= 2;
  if (chunks > lanes * 4) lanes = kRowBlock;
  const dim3 grid = row_grid(a.rows, kRowBlock / lanes);
  if (chunks <= (int64_t)lanes * 2)
    q8_save_kernel<FMT, COL, POW2, 2><<<grid, kRowBlock, 0, stream>>>(a, lanes);
  else if (chunks <= (int64_t)lanes * 4)
    q8_save_kernel<FMT, COL, POW2, 4><<<grid, kRowBlock, 0, stream>>>(a, lanes);
  else if (chunks <= (int64_t)lanes * 8)
    q8_save_kernel<FMT, COL, POW2, 8><<<grid, kRowBlock, 0, stream>>>(a, lanes);
  else
    q8_save_kernel<FMT, COL, POW2, 0><<<grid, kRowBlock, 0, stream>>>(a, lanes);
  return hipGetLastError();
}
template <int FMT>
hipError_t save_launch(const Q8Save& a, hipStream_t stream) {
  const bool pow2 = a.rule == ZS_Q8_SCALE_POW2;
  if (a.cols < 8) {
    const dim3 grid = row_grid(a.rows, kRowBlock);
    if (pow2)
      q8_save_narrow_kernel<FMT, true><<<grid, kRowBlock, 0, stream>>>(a);
    else
      q8_save_narrow_kernel<FMT, false><<<grid, kRowBlock, 0, stream>>>(a);
    return hipGetLastError();
  }
  if (a.col_scale) return pow2 ? save_launch<FMT, true, true>(a, stream) : save_launch<FMT, true, false>(a, stream);
  return pow2 ? save_launch<FMT, false, true>(a, stream) : save_launch<FMT, false, false>(a, stream);
}

template <int FMT>
hipError_t load_launch(const Q8Load& a, hipStream_t stream) {
  const int64_t chunks = (a.cols + 7) / 8;
  int lanes = 4;
  while (lanes < kRowBlock && chunks > lanes) lanes *= 2;
  q8_load_kernel<FMT><<<row_grid(a.rows, kRowBlock / lanes), kRowBlock, 0, stream>>>(a, lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q8_save(const Q8Save& a, hipStream_t stream) {
  switch (a.format) {
    case ZS_FORMAT_BF16: return save_launch<kBF16>(a, stream);
    case ZS_FORMAT_FP16: return save_launch<kFP16>(a, stream);
    default: return save_launch<kFP32>(a, stream);
  }
}

hipError_t launch_q8_load(const Q8Load& a, hipStream_t stream) {
  switch (a.format) {
    case ZS_FORMAT_BF16: return load_launch<kBF16>(a, stream);
    case ZS_FORMAT_FP16: return load_launch<kFP16>(a, stream);
    default: return load_launch<kFP32>(a, stream);
  }
}

}  // namespace zs
