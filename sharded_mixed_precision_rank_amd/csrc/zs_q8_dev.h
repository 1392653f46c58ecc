// Device helpers shared by the 8-bit operators' kernels: loads and stores of
// any alignment, conversions between storage formats, code packing.
#pragma once

#include "zs_device.h"
#include "zs_q8.h"

namespace zs {
namespace dev {

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
typedef int16_t i16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFP32 = ZS_FORMAT_FP32;

// One vector access at an address that is only aligned to its elements (the
// hardware takes any alignment in global memory).
template <class V, class E>
__device__ __forceinline__ V ld_any(const E* p) {
  typedef V U __attribute__((aligned(__alignof__(E))));
  return *(const GLB U*)(const GLB E*)p;
}
template <class V, class E>
__device__ __forceinline__ void st_any(E* p, V v) {
  typedef V U __attribute__((aligned(__alignof__(E))));
  *(GLB U*)(GLB E*)p = v;
}
// The same past the caches' normal order: for outputs that would push operands out of them.
template <class V, class E>
__device__ __forceinline__ void st_past(E* p, V v) {
  typedef V U __attribute__((aligned(__alignof__(E))));
  __builtin_nontemporal_store(v, (GLB U*)(GLB E*)p);
}

// Element i of an array in storage format FMT, as fp32.
template <int FMT>
__device__ __forceinline__ float ld_elem(const void* p, int64_t i) {
  if constexpr (FMT == kFP32)
    return ((const GLB float*)p)[i];
  else if constexpr (FMT == kBF16)
    return bf_one(((const GLB uint16_t*)p)[i]);
  else
    return fp16_one(((const GLB uint16_t*)p)[i]);
}
// A product rounded to fp32 before it is rounded again: the compiler would
// otherwise fold a product and its conversion to fp16 into one instruction
// with one rounding, in some places and not in others.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}
// Two values in a 16-bit format, packed.
template <int FMT>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
  if constexpr (FMT == kFP16) return pack_half<FMT>(rounded(a), rounded(b));
  return pack_half<FMT>(a, b);
}
template <int FMT>
__device__ __forceinline__ void st_elem(void* p, int64_t i, float v) {
  if constexpr (FMT == kFP32)
    ((GLB float*)p)[i] = v;
  else if constexpr (FMT == kBF16)
    ((GLB uint16_t*)p)[i] = to_bf16(v);
  else
    ((GLB _Float16*)p)[i] = (_Float16)rounded(v);
}
// Four consecutive values stored at element i (any alignment of an element).
template <int FMT>
__device__ __forceinline__ void st_four(void* p, int64_t i, const float* v) {
  if constexpr (FMT == kFP32)
    st_any<f32x4>((float*)p + i, (f32x4){v[0], v[1], v[2], v[3]});
  else
    st_any<u32x2>((uint16_t*)p + i, (u32x2){pack_two<FMT>(v[0], v[1]), pack_two<FMT>(v[2], v[3])});
}

}  // namespace dev
}  // namespace zs
