// The gated block's activations and their derivatives, in fp32.
#pragma once

#include "zs_device.h"

namespace zs {
namespace dev {

// 1 / (1 + e^-z), through the hardware's power of two and reciprocal (an error
// of about one step each; the product with log2 e adds |z| 2^-24, below 2^-17
// relative where e^-z is finite: 16-bit results keep 8 or 11 bits).  Below 2^-126
// (z under -87.3) it is 0: `tail` is for such z.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

constexpr float kTanhA = 1.5957691216f;                // 2 sqrt(2 / pi)
constexpr float kTanhB = 1.5957691216f * 0.044715f;

// act(v), and act'(v) in `slope` where that is asked for.
//   silu       v s(v), s the logistic function;  s + v s (1 - s)
//   gelu       v P(v), P = erfc(-v / sqrt 2) / 2;  P + v e^(-v^2/2) / sqrt(2 pi)
//   gelu_tanh  v s(z), z = 2 sqrt(2/pi) (v + 0.044715 v^3);  s + v s (1 - s) z'
//   relu       max(v, 0); 1 above 0, else 0
template <int ACT, bool SLOPE>
__device__ __forceinline__ float act_of(float v, float& slope) {
  if constexpr (ACT == ZS_ACT_RELU) {
    if constexpr (SLOPE) slope = v > 0.0f ? 1.0f : 0.0f;
    return v > 0.0f ? v : v == v ? 0.0f : v;
  } else if constexpr (ACT == ZS_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.70710678f * v);
    if constexpr (SLOPE) {
      const float e = __builtin_amdgcn_exp2f(-0.36067376f * v * v);  // e^(-v^2/4): its square may be below 2^-126
      slope = p + v * 0.39894228f * e * e;
    }
    return v * p;
  } else {
    constexpr bool silu = ACT == ZS_ACT_SILU;
    const float v2 = fminf(v * v, 1e30f);  // where it is cut, s is 0 or 1 and s (1 - s) z' has to come to 0
    const float z = silu ? v : v * (kTanhA + kTanhB * v2);
    const float s = logistic(z);
    if constexpr (SLOPE) {
      const float dz = silu ? 1.0f : kTanhA + 3.0f * kTanhB * v2;
      slope = s + v * s * (1.0f - s) * dz;
    }
    return v * s;
  }
}

// silu and gelu_tanh below kTail, where e^z comes near 2^-126, under which the hardware's power of two gives zeros; bf16, with
// fp32's exponents, has normal values of act and act' there still.  e^z is taken times 2^64 and brought down at the end
// (below 2^-190 it is zero).
template <int ACT>
constexpr float kTail = ACT == ZS_ACT_SILU ? -80.0f : -9.5f;
template <int ACT, bool SLOPE>
__device__ __forceinline__ float tail(float v, float& slope) {
  constexpr bool silu = ACT == ZS_ACT_SILU;
  constexpr float down = 0x1p-64f;
  const float v2 = fminf(v * v, 1e30f);
  const float z = silu ? v : v * (kTanhA + kTanhB * v2);
  const float s = __builtin_amdgcn_exp2f(__builtin_fmaf(1.44269504f, z, 64.0f));  // (1 + e^z and 1 - s are 1)
  if constexpr (SLOPE) {
    const float dz = silu ? 1.0f : kTanhA + 3.0f * kTanhB * v2;
    slope = (s + v * s * dz) * down;
  }
  return v * s * down;
}

// The same for N values.  The tails take one look at the least of them and a branch that a wave hardly ever takes (8192 x
// 11008 x 256, gate of size 1, forward: silu 130-144 us, gelu_tanh 136-138; with a choice for every value instead 137-150 and
// 146-147, without the tails 129-145 and 136-138).
template <int ACT, bool SLOPE, int N>
__device__ __forceinline__ void acts_of(const float* v, float* value, float* slope) {
#pragma unroll
  for (int k = 0; k < N; ++k) value[k] = act_of<ACT, SLOPE>(v[k], slope[k]);
  if constexpr (ACT == ZS_ACT_SILU || ACT == ZS_ACT_GELU_TANH) {
    float least = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k) least = fminf(least, v[k]);
    if (__builtin_expect(__any(least < kTail<ACT>), 0)) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (v[k] < kTail<ACT>) value[k] = tail<ACT, SLOPE>(v[k], slope[k]);
    }
  }
}

}  // namespace dev
}  // namespace zs
