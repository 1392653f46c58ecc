// The gated block's activations and their derivatives, in fp32.
#pragma once

#include "zs_device.h"

namespace zs {
namespace dev {

// Where an exponential is below 2^-115 (e^-80) it is taken times 2^64, and the result divided by it in the end: the
// hardware's power of two gives zeros below 2^-126, where bf16, with fp32's exponents, still has normal values of act and
// act'.
constexpr float kDown = 0x1p-64f;

// 1 / (1 + e^-z), through the hardware's power of two and reciprocal (an error
// of about one step each; the product with log2 e adds |z| 2^-24: below 2^-16
// relative where it is not zero: 16-bit results keep 8 or 11 bits).  Times 2^64 where z is
// under -80, where it is e^z, and `down` is what undoes that.
__device__ __forceinline__ float logistic(float z, float& down) {
  const bool far = z < -80.0f;
  const float e = __builtin_amdgcn_exp2f(far ? __builtin_fmaf(1.44269504f, z, 64.0f) : -1.44269504f * z);
  down = far ? kDown : 1.0f;
  return far ? e : __builtin_amdgcn_rcpf(1.0f + e);
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
      const float z = -0.72134752f * v * v;  // v^2 / 2 in powers of two
      const bool far = z < -115.0f;
      slope = p + v * 0.39894228f * __builtin_amdgcn_exp2f(far ? z + 64.0f : z) * (far ? kDown : 1.0f);
    }
    return v * p;
  } else {
    constexpr bool silu = ACT == ZS_ACT_SILU;
    const float v2 = fminf(v * v, 1e30f);  // where it is cut, s is 0 or 1 and s (1 - s) z' has to come to 0
    const float z = silu ? v : v * (kTanhA + kTanhB * v2);
    float down;
    const float s = logistic(z, down);  // (far out s, 2^64 times itself, is below 2^-51: 1 - s is 1 as it should be)
    if constexpr (SLOPE) {
      const float dz = silu ? 1.0f : kTanhA + 3.0f * kTanhB * v2;
      slope = (s + v * s * (1.0f - s) * dz) * down;
    }
    return v * s * down;
  }
}

}  // namespace dev
}  // namespace zs
