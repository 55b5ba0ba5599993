// qlora_act.cuh -- the activations of the MLP block and their derivatives, in binary32.
//
//   silu       z p, p = 1 / (1 + e^-z)                  derivative p (1 + z (1 - p))
//   gelu       z Phi(z), Phi(z) = (1 + erf(z/sqrt 2))/2 derivative Phi(z) + z phi(z)
//   gelu_tanh  z p(2u), u = sqrt(2/pi) (z + 0.044715 z^3), because (1 + tanh u)/2 = 1/(1 + e^-2u);
//              derivative p + z p (1 - p) 2 u'
// The quotient uses the fast divide: for a denominator past 2^126 it gives 0, which is the limit.
#pragma once
#include <cstdint>

namespace qlora {
namespace act {
enum Act : int { kNone = 0, kSilu = 1, kGelu = 2, kGeluTanh = 3, kNumActs = 4 };

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
// gelu_tanh's polynomials take z clamped to +-20 (a NaN stays one), where p is 0 or 1 already: z^2
// stays finite.
__device__ __forceinline__ float clamp20(float z) { return z > 20.0f ? 20.0f : (z < -20.0f ? -20.0f : z); }
// 2 sqrt(2/pi) (z + 0.044715 z^3) = 2u
__device__ __forceinline__ float tanh_arg2(float z) {
  return z * fmaf(0.0713548162726f, z * z, 1.59576912161f);
}

template <int ACT>
__device__ __forceinline__ float value(float z) {
  if constexpr (ACT == kSilu) return z * sigmoid(z);
  if constexpr (ACT == kGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678118f));
  if constexpr (ACT == kGeluTanh) return z * sigmoid(tanh_arg2(clamp20(z)));
  return z;
}

// act(z) and its derivative.
template <int ACT>
__device__ __forceinline__ void value_grad(float z, float& a, float& d) {
  if constexpr (ACT == kSilu) {
    const float p = sigmoid(z);
    a = z * p;
    d = p * fmaf(z, 1.0f - p, 1.0f);
  } else if constexpr (ACT == kGelu) {
    const float c = 0.5f * (1.0f + erff(z * 0.70710678118f));
    a = z * c;
    d = fmaf(z * 0.39894228040f, __expf(-0.5f * z * z), c);
  } else if constexpr (ACT == kGeluTanh) {
    const float c = clamp20(z), p = sigmoid(tanh_arg2(c));
    a = z * p;
    d = fmaf(c * p * (1.0f - p), fmaf(0.2140644488178f, c * c, 1.59576912161f), p);
  } else {
    a = z;
    d = 1.0f;
  }
}

// N binary32 values (as bit patterns) through activation `act`, the switch outside the loop.
template <int N>
__device__ __forceinline__ void apply(int act, uint32_t (&v)[N]) {
  if (act == kSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __float_as_uint(value<kSilu>(__uint_as_float(v[i])));
  } else if (act == kGelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __float_as_uint(value<kGelu>(__uint_as_float(v[i])));
  } else if (act == kGeluTanh) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __float_as_uint(value<kGeluTanh>(__uint_as_float(v[i])));
  }
}

// Add 8 bf16 values (one 16-byte vector) to 8 binary32 bit patterns.
__device__ __forceinline__ void add8(uint32_t* v, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __float_as_uint(__uint_as_float(v[2 * i]) + __uint_as_float(w[i] << 16));
    v[2 * i + 1] = __float_as_uint(__uint_as_float(v[2 * i + 1]) + __uint_as_float(w[i] & 0xFFFF0000u));
  }
}
}  // namespace act
}  // namespace qlora
