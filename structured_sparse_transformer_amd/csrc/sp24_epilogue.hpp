// Activations, their slopes, and what the products with an epilogue pass to it.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>

#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {

// 1 / (1 + 2^z) with the hardware's 2^z and reciprocal, within 1 ulp each; z's
// rounding adds |z| 2^-23.  2^z may overflow to infinity: the reciprocal is 0
// then.
__device__ __forceinline__ float logistic2(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z));
}

constexpr float kLog2 = 1.44269504f, kLog2InvSqrt2Pi = -1.32574806f;   // log2 e, log2(1 / sqrt(2 pi))
// x/2 (1 + tanh(sqrt(2 / pi) (x + c x^3))) = x / (1 + exp(-k (x + c x^3))), k = 2 sqrt(2 / pi)
constexpr float kTanhC = 0.044715f, kTanhK = 1.5957691216f;

// GELU: Phi(-a) = 2^P(a) for a = |x|, with the P of degree 6 that
// gen_gelu_fit.py prints: within 1.4e-6 relative, or a Phi(-a) within 4e-9, and
// |P| 2^-23 by rounding (1e-6 at a = 4), thousandths of fp16's half step.  One
// exponential and no division: about 16 issue slots for x Phi(x), counting 4 for
// the exponential, where sp24_device.hpp's form, which keeps 7e-7 relative as
// far as fp32 goes, takes 36 (forward product of 16384 x 6400 x 1600: 312 us
// with that, 290 with this).  P falls up to a = 13; past 10 it is held there,
// with x Phi(x) below 1e-22.
constexpr float kTail[7] = {-9.9999785e-01f, -1.1511753e+00f, -4.587958e-01f, -5.3436358e-02f,
                            8.12274e-03f,    -7.875215e-04f,  3.5610567e-05f};
__device__ __forceinline__ float normal_tail(float a) {
  float p = kTail[6];
#pragma unroll
  for (int k = 5; k >= 0; --k) p = __builtin_fmaf(p, a, kTail[k]);
  return __builtin_amdgcn_exp2f(p);
}
// min(|x|, 10), NaN for NaN
__device__ __forceinline__ float tail_argument(float x) {
  const float a = __builtin_fabsf(x);
  return a > 10.0f ? 10.0f : a;
}

__device__ __forceinline__ float tanh_form(float x, float x2) {
  return logistic2(x * __builtin_fmaf(x2, -kLog2 * kTanhK * kTanhC, -kLog2 * kTanhK));
}

// act(u)
template <int kAct>
__device__ __forceinline__ float activate(float u) {
  if constexpr (kAct == kActRelu) return u < 0.0f ? 0.0f : u;
  if constexpr (kAct == kActRelu2) return u < 0.0f ? 0.0f : u * u;
  if constexpr (kAct == kActGelu) {
    // x Phi(x) = max(x, 0) - a Phi(-a), NaN by the first part
    const float a = __builtin_amdgcn_fmed3f(__builtin_fabsf(u), 0.0f, 10.0f);
    return __builtin_fmaf(-a, normal_tail(a), u < 0.0f ? 0.0f : u);
  }
  if constexpr (kAct == kActGeluTanh) return u * tanh_form(u, u * u);
  if constexpr (kAct == kActSilu) return u * logistic2(u * -kLog2);
  return u;
}

// d act'(u).  RELU passes d where u is NaN: the forward's output is NaN there.
template <int kAct>
__device__ __forceinline__ float times_slope(float d, float u) {
  if constexpr (kAct == kActRelu) return u <= 0.0f ? 0.0f : d;
  if constexpr (kAct == kActRelu2) return u <= 0.0f ? 0.0f : d * (2.0f * u);
  if constexpr (kAct == kActGelu) {
    // Phi(x) + x phi(x): Phi(-a) - a phi(a) on the left, 1 less that on the right
    const float a = tail_argument(u);
    const float pdf = __builtin_amdgcn_exp2f(__builtin_fmaf(a * a, -0.5f * kLog2, kLog2InvSqrt2Pi));
    const float left = __builtin_fmaf(-a, pdf, normal_tail(a));
    return d * (u < 0.0f ? left : 1.0f - left);
  }
  if constexpr (kAct == kActGeluTanh) {
    const float x2 = u * u, s = tanh_form(u, x2);
    return d * __builtin_fmaf(u * s * (1.0f - s), kTanhK * __builtin_fmaf(3.0f * kTanhC, x2, 1.0f), s);
  }
  if constexpr (kAct == kActSilu) {
    const float s = logistic2(u * -kLog2);
    return d * __builtin_fmaf(u * s, 1.0f - s, s);
  }
  return d;
}

// f(kind) with the activation as a constant.  It is the same in all lanes: a
// wave takes one branch.
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActRelu2: f(std::integral_constant<int, kActRelu2>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}

}  // namespace sp24
