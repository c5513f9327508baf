// Activations, their slopes, and what the products with an epilogue pass to it.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {

// 1 / (1 + exp(-z)) through the hardware's 2^y and reciprocal, each within
// 1 ulp: about 2e-7 relative, and z's own rounding.  exp(-z) may overflow to
// infinity: the reciprocal is 0 then.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// GELU's tanh form, x/2 (1 + tanh(k/2 (x + c x^3))) = x / (1 + exp(-k (x + c x^3)))
constexpr float kTanhK = 1.5957691216f /* 2 sqrt(2 / pi) */, kTanhC = 0.044715f;

// act(u) of V values.  The kind is the same in all lanes, so a wave takes one
// branch for its V values.
template <int V>
__device__ __forceinline__ void activate(int act, float (&u)[V]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = u[e] < 0.0f ? 0.0f : u[e];
      break;
    case kActRelu2:
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = u[e] < 0.0f ? 0.0f : u[e] * u[e];
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = gelu_f32(u[e]);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = u[e] * logistic(kTanhK * u[e] * __builtin_fmaf(kTanhC * u[e], u[e], 1.0f));
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = u[e] * logistic(u[e]);
      break;
    default: break;
  }
}

// d[e] *= act'(u[e]).
template <int V>
__device__ __forceinline__ void times_slope(int act, const float (&u)[V], float (&d)[V]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = u[e] > 0.0f ? d[e] : 0.0f;
      break;
    case kActRelu2:
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = u[e] > 0.0f ? d[e] * (2.0f * u[e]) : 0.0f;
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float cdf, pdf;
        gelu_cdf_pdf(u[e], cdf, pdf);
        d[e] *= __builtin_fmaf(u[e], pdf, cdf);
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x2 = u[e] * u[e];
        const float s = logistic(kTanhK * u[e] * __builtin_fmaf(kTanhC, x2, 1.0f));
        d[e] *= __builtin_fmaf(u[e] * s * (1.0f - s), kTanhK * __builtin_fmaf(3.0f * kTanhC, x2, 1.0f), s);
      }
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float s = logistic(u[e]);
        d[e] *= __builtin_fmaf(u[e] * s, 1.0f - s, s);
      }
      break;
    default: break;
  }
}

}  // namespace sp24
