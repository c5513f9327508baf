// The norm of many gradients together, and AdamW over many tensors at once.
//
// Tensors go to a launch in a table of kernel arguments, as many as 4 KB hold;
// a workgroup finds its tensor from its number by the tensors' running counts
// of chunks.  Every entry is read and written once: both kernels are bound by
// memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "sp24.h"
#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// The tensor that chunk c of a launch belongs to: the last whose first chunk
// is at most c.  Tensors without chunks are not in the table.
template <int N>
__device__ __forceinline__ int tensor_of(const uint32_t (&first)[N], int count, uint32_t c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Four consecutive entries of a tensor as fp32, zeros past its end.
template <bool kF16>
__device__ __forceinline__ float4v load4(const void* p, int64_t i, int64_t n) {
  float4v v = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (kF16) {
    const _Float16* q = static_cast<const _Float16*>(p) + i;
    if (i + 4 <= n) {
      const half4 x = *reinterpret_cast<const half4*>(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)x[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < n) v[e] = (float)q[e];
    }
  } else {
    const float* q = static_cast<const float*>(p) + i;
    if (i + 4 <= n) return *reinterpret_cast<const float4v*>(q);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) v[e] = q[e];
  }
  return v;
}
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, float4v v) {
  if (i + 4 <= n) {
    *reinterpret_cast<float4v*>(p + i) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) p[i + e] = v[e];
}

// ---------------------------------------------------------------------------
// The norm.  Squares are summed in fp64: no finite gradients overflow, and the
// sum is not finite only where an entry is not.  20.5 M fp32 entries (82 MB) in 14.9
// us, 5.5 TB/s, and 2 to 4 us for the joining of the workgroups' sums.

constexpr int kNormTensors = 128;
constexpr int64_t kNormChunk = 16384;
struct NormTable {
  const void* g[kNormTensors];
  int64_t n[kNormTensors];
  uint32_t first[kNormTensors];
  int count;
};
static_assert(sizeof(NormTable) <= 3800, "kernel arguments");

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int x = 32; x >= 1; x /= 2) v += __shfl_xor(v, x);
  return v;
}

template <bool kF16>
__global__ __launch_bounds__(kThreads) void squares_kernel(NormTable tab, double* __restrict__ part) {
  __shared__ double waves[kThreads / 64];
  const int k = tensor_of(tab.first, tab.count, blockIdx.x);
  const int64_t n = tab.n[k], i0 = (int64_t)(blockIdx.x - tab.first[k]) * kNormChunk;
  double sum = 0.0;
  constexpr int kAhead = 8;   // loads under way at once
  for (int u0 = 0; u0 < kNormChunk / (4 * kThreads) && i0 + u0 * 4 * kThreads < n; u0 += kAhead) {
    float4v x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = load4<kF16>(tab.g[k], i0 + ((u0 + u) * kThreads + (int)threadIdx.x) * 4, n);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = __builtin_fma((double)x[u][e], (double)x[u][e], sum);
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = waves[0] + waves[1] + (waves[2] + waves[3]);
}

typedef sp24_step_control Control;

__global__ __launch_bounds__(1024) void norm_kernel(const double* __restrict__ part, int64_t parts, double scale,
                                                    double max_norm, Control* control) {
  __shared__ double waves[16];
  double sum = 0.0;
  for (int64_t p = threadIdx.x; p < parts; p += 1024) sum += part[p];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  sum = 0.0;
  for (int w = 0; w < 16; ++w) sum += waves[w];
  const double norm = __builtin_sqrt(sum) * scale;
  const bool fine = __builtin_isfinite(norm);
  control->norm = (float)norm;
  control->factor = fine ? (float)(norm > max_norm ? scale * (max_norm / norm) : scale) : 0.0f;
  control->skip = !fine;
  if (fine) control->step += 1;
}

// ---------------------------------------------------------------------------
// States in 8 bits.
//
// Groups of 64 consecutive entries share an exponent E (that of the fp32
// format, 0..254; 255: some entry of the group is not finite).  A magnitude
// has 4 exponent and F fraction bits: M's F = 3 and a sign, the root of V's
// F = 4.  With e and f its exponent and fraction fields it stands for
//   (e ? 1 + f / 2^F : f / 2^F) 2^(E - 127 - 15 + max(e, 1)),
// that is, for the fp32 number of bits code << (23 - F) times 2^(E - 15): the
// small magnitudes fall on fp32's own subnormals, and encoding is a scaling by
// a power of two and a rounding of the bits.
//
// V is held as its root, for half the range, and both are rounded up or down
// at random: with b2 = 0.999 a step moves a root by a 2000th, which rounding to
// nearest among steps of a 32nd would drop for ever.  A root above zero stays
// above zero, so that no entry's step is divided by eps alone.  64 entries a group
// are 16 lanes of four, a row of the lane moves: the maximum takes no LDS.

constexpr int kFracM = 3, kFracV = 4;

template <int F>
__device__ __forceinline__ float held_value(uint32_t magnitude, int E) {
  const float x = __builtin_amdgcn_ldexpf(__builtin_bit_cast(float, magnitude << (23 - F)), E - 15);
  return E == 255 ? __builtin_nanf("") : x;
}

// The exponent for a group whose largest magnitude has these bits: that of the
// magnitude rounded up to F fraction bits, so that no rounding leaves the format.
template <int F>
__device__ __forceinline__ int group_exponent(uint32_t top) {
  const uint32_t E = (top + ((1u << (23 - F)) - 1)) >> 23;
  return top >= 0x7F800000u ? 255 : (int)min(E, 254u);
}

__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

// x >= 0 (finite) rounded up where the bits that the code drops and 16 random
// ones carry.
template <int F>
__device__ __forceinline__ uint32_t held_code(float x, int E, uint32_t random16) {
  constexpr int kDrop = 23 - F;
  const uint32_t y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_ldexpf(x, 15 - E));
  const uint32_t code = (y + (random16 << (kDrop - 16)) + (1u << (kDrop - 17))) >> kDrop;
  return min(code, (1u << (4 + F)) - 1);
}

// 32 bits mixed by multiplications with the first bits of the roots of 2 and 3.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// The largest of a row of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  const auto moved = [](uint32_t v, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, true);
  };
  x = max(x, moved(x, std::integral_constant<int, 0xB1>()));    // quad_perm 1 0 3 2
  x = max(x, moved(x, std::integral_constant<int, 0x4E>()));    // quad_perm 2 3 0 1
  x = max(x, moved(x, std::integral_constant<int, 0x124>()));   // row_ror 4
  return max(x, moved(x, std::integral_constant<int, 0x128>()));   // row_ror 8
}

// Four codes, zeros past the end.
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t c = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) c |= (uint32_t)p[i + e] << (8 * e);
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, uint32_t c) {
  if (i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + i) = c;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) p[i + e] = (uint8_t)(c >> (8 * e));
}

// ---------------------------------------------------------------------------
// AdamW.  States in 32 bits: 28 bytes an entry, 30 with an fp16 copy (20.5 M entries,
// 615 MB: 107 us traced, 120 as timed from outside, against 125 for a copy's 4.9
// TB/s).  In 8 bits: 16 an entry with an exponent for each 64 of both states (80.4 M
// entries, 1.29 GB by the counters: 252-257 us, 5.1 TB/s).  48 biases of 4096 and 1024
// are a launch of 6.1 us.

constexpr int64_t kAdamChunk = 4096;
template <bool k8>
struct AdamEntry {
  const void* G;
  float* P;
  void* M;
  void* V;
  uint16_t* W;
  int64_t n;
  float lr, keep;
};
template <>
struct AdamEntry<true> : AdamEntry<false> {
  uint8_t* ME;
  uint8_t* VE;
  uint32_t place;
};
template <bool k8>
struct AdamTable {
  static constexpr int kTensors = k8 ? 44 : 64;
  AdamEntry<k8> t[kTensors];
  uint32_t first[kTensors];
  int count;
  float b1, c1, b2, c2, eps, ln_b1, ln_b2;
  int64_t step;
  const Control* control;
  uint32_t seed;
};
static_assert(sizeof(AdamTable<true>) <= 4000 && sizeof(AdamTable<false>) <= 4000, "kernel arguments");

template <bool kF16, bool k8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamTable<k8> tab) {
  int64_t step = tab.step;
  float factor = 1.0f;
  if (tab.control != nullptr) {
    step = tab.control->step;
    if (tab.control->skip != 0 || step < 1) return;
    factor = tab.control->factor;
  }
  const int k = tensor_of(tab.first, tab.count, blockIdx.x);
  const AdamEntry<k8>& t = tab.t[k];
  const int64_t n = t.n, i0 = (int64_t)(blockIdx.x - tab.first[k]) * kAdamChunk;
  // 1 - b^step through expm1: the difference keeps its precision for b near 1
  const float rate = t.lr / -expm1f((float)step * tab.ln_b1);
  const float root = 1.0f / sqrtf(-expm1f((float)step * tab.ln_b2));
  uint32_t key = 0;
  if constexpr (k8) key = mix(mix(mix((uint32_t)step) ^ tab.seed) ^ t.place);
  // groups of 4 entries, kAhead of them under way at once
  constexpr int kGroups = kAdamChunk / (4 * kThreads), kAhead = k8 ? 4 : 2;
  static_assert(kGroups % kAhead == 0, "whole batches");
  for (int u0 = 0; u0 < kGroups && i0 + u0 * 4 * kThreads < n; u0 += kAhead) {
    float4v g[kAhead], p[kAhead], m[kAhead], v[kAhead];
    uint32_t mc[kAhead], vc[kAhead];
    int me[kAhead], ve[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t i = i0 + ((u0 + u) * kThreads + (int)threadIdx.x) * 4;
      g[u] = load4<kF16>(t.G, i, n);
      p[u] = load4<false>(t.P, i, n);
      if constexpr (k8) {
        mc[u] = load_codes(static_cast<const uint8_t*>(t.M), i, n);
        vc[u] = load_codes(static_cast<const uint8_t*>(t.V), i, n);
        // lanes past the end have zeros for codes and exponents: another group's
        // exponent may be 255, NaN for every code, and is its own row's to write
        // (1.5% slower than a load by all lanes of one: 242.5 and 238.7 us a step)
        me[u] = i < n ? t.ME[i / 64] : 0;
        ve[u] = i < n ? t.VE[i / 64] : 0;
      } else {
        m[u] = load4<false>(t.M, i, n);
        v[u] = load4<false>(t.V, i, n);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t i = i0 + ((u0 + u) * kThreads + (int)threadIdx.x) * 4;
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (k8) {
          const uint32_t a = mc[u] >> (8 * e) & 255, b = vc[u] >> (8 * e) & 255;
          const float x = held_value<kFracM>(a & 127, me[u]), y = held_value<kFracV>(b, ve[u]);
          m[u][e] = a & 128 ? -x : x;
          v[u][e] = y * y;
        }
        const float x = g[u][e] * factor;
        m[u][e] = m[u][e] * tab.b1 + x * tab.c1;
        v[u][e] = v[u][e] * tab.b2 + x * x * tab.c2;
        r[e] = sqrtf(v[u][e]);
        p[u][e] = p[u][e] * t.keep - rate * m[u][e] / (r[e] * root + tab.eps);
      }
      store4(t.P, i, n, p[u]);
      if (t.W != nullptr) {
        if (i + 4 <= n) {
          *reinterpret_cast<half4*>(t.W + i) =
              half4{(_Float16)p[u][0], (_Float16)p[u][1], (_Float16)p[u][2], (_Float16)p[u][3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < n) t.W[i + e] = __builtin_bit_cast(uint16_t, (_Float16)p[u][e]);
        }
      }
      if constexpr (k8) {
        // 16 lanes hold a group.  Entries past the end are zeros: the loads
        // gave zeros, and a state of zeros stays one.
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          tm = max(tm, magnitude_bits(m[u][e]));
          tv = max(tv, magnitude_bits(r[e]));
        }
        const int em = group_exponent<kFracM>(row_max(tm)), ev = group_exponent<kFracV>(row_max(tv));
        uint32_t cm = 0, cv = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bits = mix((uint32_t)(i + e) ^ key);
          uint32_t a = held_code<kFracM>(__builtin_fabsf(m[u][e]), em, bits & 0xFFFFu);
          uint32_t b = held_code<kFracV>(r[e], ev, bits >> 16);
          if (m[u][e] < 0.0f) a |= 128;
          if (r[e] > 0.0f) b = max(b, 1u);
          cm |= a << (8 * e);
          cv |= b << (8 * e);
        }
        store_codes(static_cast<uint8_t*>(t.M), i, n, em == 255 ? 0 : cm);
        store_codes(static_cast<uint8_t*>(t.V), i, n, ev == 255 ? 0 : cv);
        if ((threadIdx.x & 15) == 0 && i < n) {
          t.ME[i / 64] = (uint8_t)em;
          t.VE[i / 64] = (uint8_t)ev;
        }
      } else {
        store4(static_cast<float*>(t.M), i, n, m[u]);
        store4(static_cast<float*>(t.V), i, n, v[u]);
      }
    }
  }
}

// What a state of 8 bits stands for, 16 entries a lane.
template <bool kRoot, bool kBf16>
__global__ __launch_bounds__(kThreads) void state8_values_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ exps, int64_t n,
                                                                 void* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16;
  if (i >= n) return;
  const int E = exps[i / 64];
  uint32_t c[4];
  if (i + 16 <= n) {
    const uint4 all = *reinterpret_cast<const uint4*>(codes + i);
    c[0] = all.x;
    c[1] = all.y;
    c[2] = all.z;
    c[3] = all.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = load_codes(codes, i + 4 * k, n);
  }
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint32_t a = c[e / 4] >> (8 * (e % 4)) & 255;
    x[e] = kRoot ? held_value<kFracV>(a, E) : held_value<kFracM>(a & 127, E);
    if (!kRoot && a & 128) x[e] = -x[e];
  }
  if constexpr (kBf16) {
    // five significant bits at most: the upper half holds them all
    uint16_t* const o = static_cast<uint16_t*>(out) + i;
    const auto upper = [&](int e) { return __builtin_bit_cast(uint32_t, x[e]) >> 16; };
    if (i + 16 <= n) {
      uint4 w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = make_uint4(upper(8 * k) | upper(8 * k + 1) << 16, upper(8 * k + 2) | upper(8 * k + 3) << 16,
                          upper(8 * k + 4) | upper(8 * k + 5) << 16, upper(8 * k + 6) | upper(8 * k + 7) << 16);
      reinterpret_cast<uint4*>(o)[0] = w[0];
      reinterpret_cast<uint4*>(o)[1] = w[1];
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (i + e < n) o[e] = (uint16_t)upper(e);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      store4(static_cast<float*>(out), i + 4 * k, n, float4v{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]});
  }
}

int64_t chunks_of(int64_t n, int64_t chunk) { return (n + chunk - 1) / chunk; }

}  // namespace

int64_t grad_norm_workspace(const int64_t* sizes, int64_t count) {
  int64_t parts = 0;
  for (int64_t k = 0; k < count; ++k) parts += chunks_of(sizes[k], kNormChunk);
  return parts * (int64_t)sizeof(double);
}

hipError_t launch_grad_norm(const void* const* grads, const int64_t* sizes, int64_t count, bool f16, double scale,
                            double max_norm, void* control, void* ws, hipStream_t s) {
  double* const part = static_cast<double*>(ws);
  int64_t parts = 0;
  NormTable tab;
  tab.count = 0;
  uint32_t chunks = 0;
  const auto flush = [&]() {
    if (tab.count == 0) return hipSuccess;
    const dim3 grid(chunks), block(kThreads);
    if (f16) hipLaunchKernelGGL(squares_kernel<true>, grid, block, 0, s, tab, part + parts);
    else hipLaunchKernelGGL(squares_kernel<false>, grid, block, 0, s, tab, part + parts);
    parts += chunks;
    tab.count = 0;
    chunks = 0;
    return hipGetLastError();
  };
  for (int64_t k = 0; k < count; ++k) {
    const int64_t c = chunks_of(sizes[k], kNormChunk);
    if (c == 0) continue;
    if (tab.count == kNormTensors || chunks + c > kMaxGrid) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    tab.g[tab.count] = grads[k];
    tab.n[tab.count] = sizes[k];
    tab.first[tab.count++] = chunks;
    chunks += (uint32_t)c;
  }
  const hipError_t e = flush();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1024), 0, s, part, parts, scale, max_norm, static_cast<Control*>(control));
  return hipGetLastError();
}

namespace {
template <bool kF16, bool k8>
hipError_t launch_adamw_of(const sp24_adamw_job* jobs, int64_t count, const AdamwParams& prm, hipStream_t s) {
  AdamTable<k8> tab;
  tab.b1 = (float)prm.beta1;
  tab.c1 = (float)(1.0 - prm.beta1);
  tab.b2 = (float)prm.beta2;
  tab.c2 = (float)(1.0 - prm.beta2);
  tab.eps = (float)prm.eps;
  tab.ln_b1 = (float)std::log(prm.beta1);
  tab.ln_b2 = (float)std::log(prm.beta2);
  tab.step = prm.step;
  tab.control = static_cast<const Control*>(prm.control);
  tab.seed = prm.seed;
  tab.count = 0;
  uint32_t chunks = 0;
  const auto flush = [&]() {
    if (tab.count == 0) return hipSuccess;
    hipLaunchKernelGGL((adamw_kernel<kF16, k8>), dim3(chunks), dim3(kThreads), 0, s, tab);
    tab.count = 0;
    chunks = 0;
    return hipGetLastError();
  };
  for (int64_t k = 0; k < count; ++k) {
    const sp24_adamw_job& j = jobs[k];
    const int64_t c = chunks_of(j.n, kAdamChunk);
    if (c == 0) continue;
    if (tab.count == AdamTable<k8>::kTensors || chunks + c > kMaxGrid) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    AdamEntry<k8>& t = tab.t[tab.count];
    t.G = j.G;
    t.P = j.P;
    t.M = j.M;
    t.V = j.V;
    t.W = static_cast<uint16_t*>(j.W);
    t.n = j.n;
    t.lr = j.lr;
    t.keep = 1.0f - j.decay;
    if constexpr (k8) {
      t.ME = j.M_exps;
      t.VE = j.V_exps;
      t.place = (uint32_t)k;
    }
    tab.first[tab.count++] = chunks;
    chunks += (uint32_t)c;
  }
  return flush();
}
}  // namespace

hipError_t launch_adamw(const sp24_adamw_job* jobs, int64_t count, bool f16, bool state8, const AdamwParams& prm, hipStream_t s) {
  if (f16) return state8 ? launch_adamw_of<true, true>(jobs, count, prm, s) : launch_adamw_of<true, false>(jobs, count, prm, s);
  return state8 ? launch_adamw_of<false, true>(jobs, count, prm, s) : launch_adamw_of<false, false>(jobs, count, prm, s);
}

hipError_t launch_state8_values(const uint8_t* codes, const uint8_t* exps, int64_t n, bool root, bool bf16, void* out,
                                hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)chunks_of(n, 16 * kThreads)), block(kThreads);
  if (root && bf16) hipLaunchKernelGGL((state8_values_kernel<true, true>), grid, block, 0, s, codes, exps, n, out);
  else if (root) hipLaunchKernelGGL((state8_values_kernel<true, false>), grid, block, 0, s, codes, exps, n, out);
  else if (bf16) hipLaunchKernelGGL((state8_values_kernel<false, true>), grid, block, 0, s, codes, exps, n, out);
  else hipLaunchKernelGGL((state8_values_kernel<false, false>), grid, block, 0, s, codes, exps, n, out);
  return hipGetLastError();
}

}  // namespace sp24
