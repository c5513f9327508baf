// The layer's 2:4 products with what surrounds them: bias, activation and
// residual after the forward product, the activation's slope and the bias
// gradient after the input gradient; and the bias gradient alone.
//
//   forward   U = A S^T + bias,  out = act(U) + add        (A = X, S = the row form)
//   backward  out = (A S^T) * act'(U), sums over tokens    (A = dY, S = the column form)
//
// Sums, activations and slopes are in fp32; results are rounded once.  The
// backward's sums are of the unrounded values, per block of tokens into the
// workspace and then over the blocks in order, so the same call gives the same
// bits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sp24_device.hpp"
#include "sp24_epilogue.hpp"
#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 half16 __attribute__((ext_vector_type(16)));
typedef float float4v __attribute__((ext_vector_type(4)));

// What a product's epilogue reads and writes besides the product.
struct Finish {
  const float* bias;       // [N] or null (forward)
  const uint16_t* add;     // [T][N] or null (forward)
  const uint16_t* u_in;    // [T][N], or null without an activation (backward)
  uint16_t* u_out;         // [T][N] or null (forward)
  uint16_t* out;           // [T][N]
  float* sums;             // [blocks of tokens][N] or null (backward)
  int act;
};

// ---------------------------------------------------------------------------
// Products of few tokens.
//
// v_smfmac_f32_16x16x64_f16 takes 16 features x 64 of the reduction, one block
// of the blocked order: lane l (g = l / 16) holds of S row l % 16, dense k in
// [16g, 16g + 16) as 8 kept values and one meta word, so that a wave's load of
// 16 rows of a block is 1 KB of consecutive memory; of B column (token) l % 16,
// k in [8g, 8g + 8) and [32 + 8g, 32 + 8g + 8); of D column l % 16, rows
// 4g .. 4g + 3.  Every byte of S is used by one wave, so S goes from memory
// straight to registers.  The waves of a workgroup share the reduction out by
// blocks and join their sums in LDS, in the order of the waves.
template <int NT, int WAVES, bool kBwd>
__global__ __launch_bounds__(64 * WAVES) void spmm_thin_kernel(const uint16_t* __restrict__ A,
                                                               const uint16_t* __restrict__ vals,
                                                               const uint16_t* __restrict__ meta, int64_t T, int64_t N,
                                                               int64_t K, Finish fin) {
  __shared__ float4v part[WAVES][NT][64];
  __shared__ float4v colsum[NT][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t f0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * NT);
  const int64_t r0 = f0 & ~(int64_t)63, h = min<int64_t>(64, N - r0), row = f0 - r0 + l16;
  const uint16_t* const band_v = vals + r0 * (K / 2);
  const uint16_t* const band_m = meta + r0 * (K / 16);
  const uint16_t* tok[NT];   // tokens past the last read the last one's row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) tok[nt] = A + min<int64_t>(t0 + nt * 16 + l16, T - 1) * K;
  float4v acc[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t whole = K / 64;
  for (int64_t b = wave; b < whole; b += WAVES) {
    const half8 s = *reinterpret_cast<const half8*>(band_v + b * 32 * h + row * 32 + g * 8);
    const int idx = band_m[b * 4 * h + row * 4 + g];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const half8 lo = *reinterpret_cast<const half8*>(tok[nt] + b * 64 + 8 * g);
      const half8 hi = *reinterpret_cast<const half8*>(tok[nt] + b * 64 + 32 + 8 * g);
      const half16 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
      acc[nt] = __builtin_amdgcn_smfmac_f32_16x16x64_f16(s, x, acc[nt], idx, 0, 0);
    }
  }
  const int left = (int)(K - whole * 64);   // 0, 16, 32 or 48 columns of a narrower last block
  if (left != 0 && wave == (int)(whole % WAVES)) {
    const int w = left / 16;   // meta words a row
    half8 s = {};
    int idx = 0;
    if (g < w) {
      s = *reinterpret_cast<const half8*>(band_v + whole * 32 * h + row * (w * 8) + g * 8);
      idx = band_m[whole * 4 * h + row * w + g];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      half8 lo = {}, hi = {};
      if (8 * g < left) lo = *reinterpret_cast<const half8*>(tok[nt] + whole * 64 + 8 * g);
      if (32 + 8 * g < left) hi = *reinterpret_cast<const half8*>(tok[nt] + whole * 64 + 32 + 8 * g);
      const half16 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
      acc[nt] = __builtin_amdgcn_smfmac_f32_16x16x64_f16(s, x, acc[nt], idx, 0, 0);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) part[wave][nt][lane] = acc[nt];
  __syncthreads();

  // a lane finishes 4 features of one token
  for (int nt = wave; nt < NT; nt += WAVES) {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float4v p = part[w][nt][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] += p[e];
    }
    const int64_t t = t0 + nt * 16 + l16, at = t * N + f0 + 4 * g;
    const bool real = t < T;
    if constexpr (kBwd) {
      if (real) {
        if (fin.u_in != nullptr) {
          const half4 u = *reinterpret_cast<const half4*>(fin.u_in + at);
          const float uf[4] = {(float)u[0], (float)u[1], (float)u[2], (float)u[3]};
          times_slope(fin.act, uf, d);
        }
        *reinterpret_cast<half4*>(fin.out + at) = half4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
      }
      if (fin.sums != nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = real ? d[e] : 0.0f;
#pragma unroll
          for (int x = 1; x < 16; x *= 2) v += __shfl_xor(v, x);
          if (l16 == 0) colsum[nt][g][e] = v;
        }
      }
    } else if (real) {
      if (fin.bias != nullptr) {
        const float4v bias = *reinterpret_cast<const float4v*>(fin.bias + f0 + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] += bias[e];
      }
      if (fin.u_out != nullptr)
        *reinterpret_cast<half4*>(fin.u_out + at) = half4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
      activate(fin.act, d);
      if (fin.add != nullptr) {
        const half4 r = *reinterpret_cast<const half4*>(fin.add + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] += (float)r[e];
      }
      *reinterpret_cast<half4*>(fin.out + at) = half4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
    }
  }
  if constexpr (kBwd) {
    __syncthreads();
    if (fin.sums != nullptr && threadIdx.x < 16) {
      float v = 0.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) v += colsum[nt][threadIdx.x / 4][threadIdx.x % 4];
      fin.sums[(int64_t)blockIdx.y * N + f0 + threadIdx.x] = v;
    }
  }
}

constexpr int kThinTokens = 64;   // of a workgroup, and of a block of the backward's sums

template <bool kBwd>
hipError_t launch_thin(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                       const Finish& fin, hipStream_t s) {
  // a grid's second dimension takes 65535 workgroups
  constexpr int64_t kMost = 65535 * (int64_t)kThinTokens;
  for (int64_t t = 0; t < T; t += kMost) {
    const int64_t rows = std::min<int64_t>(kMost, T - t);
    Finish f = fin;
    if (f.add) f.add += t * N;
    if (f.u_in) f.u_in += t * N;
    if (f.u_out) f.u_out += t * N;
    f.out += t * N;
    if (f.sums) f.sums += t / kThinTokens * N;
    const uint16_t* a = A + t * K;
    const unsigned gx = (unsigned)(N / 16);
    if (rows <= 16)
      hipLaunchKernelGGL((spmm_thin_kernel<1, 8, kBwd>), dim3(gx, 1), dim3(512), 0, s, a, vals, meta, rows, N, K, f);
    else if (rows <= 32)
      hipLaunchKernelGGL((spmm_thin_kernel<2, 8, kBwd>), dim3(gx, 1), dim3(512), 0, s, a, vals, meta, rows, N, K, f);
    else
      hipLaunchKernelGGL((spmm_thin_kernel<4, 8, kBwd>), dim3(gx, (unsigned)((rows + 63) / 64)), dim3(512), 0, s, a, vals,
                         meta, rows, N, K, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Sums over rows.

// out[c] = the sum of rows [0, P) of part[P][N], in order.
__global__ __launch_bounds__(256) void join_rows_kernel(const float* __restrict__ part, int64_t P, int64_t N,
                                                        float* __restrict__ out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  float v = 0.0f;
  for (int64_t p = 0; p < P; ++p) v += part[p * N + c];
  out[c] = v;
}

hipError_t launch_join_rows(const float* part, int64_t P, int64_t N, float* out, hipStream_t s) {
  hipLaunchKernelGGL(join_rows_kernel, dim3((unsigned)((N + 255) / 256)), dim3(256), 0, s, part, P, N, out);
  return hipGetLastError();
}

// Sums of dY's columns over a chunk of rows: a lane takes 8 columns, the four
// waves of a workgroup every fourth row.
__global__ __launch_bounds__(256) void column_sums_kernel(const uint16_t* __restrict__ dY, int64_t T, int64_t R,
                                                          int64_t rows, float* __restrict__ out) {
  __shared__ float part[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 512 + lane * 8;
  const int64_t first = (int64_t)blockIdx.y * rows, last = min<int64_t>(T, first + rows);
  float v[8] = {};
  if (c < R)
    for (int64_t t = first + wave; t < last; t += 4) {
      const half8 x = *reinterpret_cast<const half8*>(dY + t * R + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += (float)x[e];
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[wave][lane * 8 + e] = v[e];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + k;
    if (col < R) out[blockIdx.y * R + col] = part[0][k] + part[1][k] + (part[2][k] + part[3][k]);
  }
}

// Rows of a workgroup: chunks of 64 or more, about 2048 workgroups at most.
int64_t sum_chunks(int64_t T, int64_t R) {
  const int64_t panels = (R + 511) / 512;
  const int64_t most = std::max<int64_t>(1, 2048 / panels);
  return std::max<int64_t>(1, std::min<int64_t>((T + 63) / 64, most));
}

}  // namespace

int64_t bias_grad_workspace(int64_t T, int64_t R) {
  const int64_t P = sum_chunks(T, R);
  return P > 1 ? P * R * 4 : 0;
}

hipError_t launch_bias_grad(const uint16_t* dY, int64_t T, int64_t R, float* out, void* ws, hipStream_t s) {
  if (R == 0) return hipSuccess;
  const int64_t P = sum_chunks(T, R), rows = (T + P - 1) / P;
  float* part = P > 1 ? static_cast<float*>(ws) : out;
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)((R + 511) / 512), (unsigned)P), dim3(256), 0, s, dY, T, R, rows,
                     part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || P == 1) return e;
  return launch_join_rows(part, P, R, out, s);
}

hipError_t launch_spmm_act_fwd(const uint16_t* X, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N,
                               int64_t K, const float* bias, int act, const uint16_t* residual, uint16_t* U,
                               uint16_t* Y, hipStream_t s) {
  if (T == 0 || N == 0) return hipSuccess;
  const Finish fin{bias, residual, nullptr, U, Y, nullptr, act};
  return launch_thin<false>(X, vals, meta, T, N, K, fin, s);
}

int64_t spmm_act_bwd_workspace(int64_t T, int64_t N) {
  const int64_t P = (T + kThinTokens - 1) / kThinTokens;
  return P > 1 ? P * N * 4 : 0;
}

hipError_t launch_spmm_act_bwd(const uint16_t* dY, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N,
                               int64_t K, int act, const uint16_t* U, uint16_t* dU, float* dbias, void* ws,
                               hipStream_t s) {
  if (N == 0) return hipSuccess;
  if (T == 0) return dbias ? launch_bias_grad(nullptr, 0, N, dbias, nullptr, s) : hipSuccess;
  const int64_t P = (T + kThinTokens - 1) / kThinTokens;
  float* sums = dbias == nullptr ? nullptr : P > 1 ? static_cast<float*>(ws) : dbias;
  const Finish fin{nullptr, nullptr, U, nullptr, dU, sums, act};
  const hipError_t e = launch_thin<true>(dY, vals, meta, T, N, K, fin, s);
  if (e != hipSuccess || sums == nullptr || P == 1) return e;
  return launch_join_rows(sums, P, N, dbias, s);
}

}  // namespace sp24
