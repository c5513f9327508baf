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
#include "sp24_spmm_tile.hpp"

namespace sp24 {
namespace {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

// What a product's epilogue reads and writes besides the product.
struct Finish {
  const float* bias;       // [N] or null (forward)
  const uint16_t* add;     // [T][N] or null (forward)
  const uint16_t* u_in;    // [T][N] (backward; null without an activation)
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
    const h8 s = *reinterpret_cast<const h8*>(band_v + b * 32 * h + row * 32 + g * 8);
    const int idx = band_m[b * 4 * h + row * 4 + g];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const h8 lo = *reinterpret_cast<const h8*>(tok[nt] + b * 64 + 8 * g);
      const h8 hi = *reinterpret_cast<const h8*>(tok[nt] + b * 64 + 32 + 8 * g);
      const h16 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
      acc[nt] = __builtin_amdgcn_smfmac_f32_16x16x64_f16(s, x, acc[nt], idx, 0, 0);
    }
  }
  const int left = (int)(K - whole * 64);   // 0, 16, 32 or 48 columns of a narrower last block
  if (left != 0 && wave == (int)(whole % WAVES)) {
    const int w = left / 16;   // meta words a row
    h8 s = {};
    int idx = 0;
    if (g < w) {
      s = *reinterpret_cast<const h8*>(band_v + whole * 32 * h + row * (w * 8) + g * 8);
      idx = band_m[whole * 4 * h + row * w + g];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      h8 lo = {}, hi = {};
      if (8 * g < left) lo = *reinterpret_cast<const h8*>(tok[nt] + whole * 64 + 8 * g);
      if (32 + 8 * g < left) hi = *reinterpret_cast<const h8*>(tok[nt] + whole * 64 + 32 + 8 * g);
      const h16 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
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
        if (fin.act != kActNone) {
          const h4 u = *reinterpret_cast<const h4*>(fin.u_in + at);
          with_act(fin.act, [&](auto kind) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = times_slope<decltype(kind)::value>(d[e], (float)u[e]);
          });
        }
        *reinterpret_cast<h4*>(fin.out + at) = h4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
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
        *reinterpret_cast<h4*>(fin.u_out + at) = h4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
      with_act(fin.act, [&](auto kind) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = activate<decltype(kind)::value>(d[e]);
      });
      if (fin.add != nullptr) {
        const h4 r = *reinterpret_cast<const h4*>(fin.add + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] += (float)r[e];
      }
      *reinterpret_cast<h4*>(fin.out + at) = h4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
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
// Products of many tokens: the tile of sp24_spmm_tile.hpp.
//
// Epilogue.  A wave's sums go through LDS as fp32, 32 tokens x 128 features at a
// time, and come back as 8 consecutive features of one token in a lane.  All
// global accesses are whole token rows then, 16 bytes a lane; bias, slope sums
// and addresses are the same for all of a lane's tokens; and the activation's
// code is there once, in a rolled loop, where over the accumulators it would be
// there 8 times for each kind.
//
// Staging: 16-byte chunks c = 0..31 of a token's 128 features, the even ones in
// the first half of its 512 bytes and the odd ones in the second, each half
// XOR-swizzled by the token, so that 8 lanes that write one chunk of 8 tokens,
// and 16 that read 16 chunks of one, meet no bank twice.
template <int BM, int BN, int WM, int WN, bool kBwd, bool kTail>
__device__ __forceinline__ void spmm_act_tile(unsigned char* __restrict__ smem, const uint16_t* __restrict__ A,
                                              const uint16_t* __restrict__ vals, const uint16_t* __restrict__ meta,
                                              int64_t T, int64_t N, int64_t K, int tm, int tn, int tid,
                                              const Finish& fin, int64_t ld, int64_t t0) {
#include "sp24_spmm_loop.inc"

  if constexpr (kTail) {
    // the last 16, 32 or 48 of the reduction, a narrower block of the forms:
    // straight from memory, zeros past its end
    const int64_t k0 = K / 64 * 64;
    const int left = (int)(K - k0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int c = 2 * st + g;   // this lane's 16 of the reduction in S
      h8 a[Cfg::TM];
      int idx[Cfg::TM];
#pragma unroll
      for (int mt = 0; mt < Cfg::TM; ++mt) {
        const int64_t row = min<int64_t>(m0 + wm * WM + mt * 32 + l32, N - 1), r0 = row & ~(int64_t)63;
        const int64_t h = min<int64_t>(64, N - r0);
        a[mt] = h8{};
        idx[mt] = 0;
        if (16 * c < left) {
          a[mt] = *reinterpret_cast<const h8*>(vals + r0 * (K / 2) + k0 / 2 * h + (row - r0) * (left / 2) + 8 * c);
          idx[mt] = meta[r0 * (K / 16) + k0 / 16 * h + (row - r0) * (left / 16) + c];
        }
      }
#pragma unroll
      for (int nt = 0; nt < Cfg::TN; ++nt) {
        const int64_t row = min<int64_t>(wn * WN + nt * 32 + l32, T - 1);
        const uint16_t* const x = A + row * K + k0 + 32 * st + 8 * g;
        h8 lo = {}, hi = {};
        if (32 * st + 8 * g < left) lo = *reinterpret_cast<const h8*>(x);
        if (32 * st + 16 + 8 * g < left) hi = *reinterpret_cast<const h8*>(x + 16);
        const h16 b = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
        for (int mt = 0; mt < Cfg::TM; ++mt)
          acc[mt][nt] = __builtin_amdgcn_smfmac_f32_32x32x32_f16(a[mt], b, acc[mt][nt], idx[mt], 0, 0);
      }
    }
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();   // no wave reads the ring any more
  asm volatile("" ::: "memory");
  unsigned char* const staged = smem + (size_t)wave * 16384;
  const int q = lane & 15;        // this lane's 8 features
  const int64_t m = m0 + wm * WM + 8 * q;
  const bool inside = m < N;
  float bias[8] = {};
  if (!kBwd && fin.bias != nullptr && inside)
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = fin.bias[m + e];
  // What the epilogue reads beside the sums (the residual, or U) is fetched
  // eight passes of 4 tokens early, rows past the last one from the last one.
  // (Four: 293 us with a residual at 16384 x 6400 x 1600, eight: 276; none
  // early: 304.)
  const uint16_t* const beside = kBwd ? fin.u_in : fin.add;
  h8 next[8];
  const int first = lane >> 4, last = (int)T - 1;
  const uint16_t* const from_m = beside + t0 * ld + (inside ? m : 0);
  const auto fetch = [&](int pass) {
    return *reinterpret_cast<const h8*>(from_m + (int64_t)min(wn * WN + pass * 4 + first, last) * ld);
  };
  if (beside != nullptr)
#pragma unroll
    for (int k = 0; k < 8; ++k) next[k] = fetch(k);
  float sums[8] = {};
#pragma unroll
  for (int nt = 0; nt < Cfg::TN; ++nt) {
#pragma unroll
    for (int mt = 0; mt < Cfg::TM; ++mt)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const f16v& a = acc[mt][nt];
        *reinterpret_cast<float4v*>(staged + l32 * 512 + g * 256 + (((mt * 4 + i4) ^ (l32 & 15)) * 16)) =
            float4v{a[4 * i4], a[4 * i4 + 1], a[4 * i4 + 2], a[4 * i4 + 3]};
      }
    // the wave reads back only what it wrote, in order: no barrier is needed
    with_act(fin.act, [&](auto kind) __attribute__((always_inline)) {
      constexpr int kAct = decltype(kind)::value;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int t = it * 4 + first;
        const unsigned char* const from = staged + t * 512 + ((q ^ (t & 15)) * 16);
        const float4v lo = *reinterpret_cast<const float4v*>(from);
        const float4v hi = *reinterpret_cast<const float4v*>(from + 256);
        const h8 now = next[it];
        if (beside != nullptr && nt + 1 < Cfg::TN) next[it] = fetch((nt + 1) * 8 + it);
        const int n = wn * WN + nt * 32 + t;
        if (n > last || !inside) continue;
        const int64_t at = (t0 + n) * ld + m;
        float d[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if constexpr (kBwd) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (kAct != kActNone) d[e] = times_slope<kAct>(d[e], (float)now[e]);
            sums[e] += d[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] += bias[e];
          if (fin.u_out != nullptr) {
            h8 u;
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = (_Float16)d[e];
            *reinterpret_cast<h8*>(fin.u_out + at) = u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = activate<kAct>(d[e]);
          if (beside != nullptr)
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] += (float)now[e];
        }
        h8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (_Float16)d[e];
        *reinterpret_cast<h8*>(fin.out + at) = y;
      }
    });
  }
  if constexpr (kBwd) {
    if (fin.sums == nullptr) return;   // the same in all waves
    // over the wave's four tokens at a time, then over the waves side by side
    float* const all = reinterpret_cast<float*>(smem);   // [WAVES_N][BM]
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[e] += __shfl_xor(sums[e], 16);
      sums[e] += __shfl_xor(sums[e], 32);
    }
    __syncthreads();
    if (lane < 16)
#pragma unroll
      for (int e = 0; e < 8; ++e) all[wn * BM + wm * WM + 8 * q + e] = sums[e];
    __syncthreads();
    for (int c = tid; c < BM; c += Cfg::THREADS) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < Cfg::WAVES_N; ++w) v += all[w * BM + c];
      if (m0 + c < N) fin.sums[t0 / BN * ld + m0 + c] = v;
    }
  }
}

template <int BM, int BN, int WM, int WN, bool kBwd, bool kTail>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 1) void spmm_act_kernel(
    const uint16_t* __restrict__ A, const uint16_t* __restrict__ vals, const uint16_t* __restrict__ meta, int64_t T,
    int64_t N, int64_t K, Finish fin, int64_t ld, int tiles_m, int tiles_n) {
  using Cfg = FastCfg<BM, BN, WM, WN>;
  __shared__ __align__(1024) unsigned char smem[3 * (Cfg::S_BYTES + Cfg::B_BYTES + Cfg::M_BYTES)];
  static_assert(WM == 128 && WN % 32 == 0 && Cfg::WAVES * 16384 <= sizeof(smem), "staging");

  // tile order as in the products alone: groups of 8 feature tiles, token tiles
  // within a group, features fastest, a contiguous run of it for each XCD
  constexpr int kGroupM = 8;
  const int ntiles = tiles_m * tiles_n, per_xcd = (ntiles + 7) / 8;
  const int lin = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (lin >= ntiles) return;
  const int group = lin / (kGroupM * tiles_n), gm0 = group * kGroupM, gsize = min(kGroupM, tiles_m - gm0);
  const int in_group = lin - group * kGroupM * tiles_n;
  const int tn = __builtin_amdgcn_readfirstlane(in_group / gsize);
  const int tm = __builtin_amdgcn_readfirstlane(gm0 + in_group % gsize);

  // the tile's tokens as a matrix of their own, so that the direct loads' 32-bit
  // offsets count from its first row however many tokens there are
  const int64_t t0 = (int64_t)tn * BN;
  spmm_act_tile<BM, BN, WM, WN, kBwd, kTail>(smem, A + t0 * K, vals, meta, T - t0 < BN ? T - t0 : BN, N, K, tm, 0,
                                             (int)threadIdx.x, fin, ld, t0);
}

// Features [m, m + n) of a product over N, for all tokens.
template <int BM, int BN, int WM, int WN, bool kBwd>
hipError_t launch_tiles(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                        Finish f, int64_t m, int64_t n, hipStream_t s) {
  const int tiles_m = (int)((n + BM - 1) / BM), tiles_n = (int)((T + BN - 1) / BN);
  const dim3 grid((unsigned)((tiles_m * tiles_n + 7) / 8 * 8)), block(FastCfg<BM, BN, WM, WN>::THREADS);
  vals += m * (K / 2);   // m is a multiple of 64: a band's start
  meta += m * (K / 16);
  if (f.bias) f.bias += m;
  if (f.add) f.add += m;
  if (f.u_in) f.u_in += m;
  if (f.u_out) f.u_out += m;
  if (f.sums) f.sums += m;
  f.out += m;
  if (K % 64 == 0)
    hipLaunchKernelGGL((spmm_act_kernel<BM, BN, WM, WN, kBwd, false>), grid, block, 0, s, A, vals, meta, T, n, K, f, N,
                       tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((spmm_act_kernel<BM, BN, WM, WN, kBwd, true>), grid, block, 0, s, A, vals, meta, T, n, K, f, N,
                       tiles_m, tiles_n);
  return hipGetLastError();
}

// The most tokens that run without tiles.
constexpr int64_t kMostThin = 64;

// Whether the tiles take a product: its 32-bit offsets reach 256 rows of A and
// all of S, and a launch counts its work-items in 32 bits.
bool in_tiles(int64_t T, int64_t N, int64_t K) {
  constexpr int64_t kMaxBuf = (int64_t)1 << 31;
  return T > kMostThin && K >= 64 && K * 512 < kMaxBuf && N * K < kMaxBuf &&
         ((T + 63) / 64) * ((N + 127) / 128) < ((int64_t)1 << 22);
}

// A backward's partial sums: features below `features` have a row for each
// `first` tokens, the others one for each `rest`.
struct Blocks {
  int64_t features, first, rest;
};

template <bool kBwd>
hipError_t launch_product(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                          const Finish& fin, Blocks* blocks, hipStream_t s) {
  if (!in_tiles(T, N, K)) {
    *blocks = {N, T <= 16 ? 16 : T <= 32 ? 32 : kThinTokens, kThinTokens};
    return launch_thin<kBwd>(A, vals, meta, T, N, K, fin, s);
  }
  const int64_t cus = device_cu_count(), tiles = ((T + 255) / 256) * ((N + 255) / 256);
  if (tiles < cus) {
    *blocks = {N, 128, 128};
    return launch_tiles<128, 128, 128, 32, kBwd>(A, vals, meta, T, N, K, fin, 0, N, s);
  }
  *blocks = {N, 256, 256};
  return launch_tiles<256, 256, 128, 64, kBwd>(A, vals, meta, T, N, K, fin, 0, N, s);
}

// ---------------------------------------------------------------------------
// Sums over rows.

// out[c] = the sum of part[P][N]'s rows: P rows for columns below `split` (a
// multiple of 64), Q for the others.  Eight waves take every eighth row, eight
// rows at a time, of 64 columns, and their sums are added in order.
__global__ __launch_bounds__(512) void join_rows_kernel(const float* __restrict__ part, int64_t P, int64_t split,
                                                        int64_t Q, int64_t N, float* __restrict__ out) {
  __shared__ float waves[8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  if (c - lane >= split) P = Q;
  float v = 0.0f;
  if (c < N)
    for (int64_t p = wave; p < P; p += 64) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = p + 8 * k < P ? part[(p + 8 * k) * N + c] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += x[k];
    }
  waves[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= N) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) v += waves[w][lane];
  out[c] = v;
}

hipError_t launch_join_rows(const float* part, int64_t P, int64_t split, int64_t Q, int64_t N, float* out,
                            hipStream_t s) {
  hipLaunchKernelGGL(join_rows_kernel, dim3((unsigned)((N + 63) / 64)), dim3(512), 0, s, part, P, split, Q, N, out);
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
    for (int64_t t = first + wave; t < last; t += 32) {
      h8 x[8];   // eight rows under way at once
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = t + 4 * k < last ? *reinterpret_cast<const h8*>(dY + (t + 4 * k) * R + c) : h8{};
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += (float)x[k][e];
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
  return launch_join_rows(part, P, R, P, R, out, s);
}

hipError_t launch_spmm_act_fwd(const uint16_t* X, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N,
                               int64_t K, const float* bias, int act, const uint16_t* residual, uint16_t* U,
                               uint16_t* Y, hipStream_t s) {
  if (T == 0 || N == 0) return hipSuccess;
  const Finish fin{bias, residual, nullptr, U, Y, nullptr, act};
  Blocks blocks;
  return launch_product<false>(X, vals, meta, T, N, K, fin, &blocks, s);
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
  const Finish fin{nullptr, nullptr, act == kActNone ? nullptr : U, nullptr, dU, sums, act};
  Blocks b;
  const hipError_t e = launch_product<true>(dY, vals, meta, T, N, K, fin, &b, s);
  if (e != hipSuccess || sums == nullptr || P == 1) return e;
  return launch_join_rows(sums, (T + b.first - 1) / b.first, b.features, (T + b.rest - 1) / b.rest, N, dbias, s);
}

}  // namespace sp24
