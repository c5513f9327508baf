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

constexpr int64_t kCus = 256;   // of an MI355X

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

// What a kernel makes of its sums: kPartial leaves them as they are.
enum { kForward, kBackward, kPartial };

// A lane's 4 consecutive features of one token, from element `at` of the
// matrices and feature f.
template <bool kBwd>
__device__ __forceinline__ void finish4(const Finish& fin, int64_t at, int64_t f, float (&d)[4]) {
  if constexpr (kBwd) {
    if (fin.act != kActNone) {
      const h4 u = *reinterpret_cast<const h4*>(fin.u_in + at);
      with_act(fin.act, [&](auto kind) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = times_slope<decltype(kind)::value>(d[e], (float)u[e]);
      });
    }
  } else {
    if (fin.bias != nullptr) {
      const float4v bias = *reinterpret_cast<const float4v*>(fin.bias + f);
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
  }
  *reinterpret_cast<h4*>(fin.out + at) = h4{(_Float16)d[0], (_Float16)d[1], (_Float16)d[2], (_Float16)d[3]};
}

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
//
// 6400 x 1600 (11.5 MB of weight, 2.3 us at a copy's rate): 4.5 us for one token, 6.1
// for 16; 1600 x 6400, 100 workgroups: 5.8 and 9.7.  Four blocks' loads under way at
// once are slower (one token 4.2 -> 4.8), 4 or 16 waves no faster.
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
    const int64_t t = t0 + nt * 16 + l16;
    const bool real = t < T;
    if (real) finish4<kBwd>(fin, t * N + f0 + 4 * g, f0 + 4 * g, d);
    if constexpr (kBwd)
      if (fin.sums != nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = real ? d[e] : 0.0f;
#pragma unroll
          for (int x = 1; x < 16; x *= 2) v += __shfl_xor(v, x);
          if (l16 == 0) colsum[nt][g][e] = v;
        }
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

// LDS of a tile's ring.
template <int BM, int BN>
constexpr int tile_bytes(int slots) { return slots * (BM * 72 + BN * 128); }

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
//
// Two workgroups share a CU, so that the matrix units have one's products while
// the other is in its epilogue: a ring of two slots for 256 x 128 tiles.  (One
// workgroup of 256 x 256 with three slots, at 16384 x 6400 x 1600: no epilogue
// work 232 us, GELU 267, backward through GELU 310; two of 256 x 128: 226, 244 and
// 284.)
//
// With kGroups = 2 a workgroup has two groups of waves, each of which sums up half
// of the stages of the whole tile, through a ring of its own at smem + group *
// kRing; their sums meet in the staging, and each finishes half of the tokens.
template <int BM, int BN, int WM, int WN, int kSlots, int kGroups, bool kBwd, bool kTail>
__device__ __forceinline__ void spmm_act_tile(unsigned char* __restrict__ base, const uint16_t* __restrict__ A,
                                              const uint16_t* __restrict__ vals, const uint16_t* __restrict__ meta,
                                              int64_t T, int64_t N, int64_t K, int tm, int tn, int thread,
                                              const Finish& fin, int64_t t0) {
  static_assert(kGroups == 1 || (kGroups == 2 && WN == 32), "a group finishes 16 of a wave's 32 tokens");
  constexpr int kThreads = FastCfg<BM, BN, WM, WN>::THREADS, kWaves = kThreads / 64;
  const int group = kGroups == 1 ? 0 : __builtin_amdgcn_readfirstlane(thread / kThreads);
  const int tid = kGroups == 1 ? thread : thread % kThreads;
  unsigned char* const smem = base + group * tile_bytes<BM, BN>(kSlots);
  const int n = (int)(K / 64), half = (n + kGroups - 1) / kGroups, kt0 = group * half;
  const auto stages = [&] { return kGroups == 1 ? n : group == 0 ? half : n - half; };
#include "sp24_spmm_loop.inc"
  // the second of an odd number of stages' halves has one stage less: its waves
  // meet the others' last barrier here
  if (kGroups == 2 && n % 2 != 0 && group == 1) __builtin_amdgcn_s_barrier();

  if (kTail && group == kGroups - 1) {
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
  unsigned char* const staged = base + (size_t)(group * kWaves + wave) * 16384;
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
  // Outputs of the large launch (that of the two-slot rings) are past what the L2s
  // hold: streamed, they leave the operands' strips there (16384 tokens, both
  // products of the 1600-wide layer's forward: 552 -> 525 us; backward 533 -> 530).
  const auto store8 = [](uint16_t* to, h8 v) {
    if constexpr (kSlots == 2) __builtin_nontemporal_store(v, reinterpret_cast<h8*>(to));
    else *reinterpret_cast<h8*>(to) = v;
  };
  constexpr int kPasses = 8 / kGroups;
  h8 next[kPasses];
  const int first = group * (4 * kPasses) + (lane >> 4), last = (int)T - 1;
  const uint16_t* const from_m = beside + t0 * N + (inside ? m : 0);
  const auto fetch = [&](int pass) {
    return *reinterpret_cast<const h8*>(from_m + (int64_t)min(wn * WN + pass * 4 + first, last) * N);
  };
  if (beside != nullptr)
#pragma unroll
    for (int k = 0; k < kPasses; ++k) next[k] = fetch(k);
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
    // of one group, the wave reads back only what it wrote, in order: no barrier is needed
    if constexpr (kGroups == 2) __syncthreads();
    with_act(fin.act, [&](auto kind) __attribute__((always_inline)) {
      constexpr int kAct = decltype(kind)::value;
#pragma unroll
      for (int it = 0; it < kPasses; ++it) {
        const int t = it * 4 + first;
        const unsigned char* const from = base + wave * 16384 + t * 512 + ((q ^ (t & 15)) * 16);
        float4v lo = *reinterpret_cast<const float4v*>(from);
        float4v hi = *reinterpret_cast<const float4v*>(from + 256);
        if constexpr (kGroups == 2) {
          lo += *reinterpret_cast<const float4v*>(from + kWaves * 16384);
          hi += *reinterpret_cast<const float4v*>(from + kWaves * 16384 + 256);
        }
        const h8 now = next[it];
        if (beside != nullptr && nt + 1 < Cfg::TN) next[it] = fetch((nt + 1) * 8 + it);
        const int n = wn * WN + nt * 32 + t;
        if (n > last || !inside) continue;
        const int64_t at = (t0 + n) * N + m;
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
            store8(fin.u_out + at, u);
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
        store8(fin.out + at, y);
      }
    });
  }
  if constexpr (kBwd) {
    if (fin.sums == nullptr) return;   // the same in all waves
    // over the wave's four tokens at a time, then over the waves side by side
    float* const all = reinterpret_cast<float*>(base);   // [kGroups][WAVES_N][BM]
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[e] += __shfl_xor(sums[e], 16);
      sums[e] += __shfl_xor(sums[e], 32);
    }
    __syncthreads();
    if (lane < 16)
#pragma unroll
      for (int e = 0; e < 8; ++e) all[(group * Cfg::WAVES_N + wn) * BM + wm * WM + 8 * q + e] = sums[e];
    __syncthreads();
    for (int c = thread; c < BM; c += kGroups * kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kGroups * Cfg::WAVES_N; ++w) v += all[w * BM + c];
      if (m0 + c < N) fin.sums[t0 / BN * N + m0 + c] = v;
    }
  }
}

// Tile `lin` of tiles_m x tiles_n in the order of the products alone: groups of 8
// feature tiles, token tiles within a group, features fastest.
__device__ __forceinline__ void tile_at(int lin, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kGroupM = 8;
  const int group = lin / (kGroupM * tiles_n), gm0 = group * kGroupM, gsize = min(kGroupM, tiles_m - gm0);
  const int in_group = lin - group * kGroupM * tiles_n;
  tn = __builtin_amdgcn_readfirstlane(in_group / gsize);
  tm = __builtin_amdgcn_readfirstlane(gm0 + in_group % gsize);
}

// The tile's tokens are a matrix of their own to it, so that the direct loads'
// 32-bit offsets count from its first row however many tokens there are.
template <int BM, int BN, int WM, int WN, int kSlots, int kGroups, bool kBwd, bool kTail>
__device__ __forceinline__ void spmm_act_at(unsigned char* smem, const uint16_t* A, const uint16_t* vals,
                                            const uint16_t* meta, int64_t T, int64_t N, int64_t K, const Finish& fin,
                                            int tm, int tn) {
  const int64_t t0 = (int64_t)tn * BN;
  spmm_act_tile<BM, BN, WM, WN, kSlots, kGroups, kBwd, kTail>(smem, A + t0 * K, vals, meta, T - t0 < BN ? T - t0 : BN, N, K,
                                                              tm, 0, (int)threadIdx.x, fin, t0);
}

// 256 x 128 tiles of the first `big` x 256 features and 128 x 128 tiles of the
// others, after them: the last, partly filled round of workgroups takes half as
// long, and a strip of up to 128 features no more than its own work.  (16384 x
// 6400 x 1600, 24 strips and two halves instead of 25: forward with GELU 268 -> 257 us, backward 284 -> 277.)  Each XCD
// takes a contiguous run of either.
template <bool kBwd, bool kTail>
__global__ __launch_bounds__(256, 2) void spmm_large_kernel(const uint16_t* __restrict__ A,
                                                            const uint16_t* __restrict__ vals,
                                                            const uint16_t* __restrict__ meta, int64_t T, int64_t N,
                                                            int64_t K, Finish fin, int big, int tiles_n) {
  __shared__ __align__(1024) unsigned char smem[tile_bytes<256, 128>(2)];
  static_assert(sizeof(smem) >= tile_bytes<128, 128>(2) && sizeof(smem) >= 4 * 16384, "either tile and its staging");
  const int nbig = big * tiles_n, big_per_xcd = (nbig + 7) / 8;
  const int x = (int)(blockIdx.x % 8), at = (int)(blockIdx.x / 8);
  int tm, tn;
  if (at < big_per_xcd) {
    const int lin = x * big_per_xcd + at;
    if (lin >= nbig) return;
    tile_at(lin, big, tiles_n, tm, tn);
    spmm_act_at<256, 128, 128, 64, 2, 1, kBwd, kTail>(smem, A, vals, meta, T, N, K, fin, tm, tn);
  } else {
    const int small = (int)((N - big * 256 + 127) / 128), nsmall = small * tiles_n, per_xcd = (nsmall + 7) / 8;
    const int lin = x * per_xcd + at - big_per_xcd;
    if (at - big_per_xcd >= per_xcd || lin >= nsmall) return;
    tile_at(lin, small, tiles_n, tm, tn);
    spmm_act_at<128, 128, 128, 32, 2, 1, kBwd, kTail>(smem, A, vals, meta, T, N, K, fin, 2 * big + tm, tn);
  }
}

template <bool kBwd>
hipError_t launch_large(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                        const Finish& f, hipStream_t s) {
  const int64_t tiles_n = (T + 127) / 128, slots = 2 * kCus, rounds = tiles_n * ((N + 255) / 256) / slots;
  // as many strips as fill whole rounds, if the rest takes one round of small tiles
  int64_t big = std::min(N / 256, rounds * slots / tiles_n);
  if ((N - big * 256 + 127) / 128 * tiles_n > slots) big = N / 256;
  const int64_t small = (N - big * 256 + 127) / 128;
  const dim3 grid((unsigned)(((big * tiles_n + 7) / 8 + (small * tiles_n + 7) / 8) * 8)), block(256);
  if (K % 64 == 0)
    hipLaunchKernelGGL((spmm_large_kernel<kBwd, false>), grid, block, 0, s, A, vals, meta, T, N, K, f, (int)big, (int)tiles_n);
  else
    hipLaunchKernelGGL((spmm_large_kernel<kBwd, true>), grid, block, 0, s, A, vals, meta, T, N, K, f, (int)big, (int)tiles_n);
  return hipGetLastError();
}

// 128 x 128 tiles throughout, with a three-slot ring: two workgroups a CU, or, for
// no more tiles than CUs, one of two groups of waves, which halves the chain of
// stages (0.4 us each).
template <int kGroups, bool kBwd, bool kTail>
__global__ __launch_bounds__(256 * kGroups, 2 / kGroups) void spmm_small_kernel(const uint16_t* __restrict__ A,
                                                            const uint16_t* __restrict__ vals,
                                                            const uint16_t* __restrict__ meta, int64_t T, int64_t N,
                                                            int64_t K, Finish fin, int tiles_m, int tiles_n) {
  __shared__ __align__(1024) unsigned char smem[kGroups * tile_bytes<128, 128>(3)];
  static_assert(sizeof(smem) >= kGroups * 4 * 16384, "the staging");
  const int ntiles = tiles_m * tiles_n, per_xcd = (ntiles + 7) / 8;
  const int lin = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (lin >= ntiles) return;
  int tm, tn;
  tile_at(lin, tiles_m, tiles_n, tm, tn);
  spmm_act_at<128, 128, 128, 32, 3, kGroups, kBwd, kTail>(smem, A, vals, meta, T, N, K, fin, tm, tn);
}

template <int kGroups, bool kBwd>
hipError_t launch_small(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                        const Finish& f, hipStream_t s) {
  const int tiles_m = (int)((N + 127) / 128), tiles_n = (int)((T + 127) / 128);
  const dim3 grid((unsigned)((tiles_m * tiles_n + 7) / 8 * 8)), block(256 * kGroups);
  if (K % 64 == 0)
    hipLaunchKernelGGL((spmm_small_kernel<kGroups, kBwd, false>), grid, block, 0, s, A, vals, meta, T, N, K, f, tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((spmm_small_kernel<kGroups, kBwd, true>), grid, block, 0, s, A, vals, meta, T, N, K, f, tiles_m, tiles_n);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Products whose tiles are too few for the CUs: 64 features x 64 tokens a
// workgroup, and the reduction shared out inside it.
//
// A long reduction over few tiles is a chain of stages, each of which waits for
// its operands, the LDS and the matrix unit in turn (0.4 us a stage of 64 in the
// tiles above), on a part of the CUs.  Here a workgroup of 16 waves has four
// groups of four; group k sums up the stages k, k + 4, k + 8, ... of the whole
// tile, 32 x 32 a wave, through a ring of its own, so that four stages are under
// way in each CU and a quarter as many follow one another; and the tiles are a
// quarter as large.  The four sums meet in LDS, in order.  (6400 x 1600 at 64 tokens:
// 15.3 us thin, 7.8 here; 1600 x 6400 at 512: 41.9 in 128 x 128 tiles, 20.6.)
//
// With few tokens there are too few tiles even so, and a CU's loads are the
// bound (51 KB a round of stages in 0.47 us, 52 bytes a cycle): `parts`
// workgroups share a tile's reduction then (kPartial), part p the stages
// [p n / parts, (p + 1) n / parts), the last one the tail too, into
// fin.sums + p T N, and join_parts_kernel finishes.
template <int kMode, bool kTail>
__global__ __launch_bounds__(1024, 1) void spmm_mid_kernel(const uint16_t* __restrict__ A,
                                                           const uint16_t* __restrict__ vals,
                                                           const uint16_t* __restrict__ meta, int64_t T, int64_t N,
                                                           int64_t K, Finish fin, int tiles_m, int tiles_n, int parts) {
  constexpr int kStage = 4096 + 8192 + 512, kSlots = 3;   // S, A and meta of 64 x 64 in K
  __shared__ __align__(1024) unsigned char smem[4 * kSlots * kStage];
  const int all = tiles_m * tiles_n * parts, per_xcd = (all + 7) / 8;
  const int lin = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (lin >= all) return;
  // an XCD's tiles share their strip of S
  const int tn = __builtin_amdgcn_readfirstlane(lin % tiles_n), strip = lin / tiles_n;
  const int part = __builtin_amdgcn_readfirstlane(strip % parts), tm = __builtin_amdgcn_readfirstlane(strip / parts);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave >> 2, w = wave & 3, wm = w & 1, wn = w >> 1, l32 = lane & 31, g = lane >> 5;
  const int64_t m0 = (int64_t)tm * 64, t0 = (int64_t)tn * 64;
  const int64_t h = min<int64_t>(64, N - m0), tokens = min<int64_t>(64, T - t0);
  const int all_n = (int)(K / 64), first = part * all_n / parts, n = (part + 1) * all_n / parts - first;
  const int mine = (n - kg + 3) / 4, rounds = (n + 3) / 4;

  // direct loads as in the tiles above: rows past T read as zero, rows past N
  // read zero or other rows of S and feed outputs that are not stored
  const i32x4 rs = make_rsrc(vals + m0 * (K / 2), (uint32_t)((N - m0) * K));
  const i32x4 rb = make_rsrc(A + t0 * K, (uint32_t)(tokens * K * 2));
  const i32x4 rm = make_rsrc(meta + m0 * (K / 16), (uint32_t)((N - m0) * (K / 8)));
  const int st_s = (int)h * 64, st_m = (int)h * 8;
  const int rs_row = 16 * w + lane / 4, rm_row = 32 * (w & 1) + lane / 2;
  const int off_s = rs_row * 64 + (((lane % 4) ^ swz_s(rs_row)) * 16), off_m = rm_row * 8 + (lane % 2) * 4;
  int off_b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * (2 * w + i) + lane / 8;
    off_b[i] = r * (int)K * 2 + (((lane % 8) ^ swz_b(r)) * 16);
  }
  unsigned char* const ring = smem + kg * (kSlots * kStage);
  const auto issue = [&](int j) {   // this group's j-th stage: 4 loads a wave
    const int kt = first + kg + 4 * j;
    const uint32_t to = lds_addr(ring + (j % kSlots) * kStage);
    dma_b128(rs, to + w * 1024, off_s + kt * st_s);
    dma_b128(rb, to + 4096 + (2 * w) * 1024, off_b[0] + kt * 128);
    dma_b128(rb, to + 4096 + (2 * w + 1) * 1024, off_b[1] + kt * 128);
    // both pairs of waves load the 512 bytes of meta: the waits count alike
    dma_b32(rm, to + 12288 + (w & 1) * 256, off_m + kt * st_m);
  };
  int rd_s[2], rd_b[2][2];
#pragma unroll
  for (int st = 0; st < 2; ++st) {
    rd_s[st] = (wm * 32 + l32) * 64 + (((2 * st + g) ^ swz_s(l32)) * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) rd_b[st][i] = 4096 + (wn * 32 + l32) * 128 + (((4 * st + 2 * i + g) ^ swz_b(l32)) * 16);
  }
  const int rd_m = 12288 + (wm * 32 + l32) * 8;
  f16v acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;

  // Stage j is issued two rounds ahead, into the slot that round j - 3 read: every
  // wave is past the barrier of round j - 2 then, before which it has waited for
  // the reads of round j - 3.
  if (mine > 0) issue(0);
  if (mine > 1) issue(1);
  for (int j = 0; j < rounds; ++j) {
    // stage j has landed (the next one's 4 loads may be under way; vmcnt in bits
    // 3:0), and this wave's LDS reads of round j - 1 are complete, whose slot the
    // waves past the barrier overwrite (lgkmcnt, bits 11:8, 0); expcnt 7: no wait
    if (j + 1 < mine) __builtin_amdgcn_s_waitcnt(4 | (7 << 4) | (0 << 8));
    else __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (0 << 8));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (j >= mine) continue;
    if (j + 2 < mine) issue(j + 2);
    const unsigned char* const from = ring + (j % kSlots) * kStage;
    const uint2 mw = *reinterpret_cast<const uint2*>(from + rd_m);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const h8 a = *reinterpret_cast<const h8*>(from + rd_s[st]);
      const h8 lo = *reinterpret_cast<const h8*>(from + rd_b[st][0]);
      const h8 hi = *reinterpret_cast<const h8*>(from + rd_b[st][1]);
      const h16 b = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
      const uint32_t word = st ? mw.y : mw.x;
      acc = __builtin_amdgcn_smfmac_f32_32x32x32_f16(a, b, acc, (int)(g ? word >> 16 : word), 0, 0);
    }
  }
  if constexpr (kTail) {
    if (kg == 0 && part + 1 == parts) {
      // the last 16, 32 or 48 of the reduction, as in the tiles above
      const int64_t k0 = K / 64 * 64;
      const int left = (int)(K - k0);
      const int64_t row = min<int64_t>(wm * 32 + l32, h - 1), token = min<int64_t>(wn * 32 + l32, tokens - 1);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int c = 2 * st + g;
        h8 a = {}, lo = {}, hi = {};
        int idx = 0;
        if (16 * c < left) {
          a = *reinterpret_cast<const h8*>(vals + m0 * (K / 2) + k0 / 2 * h + row * (left / 2) + 8 * c);
          idx = meta[m0 * (K / 16) + k0 / 16 * h + row * (left / 16) + c];
        }
        const uint16_t* const x = A + (t0 + token) * K + k0 + 32 * st + 8 * g;
        if (32 * st + 8 * g < left) lo = *reinterpret_cast<const h8*>(x);
        if (32 * st + 16 + 8 * g < left) hi = *reinterpret_cast<const h8*>(x + 16);
        const h16 b = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
        acc = __builtin_amdgcn_smfmac_f32_32x32x32_f16(a, b, acc, idx, 0, 0);
      }
    }
  }
  __syncthreads();   // no wave reads the rings any more
  // sums of the groups, [4][64 tokens][16 chunks of 4 features, XOR-swizzled]
#pragma unroll
  for (int i4 = 0; i4 < 4; ++i4) {
    const int t = wn * 32 + l32, c = wm * 8 + 2 * i4 + g;
    *reinterpret_cast<float4v*>(smem + kg * 16384 + t * 256 + ((c ^ (t & 15)) * 16)) =
        float4v{acc[4 * i4], acc[4 * i4 + 1], acc[4 * i4 + 2], acc[4 * i4 + 3]};
  }
  __syncthreads();
  const int t = threadIdx.x >> 4, quad = threadIdx.x & 15;
  const int64_t f = m0 + 4 * quad;
  const bool real = t < tokens && f < N;
  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (real) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4v p = *reinterpret_cast<const float4v*>(smem + k * 16384 + t * 256 + ((quad ^ (t & 15)) * 16));
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] += p[e];
    }
    const int64_t at = (t0 + t) * N + f;
    if constexpr (kMode == kPartial)
      *reinterpret_cast<float4v*>(fin.sums + part * T * N + at) = float4v{d[0], d[1], d[2], d[3]};
    else
      finish4<kMode == kBackward>(fin, at, f, d);
  }
  if constexpr (kMode == kBackward) {
    if (fin.sums == nullptr) return;   // the same in all lanes
    float* const all = reinterpret_cast<float*>(smem + 65536);   // [16 waves][64]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d[e] += __shfl_xor(d[e], 16);
      d[e] += __shfl_xor(d[e], 32);
    }
    if (lane < 16) *reinterpret_cast<float4v*>(all + wave * 64 + 4 * quad) = float4v{d[0], d[1], d[2], d[3]};
    __syncthreads();
    if (threadIdx.x < 64 && m0 + (int)threadIdx.x < N) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v += all[k * 64 + threadIdx.x];
      fin.sums[(int64_t)tn * N + m0 + threadIdx.x] = v;
    }
  }
}

template <int kMode>
hipError_t launch_mid(const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N, int64_t K,
                      const Finish& f, int parts, hipStream_t s) {
  const int tiles_m = (int)((N + 63) / 64), tiles_n = (int)((T + 63) / 64);
  const dim3 grid((unsigned)((tiles_m * tiles_n * parts + 7) / 8 * 8)), block(1024);
  if (K % 64 == 0)
    hipLaunchKernelGGL((spmm_mid_kernel<kMode, false>), grid, block, 0, s, A, vals, meta, T, N, K, f, tiles_m, tiles_n, parts);
  else
    hipLaunchKernelGGL((spmm_mid_kernel<kMode, true>), grid, block, 0, s, A, vals, meta, T, N, K, f, tiles_m, tiles_n, parts);
  return hipGetLastError();
}

// Joins the parts of a product's sums, part[parts][T][N], in order, and finishes
// them: a workgroup has 16 tokens x 64 features, a lane 4 features of a token.
constexpr int kJoinTokens = 16;
template <bool kBwd>
__global__ __launch_bounds__(256) void join_parts_kernel(const float* __restrict__ part, int parts, int64_t T, int64_t N,
                                                         Finish fin) {
  __shared__ float4v col[16][16];
  const int quad = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t f = (int64_t)blockIdx.x * 64 + 4 * quad, t = (int64_t)blockIdx.y * kJoinTokens + row;
  const bool real = t < T && f < N;
  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (real) {
    const int64_t at = t * N + f;
    for (int p = 0; p < parts; p += 8) {
      float4v x[8];   // eight parts under way at once
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p + k < parts) x[k] = *reinterpret_cast<const float4v*>(part + (p + k) * T * N + at);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p + k < parts)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] += x[k][e];
    }
    finish4<kBwd>(fin, at, f, d);
  }
  if constexpr (kBwd) {
    if (fin.sums == nullptr) return;   // the same in all lanes
    col[row][quad] = real ? float4v{d[0], d[1], d[2], d[3]} : float4v{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    if (row != 0 || f >= N) return;
    float4v v = col[0][quad];
#pragma unroll
    for (int r = 1; r < 16; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += col[r][quad][e];
    *reinterpret_cast<float4v*>(fin.sums + blockIdx.y * N + f) = v;
  }
}

// How a product is run, by its sizes alone: the order of its sums does not depend
// on the device.  Where the choices change places (us in kernels; weights as
// features x reduction):
//   thin up to 16 tokens: 4096 x 1024 at 16 tokens 3.8, mid 6.2; 6400 x 1600 6.1 and
//     7.5; 1024 x 4096 7.1 and 7.6.  The longest reductions change places earlier
//     (1600 x 6400 at 8 tokens 7.8 and 8.6, at 12 8.8 and 8.6, at 16 9.8 and 8.7): one
//     border for all of them costs those 12% at most.  Up to 32 where the reduction is
//     short: 4096 x 1024 at 24 4.4 and 6.2, at 32 4.7 and 6.3, but 6400 x 1600 at 24 8.1
//     and 7.6.
//   mid while there is a tile a CU at most: 1024 x 4096 at 1024 tokens (256 tiles) 15.7,
//     pairs 24.7; 6400 x 1600 at 192 (300 tiles) 15.3 and 13.6.
//   parts of a reduction: 1600 x 6400 at 24 tokens 17.1 in one part, 9.0 in 10.
//   pairs while there is a tile a CU at most: 1024 x 4096 at 2048 tokens (128 tiles)
//     25.6, small 30.7; 6400 x 1600 at 768 (300 tiles) 28.0 and 24.8.
//   small while 256 x 128 tiles are fewer than the CUs: 1600 x 6400 at 4096 tokens
//     (224) 75.9, large 79.4; 6400 x 1600 at 1500 (300) 38.9 and 34.4.
struct Plan {
  enum { kThin, kMid, kPairs, kSmall, kLarge } how;
  int parts;       // of kMid
  int64_t block;   // tokens of one row of a backward's partial sums
  int64_t rows(int64_t T) const { return (T + block - 1) / block; }
  int64_t part_floats(int64_t T, int64_t N) const { return parts > 1 ? parts * T * N : 0; }
};

Plan plan_product(int64_t T, int64_t N, int64_t K) {
  const auto tiles = [&](int64_t features, int64_t tokens) {
    return ((T + tokens - 1) / tokens) * ((N + features - 1) / features);
  };
  // the tiles' 32-bit offsets reach 256 rows of A and all of S, and a launch
  // counts its work-items in 32 bits
  constexpr int64_t kMaxBuf = (int64_t)1 << 31;
  const bool fits = K >= 64 && K * 512 < kMaxBuf && N * K < kMaxBuf && tiles(64, 64) < ((int64_t)1 << 22);
  if (!fits || T <= 16 || (T <= 32 && K <= 1024)) return {Plan::kThin, 1, T <= 16 ? 16 : T <= 32 ? 32 : kThinTokens};
  if (tiles(64, 64) <= kCus) {
    const int64_t rounds = (K / 64 + 3) / 4, parts = std::min(kCus / tiles(64, 64), rounds / 2);
    // the joining launch costs about 3 us, a round 0.47
    if (parts > 1 && rounds - (rounds + parts - 1) / parts >= 7) return {Plan::kMid, (int)parts, kJoinTokens};
    return {Plan::kMid, 1, 64};
  }
  if (tiles(128, 128) <= kCus && K >= 128) return {Plan::kPairs, 1, 128};
  return {tiles(256, 128) < kCus ? Plan::kSmall : Plan::kLarge, 1, 128};
}

template <bool kBwd>
hipError_t launch_product(const Plan& p, const uint16_t* A, const uint16_t* vals, const uint16_t* meta, int64_t T,
                          int64_t N, int64_t K, const Finish& fin, float* ws, hipStream_t s) {
  switch (p.how) {
    case Plan::kThin: return launch_thin<kBwd>(A, vals, meta, T, N, K, fin, s);
    case Plan::kPairs: return launch_small<2, kBwd>(A, vals, meta, T, N, K, fin, s);
    case Plan::kSmall: return launch_small<1, kBwd>(A, vals, meta, T, N, K, fin, s);
    case Plan::kLarge: return launch_large<kBwd>(A, vals, meta, T, N, K, fin, s);
    case Plan::kMid: break;
  }
  if (p.parts == 1) return launch_mid<kBwd ? kBackward : kForward>(A, vals, meta, T, N, K, fin, 1, s);
  Finish part{};
  part.sums = ws;
  const hipError_t e = launch_mid<kPartial>(A, vals, meta, T, N, K, part, p.parts, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(join_parts_kernel<kBwd>, dim3((unsigned)((N + 63) / 64), (unsigned)p.rows(T)), dim3(256), 0, s, ws,
                     p.parts, T, N, fin);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Sums over rows.

// out[c] = the sum of part[P][N]'s rows.  Eight waves take every eighth row, eight
// rows at a time, of 64 columns, and their sums are added in order.
__global__ __launch_bounds__(512) void join_rows_kernel(const float* __restrict__ part, int64_t P, int64_t N,
                                                        float* __restrict__ out) {
  __shared__ float waves[8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
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

hipError_t launch_join_rows(const float* part, int64_t P, int64_t N, float* out, hipStream_t s) {
  hipLaunchKernelGGL(join_rows_kernel, dim3((unsigned)((N + 63) / 64)), dim3(512), 0, s, part, P, N, out);
  return hipGetLastError();
}

// Sums of dY's columns over all rows, for few rows: a workgroup has 64 columns, a
// wave 8 rows at a time of a workgroup's 128, four times over.
__global__ __launch_bounds__(1024) void column_sums_kernel(const uint16_t* __restrict__ dY, int64_t T, int64_t R,
                                                           float* __restrict__ out) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + (lane & 7) * 8;
  float v[8] = {};
  if (c < R)
    for (int64_t t = wave * 8 + (lane >> 3); t < T; t += 512) {
      h8 x[4];   // four rows under way at once
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = t + 128 * k < T ? *reinterpret_cast<const h8*>(dY + (t + 128 * k) * R + c) : h8{};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += (float)x[k][e];
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int x = 8; x < 64; x *= 2) v[e] += __shfl_xor(v[e], x);
    if (lane < 8) part[wave][lane * 8 + e] = v[e];
  }
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || col >= R) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) sum += part[w][threadIdx.x];
  out[col] = sum;
}

// The same over a chunk of rows: a lane takes 8 columns, the four waves of a
// workgroup every fourth row.  210 MB (16384 x 6400) in 43 us with the joining of
// the chunks, 4.9 TB/s, what a copy reaches.
__global__ __launch_bounds__(256) void chunk_sums_kernel(const uint16_t* __restrict__ dY, int64_t T, int64_t R,
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

// Chunks of rows: of 64 rows or more, about 2048 workgroups at most.  One launch
// over all rows where a workgroup's 64 columns are 128 KB at most (517 x 1600: 8 us
// a call instead of 12, most of either the launches).
int64_t sum_chunks(int64_t T, int64_t R) {
  if (T <= 1024) return 1;
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
  if (P == 1) {
    hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)((R + 63) / 64)), dim3(1024), 0, s, dY, T, R, out);
    return hipGetLastError();
  }
  float* const part = static_cast<float*>(ws);
  hipLaunchKernelGGL(chunk_sums_kernel, dim3((unsigned)((R + 511) / 512), (unsigned)P), dim3(256), 0, s, dY, T, R, rows, part);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_join_rows(part, P, R, out, s);
}

int64_t spmm_act_fwd_workspace(int64_t T, int64_t N, int64_t K) {
  return T == 0 || N == 0 ? 0 : 4 * plan_product(T, N, K).part_floats(T, N);
}

hipError_t launch_spmm_act_fwd(const uint16_t* X, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N,
                               int64_t K, const float* bias, int act, const uint16_t* residual, uint16_t* U,
                               uint16_t* Y, void* ws, hipStream_t s) {
  if (T == 0 || N == 0) return hipSuccess;
  const Finish fin{bias, residual, nullptr, U, Y, nullptr, act};
  return launch_product<false>(plan_product(T, N, K), X, vals, meta, T, N, K, fin, static_cast<float*>(ws), s);
}

int64_t spmm_act_bwd_workspace(int64_t T, int64_t N, int64_t K, bool sums) {
  if (T == 0 || N == 0) return 0;
  const Plan p = plan_product(T, N, K);
  return 4 * (p.part_floats(T, N) + (sums && p.rows(T) > 1 ? p.rows(T) * N : 0));
}

hipError_t launch_spmm_act_bwd(const uint16_t* dY, const uint16_t* vals, const uint16_t* meta, int64_t T, int64_t N,
                               int64_t K, int act, const uint16_t* U, uint16_t* dU, float* dbias, void* ws,
                               hipStream_t s) {
  if (N == 0) return hipSuccess;
  if (T == 0) return dbias ? launch_bias_grad(nullptr, 0, N, dbias, nullptr, s) : hipSuccess;
  const Plan p = plan_product(T, N, K);
  float* const parts = static_cast<float*>(ws);
  float* const sums = dbias == nullptr ? nullptr : p.rows(T) > 1 ? parts + p.part_floats(T, N) : dbias;
  const Finish fin{nullptr, nullptr, act == kActNone ? nullptr : U, nullptr, dU, sums, act};
  const hipError_t e = launch_product<true>(p, dY, vals, meta, T, N, K, fin, parts, s);
  if (e != hipSuccess || sums == nullptr || p.rows(T) == 1) return e;
  return launch_join_rows(sums, p.rows(T), N, dbias, s);
}

}  // namespace sp24
