// Orthogonalising weight updates by Newton-Schulz products, and the optimiser
// step built on it, for gfx950 matrix cores.
//
// With U the update of a weight (its gradient, or the momentum of its
// gradients), m its short side and n its long one, X [m][n] holding U or U^T:
//
//   X_0 = U / (|U|_F + eps)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X        (each step's own a, b, c)
//
// Every step maps X's singular values by s -> a s + b s^3 + c s^5 and leaves
// its singular vectors alone.  The result goes out, or steps the weight:
// P <- keep P - lr X, W = fp16(P).
//
// Number formats.  X, A and B are held as fp16 in units of 2^-12.  The
// entries of X are about (m n)^-1/2 at the start (3e-4 for a 1600 x 6400
// weight), where fp16 itself has few or no bits left; in these units values
// up to 16 fit and the typical ones keep all 11 bits.  Beside the rounded
// part hi, X keeps the rest lo = fp16(x - hi), 22 bits together.  Products are
// accumulated in fp32 in either mode:
//   rounded   products of the hi parts.  X's lo part still enters a X in the
//             first kLoSteps steps: there the small singular values grow 3.4
//             times a step, and with them the rounding error of X, which
//             without the lo part costs up to 6e-3 of the result's norm on a
//             low-rank update.  Results are within about 2e-3 of exact
//             arithmetic (bf16 operands: 1e-2 to 5e-2).
//   split     hi hi + hi lo + lo hi, for results to fp32 accuracy.
//
// A and B are symmetric: only tiles on and above the diagonal are computed,
// each stored twice.
//
// v_mfma_f32_32x32x16_f16 operands (lane l, g = l / 32):
//   A: row l % 32, k in [8g, 8g + 8)     B: column l % 32, the same k
//   D: column l % 32, rows 8*(i/4) + 4g + i%4 for accumulator i
#include <hip/hip_runtime.h>
#include <cstdint>

#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kThreads = 256;
constexpr float kScale = 4096.0f, kInvScale = 1.0f / 4096.0f;   // the units of X, A and B
constexpr int kLoSteps = 3;
constexpr int kNormChunk = 16 * kThreads;   // entries a workgroup squares at a time
constexpr int kMaxParts = 1024;             // partial sums of squares per weight
constexpr int kTile = 128;         // square tiles of the products
constexpr int kBK = 32;            // reduction per stage

// One weight, as the kernels see it.
struct Job {
  const void* G;
  float* M;
  void* out;
  float* P;
  uint16_t* W;
  float lr, keep;
  int m, n;        // short and long side
  int lda, ldx;    // row lengths of A, B and of X, multiples of 64
  bool tall;       // X is U^T
  bool g32, out32;
  double* sums;                  // of squares, `parts` of them
  int parts;
  _Float16* x[2];                // X, hi then lo part, before and after a step
  _Float16 *A, *B;               // hi then lo part
  int first;                     // first workgroup of the launch at hand
};
struct Jobs {
  Job j[kMaxNsJobs];
  int count;
};

__device__ __forceinline__ const Job& job_of(const Jobs& jobs, int block) {
  int k = 0;
  while (k + 1 < jobs.count && block >= jobs.j[k + 1].first) ++k;
  return jobs.j[k];
}

__device__ __forceinline__ float load_g(const Job& j, int64_t i) {
  return j.g32 ? static_cast<const float*>(j.G)[i] : (float)static_cast<const _Float16*>(j.G)[i];
}

// Entries i .. i + 7 of a matrix of `total`; zeros past its end.  i is a
// multiple of 8 and matrices start 16-byte aligned.
__device__ __forceinline__ void load8(const void* p, bool is32, int64_t i, int64_t total, float (&v)[8]) {
  if (i + 8 <= total) {
    if (is32) {
      const f4* q = reinterpret_cast<const f4*>(static_cast<const float*>(p) + i);
      const f4 x = q[0], y = q[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = x[e];
        v[4 + e] = y[e];
      }
    } else {
      const h8 x = *reinterpret_cast<const h8*>(static_cast<const _Float16*>(p) + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = i + e >= total ? 0.0f : is32 ? static_cast<const float*>(p)[i + e] : (float)static_cast<const _Float16*>(p)[i + e];
  }
}
__device__ __forceinline__ void store8(float* p, int64_t i, int64_t total, const float (&v)[8]) {
  if (i + 8 <= total) {
    f4* q = reinterpret_cast<f4*>(p + i);
    q[0] = f4{v[0], v[1], v[2], v[3]};
    q[1] = f4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < total) p[i + e] = v[e];
  }
}

// The update of entry i from its gradient and its new momentum.
__device__ __forceinline__ float update_of(const Job& j, int64_t i, float mu, bool nesterov) {
  if (j.M == nullptr) return load_g(j, i);
  const float m = j.M[i];
  return nesterov ? load_g(j, i) + mu * m : m;
}

// Sum over the workgroup, in every thread; a fixed order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += s[w];
  return v;
}

// Momentum, and the squares of the update summed in 64 bits (a sum of fp32
// squares would lose updates below 1e-22 or above 1e19).  Eight entries a
// thread at a time; a workgroup takes kNormChunk of them.
__global__ __launch_bounds__(kThreads) void ns_norm_kernel(Jobs jobs, float mu, bool nesterov) {
  const Job& j = job_of(jobs, blockIdx.x);
  const int block = blockIdx.x - j.first;
  const int64_t total = (int64_t)j.m * j.n;
  double sum = 0.0;
  for (int64_t base = (int64_t)block * kNormChunk; base < total; base += (int64_t)j.parts * kNormChunk) {
    float u[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t i = base + (q * kThreads + threadIdx.x) * 8;
      load8(j.G, j.g32, i, total, u[q]);
      if (j.M != nullptr) {
        float m[8];
        load8(j.M, true, i, total, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m[e] = mu * m[e] + u[q][e];
          u[q][e] = nesterov ? u[q][e] + mu * m[e] : m[e];
        }
        store8(j.M, i, total, m);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += (double)u[q][e] * (double)u[q][e];
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) j.sums[block] = sum;
}

// x in two fp16 parts
__device__ __forceinline__ void split(float x, _Float16& hi, _Float16& lo) {
  hi = (_Float16)x;
  lo = (_Float16)(x - (float)hi);
}

// X_0 in both parts, a 64 x 64 tile of it a workgroup; the columns from n to
// ldx are zeros.
__global__ __launch_bounds__(kThreads) void ns_start_kernel(Jobs jobs, float mu, bool nesterov, float eps) {
  __shared__ float tile[64][65];
  const Job& j = job_of(jobs, blockIdx.x);
  const int block = blockIdx.x - j.first, tiles_n = j.ldx / 64;
  const int i0 = block / tiles_n * 64, j0 = block % tiles_n * 64;
  double sum = 0.0;
  for (int k = threadIdx.x; k < j.parts; k += kThreads) sum += j.sums[k];
  const double norm = sqrt(block_sum(sum));
  const double scale = (double)kScale / (norm + (double)eps);
  const int64_t plane = (int64_t)j.m * j.ldx;
  if (j.tall) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int k = e * kThreads + threadIdx.x, r = j0 + k / 64, c = i0 + k % 64;   // of U [n][m]
      tile[k / 64][k % 64] = r < j.n && c < j.m ? update_of(j, (int64_t)r * j.m + c, mu, nesterov) : 0.0f;
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int k = e * kThreads + threadIdx.x, r = i0 + k / 64, c = j0 + k % 64;
    if (r >= j.m) continue;
    float u;
    if (j.tall)
      u = tile[k % 64][k / 64];
    else
      u = c < j.n ? update_of(j, (int64_t)r * j.n + c, mu, nesterov) : 0.0f;
    _Float16 hi, lo;
    split((float)((double)u * scale), hi, lo);
    j.x[0][(int64_t)r * j.ldx + c] = hi;
    j.x[0][plane + (int64_t)r * j.ldx + c] = lo;
  }
}

// vmcnt wait (expcnt and lgkmcnt not waited for)
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// What one lane of a wave has written to LDS is read by the others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Eight values in their fp16 parts; 16-byte aligned.
__device__ __forceinline__ void put8(_Float16* p, int64_t plane, bool both, const float (&v)[8]) {
  h8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    _Float16 h, l;
    split(v[e], h, l);
    hi[e] = h;
    lo[e] = l;
  }
  *reinterpret_cast<h8*>(p) = hi;
  if (both) *reinterpret_cast<h8*>(p + plane) = lo;
}

// Entries at .. at + 7 of a result's row of n, which starts at entry `row`:
// the orthogonalised update, or the weight's step by it.
__device__ __forceinline__ void finish8(const Job& j, int64_t row, int at, int n, const float (&v)[8]) {
  const bool whole = at + 8 <= n && n % 8 == 0;   // rows start 16-byte aligned
  const int64_t o = row + at;
  if (j.P != nullptr) {
    float p[8];
    if (whole) {
      load8(j.P, true, o, o + 8, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = j.keep * p[e] - j.lr * v[e];
      store8(j.P, o, o + 8, p);
      if (j.W != nullptr) {
        h8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (_Float16)p[e];
        *reinterpret_cast<h8*>(j.W + o) = h;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = at + e < n ? j.P[o + e] : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (at + e >= n) continue;
        p[e] = j.keep * p[e] - j.lr * v[e];
        j.P[o + e] = p[e];
        if (j.W != nullptr) j.W[o + e] = __builtin_bit_cast(uint16_t, (_Float16)p[e]);
      }
    }
    return;
  }
  if (j.out32) {
    float* out = static_cast<float*>(j.out);
    if (whole) {
      store8(out, o, o + 8, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) out[o + e] = v[e];
    }
  } else {
    _Float16* out = static_cast<_Float16*>(j.out);
    if (whole) {
      h8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[e];
      *reinterpret_cast<h8*>(out + o) = h;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at + e < n) out[o + e] = (_Float16)v[e];
    }
  }
}

enum : int { kGram = 0, kPoly = 1, kApply = 2 };

// The products' LDS stage: kTile rows x kBK of the left operand, then the
// right operand: kTile rows x kBK (kGram, kPoly: both are rows along the
// reduction), or kBK rows x kTile columns of X (kApply).  Rows of kBK halves
// are four 16-byte chunks; chunk c of row r is stored at c ^ (r / 4 % 4), so
// that the 16 rows a fragment read serves at a time cover all banks once.
// Rows of kTile columns are read by transpose reads; their chunk q is at
// (q + 12 (r % 4)) % 16, which puts the eight 32-byte windows that a read
// fetches from four rows in different banks.
constexpr int kOperand = kTile * kBK * 2;   // bytes of one operand's part
constexpr int kRing = 3;
constexpr int kTurn = 68;   // floats in a row of the epilogue's 32 x 64 blocks
static_assert(4 * 32 * kTurn * 4 <= kRing * 2 * kOperand, "the epilogue's blocks fit the ring");

template <int KIND, bool SPLIT, bool LAST>
__global__ __launch_bounds__(kThreads) void ns_product_kernel(Jobs jobs, int cur, float a, float b, float c, bool use_lo) {
  constexpr int PARTS = SPLIT ? 2 : 1;
  constexpr int STAGE = 2 * PARTS * kOperand;
  constexpr int LOADS = kOperand / 1024 / 4;   // direct loads per wave, operand and part
  __shared__ __align__(1024) unsigned char smem[kRing * STAGE];
  const Job& j = job_of(jobs, blockIdx.x);
  int block = blockIdx.x - j.first;
  const int tiles_m = (j.m + kTile - 1) / kTile;
  int tm, tn;
  if constexpr (KIND == kApply) {
    // workgroups go round the 8 XCDs: each takes a run of column strips, whose
    // X its L2 then fetches once
    const int tiles = tiles_m * ((j.n + kTile - 1) / kTile), run = (tiles + 7) / 8;
    const int lin = block % 8 * run + block / 8;
    if (block / 8 >= run || lin >= tiles) return;
    tm = lin % tiles_m;
    tn = lin / tiles_m;
  } else {
    // row tm of the upper triangle holds tiles_m - tm tiles
    tm = 0;
    while (block >= tiles_m - tm) block -= tiles_m - tm++;
    tn = tm + block;
  }
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int m0 = tm * kTile, n0 = tn * kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int g = lane >> 5, l32 = lane & 31;

  const int64_t xplane = (int64_t)j.m * j.ldx, aplane = (int64_t)j.m * j.lda;
  const _Float16* const X = j.x[cur];
  const _Float16* const left = KIND == kGram ? X : KIND == kPoly ? j.A : j.B;
  const _Float16* const right = KIND == kPoly ? j.A : X;
  const int lld = KIND == kGram ? j.ldx : j.lda, rld = KIND == kPoly ? j.lda : j.ldx;
  const int64_t lplane = KIND == kGram ? xplane : aplane, rplane = KIND == kPoly ? aplane : xplane;
  const int nk = lld / kBK;

  // Descriptors over whole parts: rows past m read as zero.  Columns of X past
  // ldx are the next row's and feed only outputs that are not stored.
  i32x4 rl[PARTS], rr[PARTS];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    rl[p] = make_rsrc(left + p * lplane, (uint32_t)(lplane * 2));
    rr[p] = make_rsrc(right + p * rplane, (uint32_t)(rplane * 2));
  }
  int goff_l[LOADS], goff_r[LOADS];
#pragma unroll
  for (int u = 0; u < LOADS; ++u) {
    const int s = (wave + 4 * u) * 64 + lane;   // 16-byte slot of the operand's part
    {
      const int row = s / 4, q = (s & 3) ^ ((row >> 2) & 3);
      goff_l[u] = (m0 + row) * lld * 2 + q * 16;
      if constexpr (KIND != kApply) goff_r[u] = (n0 + row) * rld * 2 + q * 16;
    }
    if constexpr (KIND == kApply) {
      const int row = s / 16, q = ((s & 15) + 16 - 12 * (row & 3) % 16) & 15;
      goff_r[u] = row * rld * 2 + (n0 + 8 * q) * 2;
    }
  }
  const int right_step = KIND == kApply ? kBK * rld * 2 : kBK * 2;
  auto issue = [&](int kt, int slot) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        const uint32_t dst = lds_addr(smem) + slot * STAGE + p * kOperand + 1024 * (wave + 4 * u);
        dma_b128(rl[p], dst, goff_l[u] + kt * kBK * 2);
        dma_b128(rr[p], dst + PARTS * kOperand, goff_r[u] + kt * right_step);
      }
  };

  // this lane's fragment offsets inside an operand's part, per 32-row block
  int l_off[2], r_off[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = wm * 64 + t * 32 + l32;
    l_off[t] = row * 64;
    if constexpr (KIND != kApply) {
      r_off[t] = (wn * 64 + t * 32 + l32) * 64;
    } else {
      const int G = lane >> 4, j4 = (lane & 15) >> 2, c4 = lane & 3;
      const int q = (wn * 64 + t * 32 + 16 * (G & 1)) / 8 + (c4 >> 1);
      r_off[t] = (8 * (G >> 1) + j4) * 256 + ((q + 12 * j4) & 15) * 16 + (c4 & 1) * 8;
    }
  }
  const int swz = (l32 >> 2) & 3;   // of both operands' rows: their blocks start at multiples of 32
  auto row_frag = [&](int base, int ks) -> h8 {
    return *reinterpret_cast<const h8*>(smem + base + (((2 * ks + g) ^ swz) * 16));
  };
  auto tr_frag = [&](int base, int ks) -> h8 {
    const int o = base + ks * 16 * 256;
    const h4 lo = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o)));
    const h4 hi = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o + 4 * 256)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f16v acc[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[s][t][e] = 0.0f;

  constexpr int PER_STAGE = 2 * PARTS * LOADS;   // this wave's loads
  issue(0, 0);
  if (nk > 1) issue(1, 1);
  for (int kt = 0; kt < nk; ++kt) {
    // this wave's loads of stage kt are done, then every wave's; nobody reads
    // the slot of stage kt - 1 any more, which stage kt + 2 takes
    if (kt + 1 < nk) wait_vm<PER_STAGE>(); else wait_vm<0>();
    __builtin_amdgcn_s_waitcnt(0xF | (7 << 4) | (0 << 8) | (3 << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (kt + 2 < nk) issue(kt + 2, (kt + 2) % kRing);
    const int base = (kt % kRing) * STAGE;
#pragma unroll
    for (int ks = 0; ks < kBK / 16; ++ks) {
      h8 fl[PARTS][2], fr[PARTS][2];
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          fl[p][t] = row_frag(base + p * kOperand + l_off[t], ks);
          const int rb = base + (PARTS + p) * kOperand + r_off[t];
          if constexpr (KIND == kApply)
            fr[p][t] = tr_frag(rb, ks);
          else
            fr[p][t] = row_frag(rb, ks);
        }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if constexpr (SPLIT) {
            acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fl[0][s], fr[1][t], acc[s][t], 0, 0, 0);
            acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fl[1][s], fr[0][t], acc[s][t], 0, 0, 0);
          }
          acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fl[0][s], fr[0][t], acc[s][t], 0, 0, 0);
        }
    }
    asm volatile("" ::: "memory");
  }

  // Epilogue.  A wave turns 32 rows x 64 columns of accumulators at a time
  // through its quarter of the ring, so that a lane holds 8 columns of a row:
  // what it reads and writes there is whole 16-byte pieces of 128-byte runs.
  // Results that go out transposed (the mirrored tile, a tall weight) are put
  // back and read again by columns.  The loads of a block are issued before
  // its first store.
  __syncthreads();   // the ring is idle
  float* const turn = reinterpret_cast<float*>(smem) + wave * (32 * kTurn);
  const int er = lane >> 3, ec = (lane & 7) * 8;   // row (of 8) and first column
  constexpr bool kLoads = KIND != kGram;
  const bool back = KIND == kApply ? LAST && j.tall : tm != tn;
  // what is read, and what is written: X, or A and B, of one shape
  const _Float16* const old = KIND == kApply ? X : j.A;
  _Float16* const D = KIND == kGram ? j.A : KIND == kPoly ? j.B : j.x[1 - cur];
  const int64_t plane = KIND == kApply ? xplane : aplane;
  const int ld = KIND == kApply ? j.ldx : j.lda;
  const bool old_lo = SPLIT || (KIND == kApply && use_lo);
  const int c0 = n0 + wn * 64 + ec;
  const bool col_in = c0 < ld;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int r0 = m0 + wm * 64 + s * 32;
    h8 ohi[4], olo[4];
    if constexpr (kLoads) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int row = r0 + p * 8 + er;
        ohi[p] = olo[p] = h8{};
        if (row < j.m && col_in) {
          const _Float16* at = old + (int64_t)row * ld + c0;
          ohi[p] = *reinterpret_cast<const h8*>(at);
          if (old_lo) olo[p] = *reinterpret_cast<const h8*>(at + plane);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) turn[(8 * (i >> 2) + 4 * g + (i & 3)) * kTurn + t * 32 + l32] = acc[s][t][i];
    wave_sync();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = r0 + p * 8 + er;
      float* const mine = turn + (p * 8 + er) * kTurn + ec;
      const f4 v0 = *reinterpret_cast<const f4*>(mine), v1 = *reinterpret_cast<const f4*>(mine + 4);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (e < 4 ? v0[e & 3] : v1[e & 3]) * kInvScale;
        if constexpr (kLoads) {
          const float o = (float)ohi[p][e] + (float)olo[p][e];
          v[e] = KIND == kPoly ? b * o + c * v[e] : a * o + v[e];
        }
      }
      if constexpr (KIND != kApply || !LAST) {
        if (row < j.m && col_in) put8(D + (int64_t)row * ld + c0, plane, KIND == kApply || SPLIT, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= kInvScale;
        if (!j.tall && row < j.m) finish8(j, (int64_t)row * j.n, c0, j.n, v);
      }
      if (back) {
        *reinterpret_cast<f4*>(mine) = f4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f4*>(mine + 4) = f4{v[4], v[5], v[6], v[7]};
      }
    }
    if (back) {
      wave_sync();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int cc = p * 16 + (lane >> 2), rr = (lane & 3) * 8, col = n0 + wn * 64 + cc, row = r0 + rr;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = turn[(rr + e) * kTurn + cc];
        if constexpr (KIND != kApply) {
          if (col < j.m) put8(D + (int64_t)col * ld + row, plane, SPLIT, v);
        } else if constexpr (LAST) {
          if (col < j.n) finish8(j, (int64_t)col * j.m, row, j.m, v);
        }
      }
    }
    wave_sync();   // the block has been read
  }
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Bytes of one weight's workspace; fills its pointers when base is given.
int64_t lay_out(Job& j, unsigned char* base) {
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    unsigned char* p = base ? base + at : nullptr;
    at += up(bytes, 256);
    return p;
  };
  const int64_t x = (int64_t)j.m * j.ldx * 4, a = (int64_t)j.m * j.lda * 4;   // two parts of 2 bytes
  j.sums = reinterpret_cast<double*>(take(kMaxParts * 8));
  j.x[0] = reinterpret_cast<_Float16*>(take(x));
  j.x[1] = reinterpret_cast<_Float16*>(take(x));
  j.A = reinterpret_cast<_Float16*>(take(a));
  j.B = reinterpret_cast<_Float16*>(take(a));
  return at;
}

int64_t fill(Jobs& jobs, const NsJob* in, int count, unsigned char* ws) {
  int64_t at = 0;
  jobs.count = 0;
  for (int k = 0; k < count; ++k) {
    const NsJob& s = in[k];
    if (s.R == 0 || s.C == 0) continue;
    Job& j = jobs.j[jobs.count++];
    j = Job{};
    j.G = s.G;
    j.M = s.M;
    j.out = s.out;
    j.P = s.P;
    j.W = s.W;
    j.lr = s.lr;
    j.keep = s.keep;
    j.tall = s.R > s.C;
    j.m = (int)(j.tall ? s.C : s.R);
    j.n = (int)(j.tall ? s.R : s.C);
    j.lda = (int)up(j.m, 64);
    j.ldx = (int)up(j.n, 64);
    const int64_t parts = ((int64_t)j.m * j.n + kNormChunk - 1) / kNormChunk;
    j.parts = (int)(parts < kMaxParts ? parts : kMaxParts);
    j.g32 = s.g32;
    j.out32 = s.out32;
    at += lay_out(j, ws ? ws + at : nullptr);
  }
  return at;
}

// Deals workgroups to the jobs; returns their number.
template <typename F>
unsigned deal(Jobs& jobs, F blocks) {
  int64_t at = 0;
  for (int k = 0; k < jobs.count; ++k) {
    jobs.j[k].first = (int)at;
    at += blocks(jobs.j[k]);
  }
  return (unsigned)at;
}

template <bool SPLIT>
void step(Jobs& jobs, const NsParams& prm, int k, hipStream_t s) {
  const float a = prm.coef[3 * k], b = prm.coef[3 * k + 1], c = prm.coef[3 * k + 2];
  const int cur = k & 1;
  const bool lo = k < kLoSteps;
  const unsigned square = deal(jobs, [](const Job& j) {
    const int64_t t = up(j.m, kTile) / kTile;
    return t * (t + 1) / 2;
  });
  hipLaunchKernelGGL((ns_product_kernel<kGram, SPLIT, false>), dim3(square), dim3(kThreads), 0, s, jobs, cur, a, b, c, lo);
  hipLaunchKernelGGL((ns_product_kernel<kPoly, SPLIT, false>), dim3(square), dim3(kThreads), 0, s, jobs, cur, a, b, c, lo);
  const unsigned wide = deal(jobs, [](const Job& j) { return up(up(j.m, kTile) / kTile * (up(j.n, kTile) / kTile), 8); });
  if (k + 1 < prm.steps)
    hipLaunchKernelGGL((ns_product_kernel<kApply, SPLIT, false>), dim3(wide), dim3(kThreads), 0, s, jobs, cur, a, b, c, lo);
  else
    hipLaunchKernelGGL((ns_product_kernel<kApply, SPLIT, true>), dim3(wide), dim3(kThreads), 0, s, jobs, cur, a, b, c, lo);
}

}  // namespace

int64_t ns_workspace(const NsJob* jobs, int count) {
  Jobs j{};
  return fill(j, jobs, count, nullptr);
}

hipError_t launch_newton_schulz(const NsJob* in, int count, const NsParams& prm, void* ws, hipStream_t s) {
  Jobs jobs{};
  fill(jobs, in, count, static_cast<unsigned char*>(ws));
  if (jobs.count == 0) return hipSuccess;
  const unsigned norm = deal(jobs, [](const Job& j) { return (int64_t)j.parts; });
  hipLaunchKernelGGL(ns_norm_kernel, dim3(norm), dim3(kThreads), 0, s, jobs, prm.mu, prm.nesterov);
  const unsigned start = deal(jobs, [](const Job& j) { return up(j.m, 64) / 64 * (int64_t)(j.ldx / 64); });
  hipLaunchKernelGGL(ns_start_kernel, dim3(start), dim3(kThreads), 0, s, jobs, prm.mu, prm.nesterov, prm.eps);
  for (int k = 0; k < prm.steps; ++k) {
    if (prm.split)
      step<true>(jobs, prm, k, s);
    else
      step<false>(jobs, prm, k, s);
  }
  return hipGetLastError();
}

}  // namespace sp24
