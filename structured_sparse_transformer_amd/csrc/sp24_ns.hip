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
// below 16 fit and the typical ones keep all 11 bits.  Beside the rounded
// part hi, X keeps the rest lo = fp16(x - hi), 22 bits together; values below
// 2^-36 are lost.  Products are accumulated in fp32 in either mode:
//   split     hi hi + hi lo + lo hi, for results to fp32 accuracy.  B has a I
//             in it (Q = a I + B, X <- Q X), so that the last product of a step
//             reads X once.
//   rounded   products of the hi parts, when the caller asks for them: a third
//             of the matrix work.  Every step takes a X in the epilogue, from
//             both parts.  A step multiplies what X has in directions that the
//             update lacks by a (3.4): X's rounding to 11 bits would be 1.4e-2
//             of a rank-one result after five steps and 0.36 after eight, that
//             to 22 bits is 1e-4 and 3e-3, in either mode and as in fp32.  The
//             roundings of A and B and of X inside the products do not grow
//             so: what they change of B X has the update's rows or its columns,
//             and no new direction of both.  Where singular values are nearly
//             equal B is nearly a multiple of I, and its diagonal's roundings
//             are all the same one: that part of them is taken along, row by
//             row, with a X (2.9e-3 without it in five steps of equal values of
//             a 300 x 900 weight).  The rest costs up to 6e-4 of the norm a
//             step where the short side is 128 or more (largest of an emulation
//             over spectra from one value to all equal: 5.3e-4), and up to
//             3e-3 where few roundings average out: small weights, and entries
//             that are all alike or mostly zero.
//
// A and B are symmetric: only tiles on and above the diagonal are computed,
// each stored twice.
//
// What bounds it.  A step costs m^2 n (A) + m^3 (A^2) + 2 m^2 n (BX) flops, in
// two parts three times that: 266 GFLOP for five steps of a 1600 x 6400 weight,
// 192 us (in two parts 574) at the 1.39 PFLOP/s that a large fp16 library
// product reaches here.  Medians of the kernels at that size over several cards,
// in us, with the rate in PFLOP/s and the share of cycles in which the matrix
// units are busy:
//                   two parts                        fp16 operands
//   B X             113 - 119      0.82 - 0.87  0.41   46 - 47       0.70 - 0.71  0.33
//   B X of two      189 - 198      0.99 - 1.04  0.53   82 - 86       0.77 - 0.80  0.35
//   A and its join  58 - 60 + 9    0.71 - 0.73  0.43   25 + 8        0.50         0.29
//   A^2             25 - 26        0.48         0.19   15            0.27         0.09
// The matrix instructions alone, without loads or LDS reads, run at 1.56
// PFLOP/s, the clock down to 1.8 GHz.  What keeps the products from that: the
// latency of a stage's LDS reads and its barrier, with 24 MFMAs a wave between
// two of them (12 in A^2; of fp16 operands 8 and 4) and in two parts one
// workgroup a CU; few tiles (650 of one weight's B X, 181 of A^2, on 256 CUs);
// and at the ends, where all tiles come together, the traffic of X's parts and
// in the last step of P and W.
//
// v_mfma_f32_32x32x16_f16 operands (lane l, g = l / 32):
//   A: row l % 32, k in [8g, 8g + 8)     B: column l % 32, the same k
//   D: column l % 32, rows 8*(i/4) + 4g + i%4 for accumulator i
#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kThreads = 256;
constexpr float kScale = 4096.0f, kInvScale = 1.0f / 4096.0f;   // the units of X, A and B
constexpr int kNormChunk = 16 * kThreads;   // entries a workgroup squares at a time
constexpr int kMaxParts = 1024;             // partial sums of squares per weight
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
  int na, nx;      // blocks of 32 along them: A and B are na x na blocks, X na x nx
  bool tall;       // X is U^T
  bool g32, out32;
  double* sums;                  // of squares, `parts` of them
  int parts;
  _Float16* x[2];                // X, hi then lo part, before and after a step
  _Float16 *A, *B;               // hi then lo part
  int gram_splits;               // items that share the reduction of a tile of A
  float* partial;                // their sums
  int first;                     // first workgroup of the launch at hand
};
struct Jobs {
  Job j[kMaxNsJobs];
  int count;
  bool fine;   // few tiles: small ones throughout
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

__device__ __forceinline__ void update8(const Job& j, int64_t i, float mu, bool nesterov, float (&u)[8]) {
  load8(j.G, j.g32, i, i + 8, u);
  if (j.M == nullptr) return;
  float m[8];
  load8(j.M, true, i, i + 8, m);
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = nesterov ? u[e] + mu * m[e] : m[e];
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
// thread at a time; a workgroup takes kNormChunk of them.  Memory-bound: 46 to 49
// us (4.2 to 4.4 TB/s) for the momentum of 6400 x 1600 and 1600 x 6400, 9 us for
// the norm of one.
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

// X, A and B are stored in blocks of 32 x 32, row-major among themselves and
// within: element (r, c) of a matrix of nb blocks a row.  A stage of a product
// reads whole blocks (2 KiB), whichever side of the reduction its rows are on;
// row-major matrices would give it half cache lines.
__device__ __forceinline__ int64_t at_block(int r, int c, int nb) {
  return ((int64_t)(r >> 5) * nb + (c >> 5)) * 1024 + (r & 31) * 32 + (c & 31);
}

// x in two fp16 parts
__device__ __forceinline__ void split(float x, _Float16& hi, _Float16& lo) {
  hi = (_Float16)x;
  lo = (_Float16)(x - (float)hi);
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

// X_0 in both parts, 32 x 64 of it a workgroup (two blocks side by side);
// zeros past m and n.  Memory-bound: 48 to 51 us (3.9 to 4.3 TB/s) for those two
// weights, 19 for the one; a pass of its own because it needs the norm of all of
// U.
__global__ __launch_bounds__(kThreads) void ns_start_kernel(Jobs jobs, float mu, bool nesterov, float eps) {
  __shared__ float tile[64][33];
  const Job& j = job_of(jobs, blockIdx.x);
  const int block = blockIdx.x - j.first, tiles_n = (j.nx + 1) / 2;
  const int i0 = block / tiles_n * 32, j0 = block % tiles_n * 64;
  const int tid = threadIdx.x;
  // this thread's eight entries of a row of X
  const int r = tid >> 3, c = (tid & 7) * 8;
  float u[8];
  if (!j.tall) {
    // of a row of U
    const int row = i0 + r, col = j0 + c;
    const int64_t i = (int64_t)row * j.n + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = 0.0f;
    if (row < j.m) {
      if (j.n % 8 == 0) {
        if (col < j.n) update8(j, i, mu, nesterov, u);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < j.n) u[e] = update_of(j, i + e, mu, nesterov);
      }
    }
  } else {
    // U [n][m]: 64 rows of 32, turned in LDS
    const int row = j0 + (tid >> 2), col = i0 + (tid & 3) * 8;
    const int64_t i = (int64_t)row * j.m + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = 0.0f;
    if (row < j.n) {
      if (j.m % 8 == 0) {
        if (col < j.m) update8(j, i, mu, nesterov, u);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < j.m) u[e] = update_of(j, i + e, mu, nesterov);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[tid >> 2][(tid & 3) * 8 + e] = u[e];
  }
  double sum = 0.0;
  for (int k = tid; k < j.parts; k += kThreads) sum += j.sums[k];
  const double norm = sqrt(block_sum(sum));   // its barrier also orders the turn
  const double scale = (double)kScale / (norm + (double)eps);
  if (j.tall) {
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = tile[c + e][r];
  }
  if ((j0 >> 5) + (c >> 5) >= j.nx) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = (float)((double)u[e] * scale);
  put8(j.x[0] + at_block(i0 + r, j0 + c, j.nx), (int64_t)j.na * j.nx * 1024, true, u);
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

enum : int { kGram = 0, kPoly = 1, kApply = 2 };

// A product's tile: BM x BN a workgroup, WM x WN each of its waves; RING stages
// of its operands in LDS, and at least OCC waves on a SIMD.
template <int BM_, int BN_, int WM_, int WN_, int RING_, int OCC_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, RING = RING_, OCC = OCC_;
  static constexpr int WAVES_M = BM / WM, WAVES = WAVES_M * (BN / WN), TM = WM / 32, TN = WN / 32;
  static_assert(TN % 2 == 0, "columns in pairs of blocks");
};


// The products' LDS stage: the BM / 32 blocks of the left operand's parts, then
// the BN / 32 of the right one's, each 32 rows of four 16-byte chunks.  Rows run
// along the reduction, but those of kApply's right operand, X, across it: its
// fragments are made by transpose reads.  Chunk c of row r is stored at
// c ^ (r / 4 % 4): the 16 rows that a plain read serves at a time then cover all
// banks once, and the four rows of a transpose read are whole rows either way.

// Floats in a row of the epilogue's blocks of 32 x 64, one a wave.
constexpr int kTurn = 68;

// dma_b128 with a part of the offset in a scalar register.
__device__ __forceinline__ void dma_at(i32x4 rsrc, uint32_t lds, uint32_t voffset, int soffset) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voffset), "s"(rsrc), "s"(soffset), "{m0}"(lds)
               : "memory");
}

// The tiles of A and B: those on and above the diagonal, row by row.  Tiles are
// as high as wide or a whole part of that, and the ones that hold the diagonal
// cover its whole squares; the others are mirrored.
template <class T>
__host__ __device__ __forceinline__ int64_t upper_tiles(int m) {
  constexpr int Q = T::BN / T::BM;
  static_assert(T::BN % T::BM == 0, "diagonal squares");
  const int64_t rows = (m + T::BM - 1) / T::BM, cols = (m + T::BN - 1) / T::BN, full = rows / Q, rest = rows % Q;
  return rows * cols - Q * (full * (full - 1) / 2) - rest * full;   // row r holds cols - r / Q
}
template <class T>
__device__ __forceinline__ void upper_tile(int m, int k, int& tm, int& tn) {
  constexpr int Q = T::BN / T::BM;
  const int cols = (m + T::BN - 1) / T::BN;
  tm = 0;
  while (k >= cols - tm / Q) k -= cols - tm++ / Q;
  tn = tm / Q + k;
}

// What a step's kernels take besides the weights.
struct Step {
  int cur;          // which of x[] holds X
  float a, b, c;
};

// The end of a product for 32 rows from r0 and 64 columns from c0 of its result,
// in a wave's accumulators v0 and v1 (32 columns each): A; B = b A + c v, plus
// a I if split; X <- v if split, else (a + d) X + v with d what rounding took off
// B's diagonal; or the outcome of the last step.
// They are turned through the wave's block of LDS, so that a lane holds 8
// columns of a row and what it reads and writes is whole 16-byte pieces of
// contiguous runs.  What goes out transposed (the mirrored tile, a tall weight)
// is put back and read by columns.
template <int KIND, bool SPLIT, bool LAST>
__device__ __forceinline__ void finish(const Job& j, const Step& st, bool mirror, int r0, int c0, const f16v& v0,
                                       const f16v& v1, float* turn, int lane) {
  const int g = lane >> 5, l32 = lane & 31, er = lane >> 3, ec = (lane & 7) * 8;
  // what is read, and what is written: X, or A and B, of one shape
  const _Float16* const old = KIND == kApply ? j.x[st.cur] : j.A;
  _Float16* const D = KIND == kGram ? j.A : KIND == kPoly ? j.B : j.x[1 - st.cur];
  const int nb = KIND == kApply ? j.nx : j.na;
  const int64_t plane = (int64_t)j.na * nb * 1024;
  const bool in = r0 < 32 * j.na && c0 + ec < 32 * nb;
  const int64_t at0 = at_block(r0 + er, c0 + ec, nb);   // rows 8 apart are 256 elements apart
  constexpr bool kAddX = KIND == kApply && !SPLIT, kLoads = KIND == kPoly || kAddX;
  h8 ohi[4], olo[4];
  float rest = 0.0f;   // of B's diagonal, for row l32 of the 32
  if constexpr (kAddX)
    if (r0 < 32 * j.na) rest = (float)j.B[(int64_t)j.na * j.na * 1024 + at_block(r0 + l32, r0 + l32, j.na)] * kInvScale;
  if constexpr (kLoads) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      ohi[p] = olo[p] = h8{};
      if (in) {
        ohi[p] = *reinterpret_cast<const h8*>(old + at0 + p * 256);
        if constexpr (SPLIT || kAddX) olo[p] = *reinterpret_cast<const h8*>(old + at0 + p * 256 + plane);
      }
    }
  }
  // the outcome's place: rows of n, or for a tall weight of m, read and written
  // 16 bytes at a time where they allow it
  const bool by_col = KIND == kApply ? LAST && j.tall : mirror;
  const int width = j.tall ? j.m : j.n;
  const bool whole = width % 8 == 0;
  int64_t o[4];
  int left[4];   // entries of the eight that exist
  float pw[4][8];
  if constexpr (LAST) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = j.tall ? c0 + p * 16 + (lane >> 2) : r0 + p * 8 + er;
      const int col = j.tall ? r0 + (lane & 3) * 8 : c0 + ec;
      o[p] = (int64_t)row * width + col;
      left[p] = row < (j.tall ? j.n : j.m) ? min(8, width - col) : 0;
      if (j.P != nullptr && left[p] > 0) {
        if (whole) {
          load8(j.P, true, o[p], o[p] + 8, pw[p]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) pw[p][e] = j.P[o[p] + min(e, left[p] - 1)];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float* const to = turn + (8 * (i >> 2) + 4 * g + (i & 3)) * kTurn + l32;
    to[0] = v0[i];
    to[32] = v1[i];
  }
  wave_sync();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float* const mine = turn + (p * 8 + er) * kTurn + ec;
    const f4 x = *reinterpret_cast<const f4*>(mine), y = *reinterpret_cast<const f4*>(mine + 4);
    const float a = kAddX ? st.a + __shfl(rest, p * 8 + er) : st.a;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = (e < 4 ? x[e & 3] : y[e & 3]) * kInvScale;
      if constexpr (kLoads) {
        const float was = (float)ohi[p][e] + (float)olo[p][e];
        v[e] = KIND == kPoly ? st.b * was + st.c * v[e] : a * was + v[e];
        if constexpr (KIND == kPoly && SPLIT)
          if (r0 + p * 8 + er == c0 + ec + e) v[e] += a * kScale;
      }
      if constexpr (LAST) v[e] *= kInvScale;
    }
    if constexpr (!LAST)
      if (in) put8(D + at0 + p * 256, plane, SPLIT || KIND == kApply || (KIND == kPoly && !mirror), v);
    if (LAST || by_col) {
      *reinterpret_cast<f4*>(mine) = f4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f4*>(mine + 4) = f4{v[4], v[5], v[6], v[7]};
    }
  }
  if (LAST || by_col) {
    wave_sync();
    const int step = by_col ? kTurn : 1;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float* const from = by_col ? turn + (lane & 3) * 8 * kTurn + p * 16 + (lane >> 2) : turn + (p * 8 + er) * kTurn + ec;
      if constexpr (!LAST) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = from[e * step];
        const int row = c0 + p * 16 + (lane >> 2), col = r0 + (lane & 3) * 8;
        if (row < 32 * j.na && col < 32 * j.na) put8(D + at_block(row, col, nb), plane, SPLIT, v);
      } else {
        if (left[p] <= 0) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = from[e * step];
        if (j.P != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = j.keep * pw[p][e] - j.lr * v[e];
        }
        float* const to32 = j.P != nullptr ? j.P : j.out32 ? static_cast<float*>(j.out) : nullptr;
        _Float16* const to16 = j.P != nullptr ? reinterpret_cast<_Float16*>(j.W) : j.out32 ? nullptr : static_cast<_Float16*>(j.out);
        if (whole) {
          if (to32 != nullptr) store8(to32, o[p], o[p] + 8, v);
          if (to16 != nullptr) {
            h8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[e];
            *reinterpret_cast<h8*>(to16 + o[p]) = h;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e >= left[p]) continue;
            if (to32 != nullptr) to32[o[p] + e] = v[e];
            if (to16 != nullptr) to16[o[p] + e] = (_Float16)v[e];
          }
        }
      }
    }
  }
  wave_sync();   // the block has been read
}

template <int KIND, bool SPLIT, bool LAST, class T>
__global__ __launch_bounds__(64 * T::WAVES, T::OCC) void ns_product_kernel(Jobs jobs, Step st) {
  constexpr int PARTS = SPLIT ? 2 : 1;
  constexpr int LEFT = T::BM * kBK * 2, RIGHT = T::BN * kBK * 2;   // bytes of one operand's part
  constexpr int STAGE = PARTS * (LEFT + RIGHT);
  constexpr int LL = LEFT / 1024, RL = RIGHT / 1024;   // 1 KiB direct loads of a part
  constexpr int W = T::WAVES, LN = (PARTS * LL + W - 1) / W, RN = (PARTS * RL + W - 1) / W;   // a wave's, at most
  static_assert((T::RING - 2) * (LN + RN) < 64, "vmcnt immediate");
  static_assert(W * 32 * kTurn * 4 <= T::RING * STAGE, "the epilogue's blocks fit the ring");
  __shared__ __align__(1024) unsigned char smem[T::RING * STAGE];
  const Job& j = job_of(jobs, blockIdx.x);
  const int block = blockIdx.x - j.first;
  const int tiles_m = (j.m + T::BM - 1) / T::BM;

  // Workgroups go round the 8 XCDs; each takes a run of the items, so that its
  // L2 fetches an operand strip or a slice of the reduction once.
  int tiles;
  if constexpr (KIND == kApply)
    tiles = tiles_m * ((j.n + T::BN - 1) / T::BN);
  else
    tiles = (int)upper_tiles<T>(j.m);
  const int splits = KIND == kGram ? j.gram_splits : 1;
  const int items = tiles * splits, run = (items + 7) / 8;
  const int lin = block % 8 * run + block / 8;
  if (block / 8 >= run || lin >= items) return;
  const int tile = lin % tiles, sp = lin / tiles;
  int tm, tn;
  if constexpr (KIND == kApply) {
    tm = tile % tiles_m;
    tn = tile / tiles_m;
  } else {
    upper_tile<T>(j.m, tile, tm, tn);
  }
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % T::WAVES_M, wn = wave / T::WAVES_M;
  const int g = lane >> 5, l32 = lane & 31;

  const int64_t xplane = (int64_t)j.na * j.nx * 1024, aplane = (int64_t)j.na * j.na * 1024;
  const _Float16* const X = j.x[st.cur];
  const _Float16* const left = KIND == kGram ? X : KIND == kPoly ? j.A : j.B;
  const _Float16* const right = KIND == kPoly ? j.A : X;
  const int lnb = KIND == kGram ? j.nx : j.na, rnb = KIND == kPoly ? j.na : j.nx;
  const int64_t lplane = KIND == kGram ? xplane : aplane, rplane = KIND == kPoly ? aplane : xplane;
  // this item's stages of the reduction
  const int nk_all = lnb, k_lo = nk_all * sp / splits, nk = nk_all * (sp + 1) / splits - k_lo;

  // One descriptor over each operand's parts.  This wave's direct loads of a
  // stage are every W-th KiB of the left operand's, then of the right one's;
  // a lane's offset is that of the chunk that belongs in its slot, and past
  // everything, which reads as zero, for blocks outside the matrix.
  const i32x4 lrsrc = make_rsrc(left, (uint32_t)(PARTS * lplane * 2)), rrsrc = make_rsrc(right, (uint32_t)(PARTS * rplane * 2));
  constexpr int kBlock = 2048;
  constexpr uint32_t kNowhere = 0x80000000u;
  const int left_step = kBlock, right_step = KIND == kApply ? rnb * kBlock : kBlock;
  uint32_t loff[LN], roff[RN];
#pragma unroll
  for (int u = 0; u < LN; ++u) {
    const int ld = wave + W * u, s = ld % LL * 64 + lane, row = s / 4 % 32, blk = m0 / 32 + s / 128;
    loff[u] = blk < j.na ? (uint32_t)(ld / LL * lplane * 2 + ((int64_t)blk * lnb + k_lo) * kBlock + row * 64 + ((s & 3) ^ (row >> 2 & 3)) * 16)
                         : kNowhere;
  }
#pragma unroll
  for (int u = 0; u < RN; ++u) {
    const int ld = wave + W * u, s = ld % RL * 64 + lane, row = s / 4 % 32, blk = n0 / 32 + s / 128;
    const int64_t first = KIND == kApply ? (int64_t)k_lo * rnb + blk : (int64_t)blk * rnb + k_lo;
    roff[u] = blk < (KIND == kApply ? rnb : j.na)
                  ? (uint32_t)(ld / RL * rplane * 2 + first * kBlock + row * 64 + ((s & 3) ^ (row >> 2 & 3)) * 16)
                  : kNowhere;
  }
  const uint32_t ring = lds_addr(smem) + 1024 * wave;
  auto issue_one = [&](int u, int kt, int slot) __attribute__((always_inline)) {
    const uint32_t dst = ring + slot * STAGE;
    if (u < LN) {
      if (W * (u + 1) <= PARTS * LL || wave < PARTS * LL % W) dma_at(lrsrc, dst + 1024 * W * u, loff[u], kt * left_step);
    } else {
      const int v = u - LN;
      if (W * (v + 1) <= PARTS * RL || wave < PARTS * RL % W)
        dma_at(rrsrc, dst + PARTS * LEFT + 1024 * W * v, roff[v], kt * right_step);
    }
  };
  auto issue = [&](int kt, int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < LN + RN; ++u) issue_one(u, kt, slot);
  };
  // allow `stages` stages of this wave's loads to stay in flight
  const int nl = PARTS * LL / W + PARTS * RL / W + (wave < PARTS * LL % W) + (wave < PARTS * RL % W);
  auto wait_loads = [&]<int I>(std::integral_constant<int, I>) __attribute__((always_inline)) {
    constexpr int lo = PARTS * LL / W + PARTS * RL / W;
    if (PARTS * LL % W == 0 && PARTS * RL % W == 0)
      wait_vm<I * lo>();
    else if (nl == lo)
      wait_vm<I * lo>();
    else if (nl == lo + 1)
      wait_vm<I * (lo + 1)>();
    else
      wait_vm<I * (lo + 2)>();
  };

  // this lane's fragment offsets inside an operand's part, per block
  int l_off[T::TM], r_off[T::TN];
  const int G = lane >> 4, j4 = (lane & 15) >> 2, c4 = lane & 3;   // transpose reads: 16-lane group, row, 4 columns
#pragma unroll
  for (int t = 0; t < T::TM; ++t) l_off[t] = (wm * T::TM + t) * kBlock + l32 * 64;
#pragma unroll
  for (int t = 0; t < T::TN; ++t)
    r_off[t] = PARTS * LEFT + (wn * T::TN + t) * kBlock + (KIND == kApply ? (8 * (G >> 1) + j4) * 64 + (c4 & 1) * 8 : l32 * 64);
  const int swz = (l32 >> 2) & 3;
  auto row_frag = [&](int base, int ks) -> h8 {
    return *reinterpret_cast<const h8*>(smem + base + (((2 * ks + g) ^ swz) * 16));
  };
  // rows 8 (G / 2) + j4 and the row 4 below, columns 16 (G % 2) + 4 c4 .. + 3
  const int tr_q = 2 * (G & 1) + (c4 >> 1), tr_lo = (tr_q ^ (2 * (G >> 1))) * 16, tr_hi = (tr_q ^ (2 * (G >> 1) + 1)) * 16 + 4 * 64;
  auto tr_frag = [&](int base, int ks) -> h8 {
    const int o = base + ks * 16 * 64;
    const h4 lo = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o + tr_lo)));
    const h4 hi = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o + tr_hi)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  struct Frags {
    h8 l[PARTS][T::TM], r[PARTS][T::TN];
  };
  // fragments of step ks (of 16) of the stage in ring slot `slot`
  auto load_frags = [&](int slot, int ks, Frags& f) __attribute__((always_inline)) {
    const int base = slot * STAGE;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
      for (int t = 0; t < T::TM; ++t) f.l[p][t] = row_frag(base + p * LEFT + l_off[t], ks);
#pragma unroll
      for (int t = 0; t < T::TN; ++t) {
        if constexpr (KIND == kApply)
          f.r[p][t] = tr_frag(base + p * RIGHT + r_off[t], ks);
        else
          f.r[p][t] = row_frag(base + p * RIGHT + r_off[t], ks);
      }
    }
  };

  f16v acc[T::TM][T::TN];
#pragma unroll
  for (int s = 0; s < T::TM; ++s)
#pragma unroll
    for (int t = 0; t < T::TN; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[s][t][e] = 0.0f;
  // the MFMAs of one step; with LOAD this wave's loads of stage kt go out
  // between them
  auto mfmas = [&]<bool LOAD>(const Frags& f, std::bool_constant<LOAD>, int kt, int slot) __attribute__((always_inline)) {
    constexpr int each = (LN + RN + T::TM * T::TN - 1) / (T::TM * T::TN);
#pragma unroll
    for (int s = 0; s < T::TM; ++s)
#pragma unroll
      for (int t = 0; t < T::TN; ++t) {
        if constexpr (SPLIT) {
          acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.l[0][s], f.r[1][t], acc[s][t], 0, 0, 0);
          acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.l[1][s], f.r[0][t], acc[s][t], 0, 0, 0);
        }
        acc[s][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.l[0][s], f.r[0][t], acc[s][t], 0, 0, 0);
        if constexpr (LOAD) {
#pragma unroll
          for (int u = (s * T::TN + t) * each; u < (s * T::TN + t + 1) * each; ++u)
            if (u < LN + RN) issue_one(u, kt, slot);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  };

  // Pipeline: stage s goes to ring slot s % RING, RING stages ahead.  In a
  // stage the second step's fragments are read during the first step's MFMAs;
  // in its middle the wave waits for the next stage's loads and for its own
  // reads, all waves meet (nobody reads this stage's slot afterwards), and the
  // stage RING further is loaded into it while the next stage's first fragments
  // are read.
  constexpr int R = T::RING;
#pragma unroll
  for (int s = 0; s < R; ++s)
    if (s < nk) issue(s, s);
  if (nk > 0) {
    // stages that may still be on their way when `left` of them come after the
    // one that is needed
    auto wait_at_most = [&](int left) __attribute__((always_inline)) {
      [&]<int... I>(std::integer_sequence<int, I...>) __attribute__((always_inline)) {
        ((left == I || (I == R - 1 && left > I) ? wait_loads(std::integral_constant<int, I>{}) : (void)0), ...);
      }(std::make_integer_sequence<int, R>{});
    };
    wait_at_most(nk - 1);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frags f0, f1;
    load_frags(0, 0, f0);
    int slot = 0;
    auto stage = [&]<bool LOAD>(std::bool_constant<LOAD>, int kt) __attribute__((always_inline)) {
      const int next = slot + 1 == R ? 0 : slot + 1;
      load_frags(slot, 1, f1);
      __builtin_amdgcn_sched_barrier(0);
      mfmas(f0, std::false_type{}, 0, 0);
      if constexpr (LOAD)
        wait_loads(std::integral_constant<int, R - 2>{});
      else
        wait_at_most(max(nk - 2 - kt, 0));
      __builtin_amdgcn_s_waitcnt(0xF | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      load_frags(next, 0, f0);   // after the last stage: of no use, and none made
      __builtin_amdgcn_sched_barrier(0);
      mfmas(f1, std::bool_constant<LOAD>{}, kt + R, slot);
      slot = next;
    };
    int kt = 0;
#pragma unroll 1
    for (; kt + R < nk; ++kt) stage(std::true_type{}, kt);
#pragma unroll 1
    for (; kt < nk; ++kt) stage(std::false_type{}, kt);
  }
  __syncthreads();   // the ring is idle

  if constexpr (KIND == kGram) {
    if (splits > 1) {
      // the item's share of the sums, for ns_join_kernel
      constexpr int FLOATS = T::BM * T::BN;
      float* const mine = j.partial + ((int64_t)tile * splits + sp) * FLOATS + wave * (FLOATS / W);
#pragma unroll
      for (int s = 0; s < T::TM; ++s)
#pragma unroll
        for (int t = 0; t < T::TN; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f4*>(mine + ((s * T::TN + t) * 4 + q) * 256 + lane * 4) =
                f4{acc[s][t][4 * q], acc[s][t][4 * q + 1], acc[s][t][4 * q + 2], acc[s][t][4 * q + 3]};
      return;
    }
  }
  // A wave's accumulators go out 32 rows x 64 columns at a time.
  float* const turn = reinterpret_cast<float*>(smem) + wave * (32 * kTurn);
  constexpr int Q = T::BN < T::BM ? 1 : T::BN / T::BM;
  const bool mirror = KIND != kApply && tn != tm / Q;
  [&]<int... I>(std::integer_sequence<int, I...>) __attribute__((always_inline)) {
    (
        [&]() __attribute__((always_inline)) {
          constexpr int s = I / (T::TN / 2), t = I % (T::TN / 2) * 2;
          finish<KIND, SPLIT, LAST>(j, st, mirror, m0 + wm * T::WM + s * 32, n0 + wn * T::WN + t * 32, acc[s][t],
                                         acc[s][t + 1], turn, lane);
          __builtin_amdgcn_sched_barrier(0);   // one block's registers at a time
        }(),
        ...);
  }(std::make_integer_sequence<int, T::TM * T::TN / 2>{});
}

// Adds up the shares of split reductions, in their order, 32 x 64 a wave.  8 to
// 9 us for those of a 1600 x 1600 A.  With the last item of a tile to arrive
// adding them up in the product's launch, the two took 52 us together, here 33
// (fp16 operands).
template <bool SPLIT, class T>
__global__ __launch_bounds__(64 * T::WAVES) void ns_join_kernel(Jobs jobs, Step st) {
  __shared__ __align__(16) float smem[T::WAVES * 32 * kTurn];
  const Job& j = job_of(jobs, blockIdx.x);
  const int splits = j.gram_splits;
  if (splits <= 1) return;
  constexpr int PAIRS = T::TM * T::TN / 2;   // of a wave's tile, and workgroups of a tile
  const int k = (blockIdx.x - j.first) / PAIRS;
  const int pair = (blockIdx.x - j.first) % PAIRS, s = pair / (T::TN / 2), t = pair % (T::TN / 2) * 2;
  constexpr int FLOATS = T::BM * T::BN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* p = j.partial + (int64_t)k * splits * FLOATS + wave * (FLOATS / T::WAVES) + (s * T::TN + t) * 1024 + lane * 4;
  int tm, tn;
  upper_tile<T>(j.m, k, tm, tn);
  f16v acc[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[h][e] = 0.0f;
#pragma unroll 2
  for (int i = 0; i < splits; ++i, p += FLOATS) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const f4 v = *reinterpret_cast<const f4*>(p + q * 256);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[q >> 2][4 * (q & 3) + e] += v[e];
    }
  }
  finish<kGram, SPLIT, false>(j, st, tn != tm / (T::BN / T::BM), tm * T::BM + wave % T::WAVES_M * T::WM + s * 32,
                             tn * T::BN + wave / T::WAVES_M * T::WN + t * 32, acc[0], acc[1], smem + wave * (32 * kTurn), lane);
}

// All of a small weight's steps in one workgroup, with X, A and B in LDS, in the
// blocks and swizzle that a stage of the large products has there.  A chain of
// launches takes 4 us a product whatever its size; 64 x 64 and five steps took
// 76 us of them, and 23 here (fp16 operands: 21).  What is left is latency: each
// step's three products wait for LDS and for each other.  Every product's tiles
// are made with the operands such that a lane ends up with four neighbours of a row of the result: of A and B, which
// are symmetric, both halves are computed; of X, a wave makes whole columns of
// blocks, which nothing else reads, and puts them back in place.
constexpr int kSmallThreads = 512, kSmallBytes = 152 * 1024, kSmallRows = 4;   // blocks of 32
struct Coefs {
  float c[3 * kMaxNsSteps];
};

template <bool SPLIT>
constexpr int64_t small_bytes(int64_t na, int64_t nx) {
  return 2048 * (2 * na * nx + (SPLIT ? 4 : 2) * na * na);
}

template <bool SPLIT>
__global__ __launch_bounds__(kSmallThreads) void ns_small_kernel(Jobs jobs, Coefs coefs, int steps, float mu, bool nesterov,
                                                                  float eps) {
  constexpr int PARTS = SPLIT ? 2 : 1, WAVES = kSmallThreads / 64;
  __shared__ __align__(1024) unsigned char smem[kSmallBytes];
  __shared__ double wave_sums[WAVES];
  __shared__ float rest[32 * kSmallRows];   // what rounding took off B's diagonal, if not split
  const Job& j = jobs.j[blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 5, l32 = lane & 31, na = j.na, nx = j.nx;
  const int xplane = na * nx * 2048, aplane = na * na * 2048;
  const int X = 0, A = 2 * xplane, B = A + PARTS * aplane;   // byte offsets

  // momentum and norm, eight entries of U at a time
  const int total = j.m * j.n, width = j.tall ? j.m : j.n;
  double sum = 0.0;
  for (int i = tid * 8; i < total; i += kSmallThreads * 8) {
    float u[8];
    load8(j.G, j.g32, i, total, u);
    if (j.M != nullptr) {
      float m[8];
      load8(j.M, true, i, total, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = mu * m[e] + u[e];
        u[e] = nesterov ? u[e] + mu * m[e] : m[e];
      }
      store8(j.M, i, total, m);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)u[e] * (double)u[e];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) wave_sums[wave] = sum;
  for (int i = tid; i < 2 * xplane / 16; i += kSmallThreads) reinterpret_cast<i32x4*>(smem + X)[i] = i32x4{};
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += wave_sums[w];
  const double scale = (double)kScale / (sqrt(sum) + (double)eps);

  // Where X has U's entries i .. i + 7: in one 16-byte piece if U's rows are X's
  // and hold whole eights, else each for itself.
  const bool pieces = !j.tall && width % 8 == 0;
  const auto place = [&](int row, int col) __attribute__((always_inline)) {
    return X + ((row >> 5) * nx + (col >> 5)) * 2048 + (row & 31) * 64 + ((col >> 3 & 3) ^ (row >> 2 & 3)) * 16 + (col & 7) * 2;
  };
  const auto places = [&](int i, int (&at)[8]) __attribute__((always_inline)) {
    int r = i / width, k = i - r * width;   // of U
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      at[e] = j.tall ? place(k, r) : place(r, k);
      if (++k == width) {
        k = 0;
        ++r;
      }
    }
  };
  for (int i = tid * 8; i < total; i += kSmallThreads * 8) {
    float u[8];
    load8(j.G, j.g32, i, total, u);
    if (j.M != nullptr) {
      float m[8];   // this thread's own stores
      load8(j.M, true, i, total, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = nesterov ? u[e] + mu * m[e] : m[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = (float)((double)u[e] * scale);
    int at[8];
    places(i, at);
    if (pieces) {
      put8(reinterpret_cast<_Float16*>(smem + at[0]), xplane / 2, true, u);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (i + e >= total) continue;
        _Float16 hi, lo;
        split(u[e], hi, lo);
        *reinterpret_cast<_Float16*>(smem + at[e]) = hi;
        *reinterpret_cast<_Float16*>(smem + at[e] + xplane) = lo;
      }
    }
  }
  __syncthreads();

  const int swz = l32 >> 2 & 3;
  const int G = lane >> 4, j4 = (lane & 15) >> 2, c4 = lane & 3;
  const int tr_q = 2 * (G & 1) + (c4 >> 1), tr_row = (8 * (G >> 1) + j4) * 64 + (c4 & 1) * 8;
  const int tr_lo = tr_row + (tr_q ^ (2 * (G >> 1))) * 16, tr_hi = tr_row + (tr_q ^ (2 * (G >> 1) + 1)) * 16 + 4 * 64;
  auto row_frag = [&](int block, int ks) __attribute__((always_inline)) {
    return *reinterpret_cast<const h8*>(smem + block + l32 * 64 + (((2 * ks + g) ^ swz) * 16));
  };
  auto tr_frag = [&](int block, int ks) __attribute__((always_inline)) {
    const int o = block + ks * 16 * 64;
    const h4 lo = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o + tr_lo)));
    const h4 hi = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)((lds_u8*)smem + o + tr_hi)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto mfma = [&](f16v& acc, const h8 (&l)[PARTS], const h8 (&r)[PARTS]) __attribute__((always_inline)) {
    if constexpr (SPLIT) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(l[0], r[1], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(l[1], r[0], acc, 0, 0, 0);
    }
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(l[0], r[0], acc, 0, 0, 0);
  };
  // this lane's four values 4 q .. 4 q + 3 of a tile: row l32, columns 8 q + 4 g ..
  auto four = [&](int block, int q) __attribute__((always_inline)) { return block + l32 * 64 + (q ^ swz) * 16 + g * 8; };
  auto get4 = [&](int at, int plane, bool both, float (&v)[4]) __attribute__((always_inline)) {
    const h4 hi = *reinterpret_cast<const h4*>(smem + at);
    const h4 lo = both ? *reinterpret_cast<const h4*>(smem + at + plane) : h4{};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)hi[e] + (float)lo[e];
  };
  auto put4 = [&](int at, int plane, bool both, const float (&v)[4]) __attribute__((always_inline)) {
    h4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      _Float16 h, l;
      split(v[e], h, l);
      hi[e] = h;
      lo[e] = l;
    }
    *reinterpret_cast<h4*>(smem + at) = hi;
    if (both) *reinterpret_cast<h4*>(smem + at + plane) = lo;
  };
  auto zero = [](f16v& acc) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  };

  for (int k = 0; k < steps; ++k) {
    const float a = coefs.c[3 * k], b = coefs.c[3 * k + 1], c = coefs.c[3 * k + 2];
    // A = X X^T, then B = b A + c A A (+ a I if split); tile (t / na, t % na) is stored transposed
    for (int t = wave; t < na * na; t += WAVES) {
      const int ti = t / na, tj = t % na;
      f16v acc;
      zero(acc);
      for (int kb = 0; kb < nx; ++kb)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          h8 l[PARTS], r[PARTS];
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            l[p] = row_frag(X + p * xplane + (ti * nx + kb) * 2048, ks);
            r[p] = row_frag(X + p * xplane + (tj * nx + kb) * 2048, ks);
          }
          mfma(acc, l, r);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[4 * q + e] * kInvScale;
        put4(four(A + (tj * na + ti) * 2048, q), aplane, SPLIT, v);
      }
    }
    __syncthreads();
    for (int t = wave; t < na * na; t += WAVES) {
      const int ti = t / na, tj = t % na;
      f16v acc;
      zero(acc);
      for (int kb = 0; kb < na; ++kb)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          h8 l[PARTS], r[PARTS];
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            l[p] = row_frag(A + p * aplane + (ti * na + kb) * 2048, ks);
            r[p] = row_frag(A + p * aplane + (tj * na + kb) * 2048, ks);
          }
          mfma(acc, l, r);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4], was[4];
        get4(four(A + (tj * na + ti) * 2048, q), aplane, SPLIT, was);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = b * was[e] + c * (acc[4 * q + e] * kInvScale);
          if (ti == tj && l32 == 8 * q + 4 * g + e) {
            if constexpr (SPLIT)
              v[e] += a * kScale;
            else
              rest[32 * ti + l32] = v[e] - (float)(_Float16)v[e];
          }
        }
        put4(four(B + (tj * na + ti) * 2048, q), aplane, SPLIT, v);
      }
    }
    __syncthreads();
    // X <- a X + B X, or B X if split: transposed, X^T B, so that a lane has four columns of a row
    for (int t = wave; t < nx; t += WAVES) {
      f16v acc[kSmallRows];
#pragma unroll
      for (int i = 0; i < kSmallRows; ++i) {
        zero(acc[i]);
        if (i >= na) continue;
        for (int kb = 0; kb < na; ++kb)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            h8 l[PARTS], r[PARTS];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
              l[p] = tr_frag(X + p * xplane + (kb * nx + t) * 2048, ks);
              r[p] = row_frag(B + p * aplane + (i * na + kb) * 2048, ks);
            }
            mfma(acc[i], l, r);
          }
      }
#pragma unroll
      for (int i = 0; i < kSmallRows; ++i) {
        if (i >= na) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = four(X + (i * nx + t) * 2048, q);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][4 * q + e] * kInvScale;
          if constexpr (!SPLIT) {
            float was[4];
            get4(at, xplane, true, was);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += (a + rest[32 * i + l32] * kInvScale) * was[e];
          }
          put4(at, xplane, true, v);
        }
      }
    }
    __syncthreads();
  }

  // the outcome, in U's order; both parts of X are 22 bits of it
  for (int i = tid * 8; i < total; i += kSmallThreads * 8) {
    float p[8], x[8];
    if (j.P != nullptr) load8(j.P, true, i, total, p);
    int at[8];
    places(i, at);
    h8 hi, lo;
    if (pieces) {
      hi = *reinterpret_cast<const h8*>(smem + at[0]);
      lo = *reinterpret_cast<const h8*>(smem + at[0] + xplane);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = i + e < total ? at[e] : at[0];
        hi[e] = *reinterpret_cast<const _Float16*>(smem + k);
        lo[e] = *reinterpret_cast<const _Float16*>(smem + k + xplane);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = ((float)hi[e] + (float)lo[e]) * kInvScale;
      if (j.P != nullptr) x[e] = j.keep * p[e] - j.lr * x[e];
    }
    if (j.P != nullptr || j.out32) store8(j.P != nullptr ? j.P : static_cast<float*>(j.out), i, total, x);
    if (j.P != nullptr ? j.W != nullptr : !j.out32) {
      _Float16* const to = (j.P != nullptr ? reinterpret_cast<_Float16*>(j.W) : static_cast<_Float16*>(j.out)) + i;
      h8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[e];
      if (i + 8 <= total) {
        *reinterpret_cast<h8*>(to) = h;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e < total) to[e] = h[e];
      }
    }
  }
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The tiles.  Square, for A and for all last products too small for the others:
// three of its workgroups share a CU when the products are rounded, one when
// they are split.  Small, for B, whose short reduction wants more workgroups: one
// 1600 x 1600 takes 15 us in 181 of them and 20 us in 91 squares (fp16 operands).
// Tall and Broad, for last products, read fewer bytes a product.
template <bool SPLIT> using Square = Tile<128, 128, 64, 64, 3, SPLIT ? 1 : 3>;
template <bool SPLIT> using Small = Tile<64, 128, 32, 64, SPLIT ? 3 : 4, SPLIT ? 2 : 3>;
using Tall = Tile<320, 256, 160, 64, 4, 2>;
using Broad = Tile<128, 256, 64, 64, 3, 2>;

// Items per tile of A's reduction over `stages` of it, for a launch of `tiles`
// tiles of `area`: the cheapest by a model of a stage's time on a CU, the items
// on the fullest CU (side by side they take 0.8 of one after the other; split
// products have no room for two), and the join, which costs a launch and the
// traffic of every item's sums.  Measured with the join and fp16 operands: one
// 1600 x 6400 weight 33 us in 5 items a tile, 36 in 2, 38 in 3, 35 in 8; two of
// them 57 us in 2, 63 in 1, 55 in 3.
int splits_for(int64_t tiles, int64_t area, bool split, int stages) {
  const double stage = (split ? 0.75e-6 : 0.3e-6) * (area < 128 * 128 ? 0.6 : 1.0), join = 5e-6, rate = 8e12;
  const int64_t cus = device_cu_count();
  int best = 1;
  double best_t = 0.0;
  for (int n = 1; n <= 16 && (n == 1 || stages / n >= 8); ++n) {
    const double items = (double)((tiles * n + cus - 1) / cus);
    const double t = (double)stages / n * stage * items * (items > 1.0 && !split ? 0.8 : 1.0) +
                     (n > 1 ? join + 2.0 * 4.0 * (double)(tiles * n * area) / rate : 0.0);
    if (n == 1 || t < best_t) {
      best = n;
      best_t = t;
    }
  }
  return best;
}

template <class T>
int64_t partial_bytes(const Job& j) {
  return upper_tiles<T>(j.m) * j.gram_splits * T::BM * T::BN * 4;
}

// Bytes of one weight's workspace; fills its pointers when base is given.
int64_t lay_out(Job& j, bool fine, unsigned char* base) {
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    unsigned char* p = base ? base + at : nullptr;
    at += up(bytes, 256);
    return p;
  };
  const int64_t x = (int64_t)j.na * j.nx * 4096, a = (int64_t)j.na * j.na * 4096;   // two parts of 2 bytes
  j.sums = reinterpret_cast<double*>(take(kMaxParts * 8));
  j.x[0] = reinterpret_cast<_Float16*>(take(x));
  j.x[1] = reinterpret_cast<_Float16*>(take(x));
  j.A = reinterpret_cast<_Float16*>(take(a));
  j.B = reinterpret_cast<_Float16*>(take(a));
  const int splits = j.gram_splits;
  j.partial = reinterpret_cast<float*>(take(splits <= 1 ? 0
                                                : fine    ? partial_bytes<Small<false>>(j)
                                                          : partial_bytes<Square<false>>(j)));
  return at;
}

template <bool SPLIT>
bool is_small(const Job& j) {
  return j.na <= kSmallRows && small_bytes<SPLIT>(j.na, j.nx) <= kSmallBytes;
}

// The launch's weights, small ones apart; returns the workspace's bytes, which
// do not depend on `split`.
int64_t fill(Jobs& large, Jobs& small, const NsJob* in, int count, bool split, unsigned char* ws) {
  int64_t at = 0, squares = 0, upper = 0, upper_fine = 0;
  Jobs all{};
  for (int k = 0; k < count; ++k) {
    const NsJob& s = in[k];
    if (s.R == 0 || s.C == 0) continue;
    Job& j = all.j[all.count++];
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
    j.na = (j.m + 31) / 32;
    j.nx = (j.n + 31) / 32;
    const int64_t parts = ((int64_t)j.m * j.n + kNormChunk - 1) / kNormChunk;
    j.parts = (int)(parts < kMaxParts ? parts : kMaxParts);
    j.g32 = s.g32;
    j.out32 = s.out32;
    if (is_small<true>(j)) continue;
    squares += up(j.m, Square<false>::BM) / Square<false>::BM * (up(j.n, Square<false>::BN) / Square<false>::BN);
    upper += upper_tiles<Square<false>>(j.m);
    upper_fine += upper_tiles<Small<false>>(j.m);
  }
  // where even twice the tiles leave CUs idle, tiles half as large
  large.fine = 2 * squares <= device_cu_count();
  for (int k = 0; k < all.count; ++k) {
    Job& j = all.j[k];
    if (is_small<true>(j)) {
      at += 256;   // so that every call has a workspace
      small.j[small.count++] = j;
      continue;
    }
    const int64_t tiles = large.fine ? upper_fine : upper;
    const int64_t area = large.fine ? Small<false>::BM * Small<false>::BN : Square<false>::BM * Square<false>::BN;
    const int rounded = splits_for(tiles, area, false, j.nx), in_parts = splits_for(tiles, area, true, j.nx);
    j.gram_splits = rounded > in_parts ? rounded : in_parts;
    at += lay_out(j, large.fine, ws ? ws + at : nullptr);
    j.gram_splits = split ? in_parts : rounded;
    Jobs& to = !split && is_small<false>(j) ? small : large;
    to.j[to.count++] = j;
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

template <int KIND, bool SPLIT, bool LAST, class T>
void product(Jobs& jobs, const Step& st, hipStream_t s) {
  const unsigned grid = deal(jobs, [](const Job& j) {
    if constexpr (KIND == kApply)
      return up(up(j.m, T::BM) / T::BM * (up(j.n, T::BN) / T::BN), 8);
    else
      return up(upper_tiles<T>(j.m) * (KIND == kGram ? j.gram_splits : 1), 8);
  });
  hipLaunchKernelGGL((ns_product_kernel<KIND, SPLIT, LAST, T>), dim3(grid), dim3(64 * T::WAVES), 0, s, jobs, st);
  if constexpr (KIND == kGram) {
    const unsigned blocks =
        deal(jobs, [](const Job& j) { return j.gram_splits > 1 ? upper_tiles<T>(j.m) * (T::TM * T::TN / 2) : 0; });
    if (blocks > 0) hipLaunchKernelGGL((ns_join_kernel<SPLIT, T>), dim3(blocks), dim3(64 * T::WAVES), 0, s, jobs, st);
  }
}

template <class T>
int64_t apply_tiles(const Jobs& jobs) {
  int64_t t = 0;
  for (int k = 0; k < jobs.count; ++k) t += up(jobs.j[k].m, T::BM) / T::BM * (up(jobs.j[k].n, T::BN) / T::BN);
  return t;
}

template <bool SPLIT, class T>
void apply(Jobs& jobs, const Step& st, bool last, hipStream_t s) {
  if (last)
    product<kApply, SPLIT, true, T>(jobs, st, s);
  else
    product<kApply, SPLIT, false, T>(jobs, st, s);
}

template <bool SPLIT>
void step(Jobs& jobs, const NsParams& prm, int k, hipStream_t s) {
  const Step st{k & 1, prm.coef[3 * k], prm.coef[3 * k + 1], prm.coef[3 * k + 2]};
  if (jobs.fine)
    product<kGram, SPLIT, false, Small<SPLIT>>(jobs, st, s);
  else
    product<kGram, SPLIT, false, Square<SPLIT>>(jobs, st, s);
  product<kPoly, SPLIT, false, Small<SPLIT>>(jobs, st, s);
  const bool last = k + 1 == prm.steps;
  // The larger tile where its whole rounds over the CUs cost less, by area over
  // measured speed (the squares of rounded products, three to a CU, are taken to
  // fill the CUs evenly).  Rounded products, whole calls of five steps: two 1600 x
  // 6400 weights 852 us with Tall tiles and 895 with Square ones, 4096 x 14336 4.73
  // and 5.20 ms; the product of one 1600 x 6400 without a X took 52 us in 125 Tall
  // tiles and 41 in 650 squares.  Split ones: 1024 x 4096 and its transpose take
  // 51 us in 256 Broad tiles, 59 us in 512 Square ones.
  if (jobs.fine) {
    apply<SPLIT, Small<SPLIT>>(jobs, st, last, s);
    return;
  }
  const int64_t cus = device_cu_count();
  const int64_t squares = apply_tiles<Square<SPLIT>>(jobs);
  if constexpr (SPLIT) {
    const int64_t rounds = (apply_tiles<Broad>(jobs) + cus - 1) / cus;
    if (rounds * 2 * 6 < (squares + cus - 1) / cus * 7)
      apply<SPLIT, Broad>(jobs, st, last, s);
    else
      apply<SPLIT, Square<SPLIT>>(jobs, st, last, s);
  } else {
    const int64_t rounds = (apply_tiles<Tall>(jobs) + cus - 1) / cus;
    if (rounds * 5 * 5 * cus < squares * 6)
      apply<SPLIT, Tall>(jobs, st, last, s);
    else
      apply<SPLIT, Square<SPLIT>>(jobs, st, last, s);
  }
}

}  // namespace

int64_t ns_workspace(const NsJob* jobs, int count) {
  Jobs large{}, small{};
  return fill(large, small, jobs, count, false, nullptr);
}

hipError_t launch_newton_schulz(const NsJob* in, int count, const NsParams& prm, void* ws, hipStream_t s) {
  Jobs jobs{}, small{};
  fill(jobs, small, in, count, prm.split, static_cast<unsigned char*>(ws));
  if (small.count > 0) {
    Coefs c{};
    for (int k = 0; k < 3 * prm.steps; ++k) c.c[k] = prm.coef[k];
    const auto kernel = prm.split ? ns_small_kernel<true> : ns_small_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)small.count), dim3(kSmallThreads), 0, s, small, c, prm.steps, prm.mu,
                       prm.nesterov, prm.eps);
  }
  if (jobs.count == 0) return hipGetLastError();
  const unsigned norm = deal(jobs, [](const Job& j) { return (int64_t)j.parts; });
  hipLaunchKernelGGL(ns_norm_kernel, dim3(norm), dim3(kThreads), 0, s, jobs, prm.mu, prm.nesterov);
  const unsigned start = deal(jobs, [](const Job& j) { return (int64_t)j.na * ((j.nx + 1) / 2); });
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
