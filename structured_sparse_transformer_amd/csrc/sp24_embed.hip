// Token embedding of the FFN path's input, and its gradient, for gfx950.
//
//   forward    out[t][:] = scale * table[ids[t]][:]
//   gradient   dtable[v][:] (+)= scale * sum over t with ids[t] == v of dout[t][:]
//
// An id outside [0, V) is padding: its output row is zero and it adds nothing
// to the gradient.  The method's pages name no embedding; it is the layer that
// makes the FFN path's X from token ids and takes its dX.
//
// The gradient sorts the tokens by id (stably, so that every row's sum runs in
// token order and results do not depend on timing), then sums runs of equal
// ids.  No atomics on floating point, no dense [T, V] anything.  Sums are held
// in fp32.
//
// Both move bytes and nothing else.  At 16384 tokens, width 1600 and 50257 rows
// the forward from an fp32 table takes 18 us (5.0 TB/s; a large copy reaches
// 5.1), the dense gradient 9 us to sort, 64 to sum and clear (5.8 TB/s, of which
// 86% are writes) and 6 to join the runs that chunks cut.  131072 tokens of
// width 1024 added to a gradient: 27, 93 (4.2 TB/s: rows of 2 and 4 KiB in the
// ids' order, a quarter of them read and written back) and 13 us.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

// Rows of any width are read and written 16 bytes at a time: the hardware takes
// such accesses at the element's alignment.  The last piece of a row begins at
// d - 8, over a part of the one before, whose values it has too; rows narrower
// than 8 go an element at a time.
typedef h8 h8u __attribute__((aligned(2)));
typedef f4 f4u __attribute__((aligned(4)));

constexpr int kThreads = 256;
constexpr int kItems = 4;   // row chunks per thread of the forward: that many gathers in flight

template <typename T>
__device__ __forceinline__ void load_row8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load_row8<_Float16>(const _Float16* p, float (&v)[8]) {
  const h8 x = *reinterpret_cast<const h8u*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
}
template <>
__device__ __forceinline__ void load_row8<float>(const float* p, float (&v)[8]) {
  const f4 x = *reinterpret_cast<const f4u*>(p), y = *reinterpret_cast<const f4u*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = x[e];
    v[4 + e] = y[e];
  }
}

// One gather per item from a row that its id names; kItems of them in flight a
// thread.  A row is d / VEC chunks, rounded up; a workgroup takes kThreads * kItems
// consecutive chunks of all rows'.
template <typename Table, typename Id, int VEC>
__global__ __launch_bounds__(kThreads) void embed_fwd_kernel(const Id* __restrict__ ids, const Table* __restrict__ table,
                                                              int64_t T, int64_t V, int64_t d, float scale,
                                                              _Float16* __restrict__ out) {
  const uint32_t chunks = (uint32_t)((d + VEC - 1) / VEC);
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kItems);
  const int64_t t0 = first / chunks;
  const uint32_t c0 = (uint32_t)(first - t0 * chunks);
  // no branches around the loads: kItems gathers are in flight
  int64_t t[kItems], id[kItems];
  int64_t c[kItems];   // first column
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = c0 + threadIdx.x + k * kThreads;   // c0 < chunks <= 2^31
    const uint32_t q = i / chunks;
    t[k] = t0 + q;
    c[k] = min<int64_t>((int64_t)(i - q * chunks) * VEC, d - VEC);
    id[k] = (int64_t)ids[min<int64_t>(t[k], T - 1)];
  }
  float v[kItems][VEC];
#pragma unroll
  for (int k = 0; k < kItems; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[k][e] = 0.0f;
  if (V > 0) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int64_t r = id[k] >= 0 && id[k] < V ? id[k] : 0;
      const Table* row = table + r * d + c[k];
      if constexpr (VEC == 8)
        load_row8<Table>(row, v[k]);
      else
        v[k][0] = (float)row[0];
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = id[k] >= 0 && id[k] < V ? v[k][e] * scale : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (t[k] >= T) continue;
    _Float16* o = out + t[k] * d + c[k];
    if constexpr (VEC == 8) {
      h8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[k][e];
      *reinterpret_cast<h8u*>(o) = h;
    } else {
      o[0] = (_Float16)v[k][0];
    }
  }
}

template <typename Table, typename Id>
hipError_t launch_fwd(const void* ids, const void* table, int64_t T, int64_t V, int64_t d, float scale, uint16_t* out,
                      hipStream_t s) {
  const Id* i = static_cast<const Id*>(ids);
  const Table* tb = static_cast<const Table*>(table);
  _Float16* o = reinterpret_cast<_Float16*>(out);
  const int vec = d >= 8 ? 8 : 1;
  const int64_t items = T * ((d + vec - 1) / vec);
  const dim3 grid((unsigned)((items + kThreads * kItems - 1) / (kThreads * kItems)));
  if (vec == 8)
    hipLaunchKernelGGL((embed_fwd_kernel<Table, Id, 8>), grid, dim3(kThreads), 0, s, i, tb, T, V, d, scale, o);
  else
    hipLaunchKernelGGL((embed_fwd_kernel<Table, Id, 1>), grid, dim3(kThreads), 0, s, i, tb, T, V, d, scale, o);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gradient: stable counting sort by id, then sums of runs.
//
// The ids are dealt in ranges of kRange to workgroups of kWaves waves, and the
// tokens in at most kMaxSegs segments, kMinSeg tokens long or more.  A workgroup
// keeps those tokens of its segment that are in its range; each wave has a
// contiguous part of the segment and its own counters, so that tokens of one
// id are placed in token order.
//   place: start[v], where id v's run begins in sorted order, and
//          sorted[p] = (token, id)
// For that it needs the number of tokens of each of its ids, in earlier
// segments and in all, and of those with ids below its range.  Up to
// kSelfCount tokens every workgroup counts them itself (16384 tokens are 128
// KiB from L2, less than a launch); beyond, a kernel before it does, once a
// segment:
//   count: cnt[seg][v] and below[seg][range]
constexpr int kRange = 2048, kWaves = 8, kSortThreads = 64 * kWaves, kEach = kRange / kSortThreads;
constexpr int kMinSeg = 2048, kMaxSegs = 16, kSelfCount = 32768;
constexpr int kGroups = 4;   // groups of 64 tokens that a wave loads at once
constexpr int kIdBits = 11;
static_assert(kMinSeg % (64 * kWaves) == 0 && 1 << kIdBits == kRange && kEach == 4, "whole waves of tokens, ids in fours");

// What one lane of a wave has written to LDS is read by the others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Token t's id; past the end and for every id beyond 32 bits, the largest
// number, which is no id (V < 2^31).  Scanning is the sort's work: every id is
// looked at once a range, in a few 32-bit operations, and without a branch, so
// that several loads are in flight.  end > 0.
__device__ __forceinline__ uint32_t id_at(const int32_t* ids, int t, int end) {
  const uint32_t w = (uint32_t)ids[min(t, end - 1)];
  return t < end ? w : ~0u;
}
__device__ __forceinline__ uint32_t id_at(const int64_t* ids, int t, int end) {
  const uint2 w = reinterpret_cast<const uint2*>(ids)[min(t, end - 1)];
  return t < end && w.y == 0 ? w.x : ~0u;
}

// Counts the tokens t0 .. end - 1 of the range's ids into n; returns, in
// every lane, how many of the wave's were below the range.
template <typename Id>
__device__ __forceinline__ int count_tokens(const Id* ids, int t0, int end, uint32_t lo, uint32_t span, int32_t* n) {
  int under = 0;
  constexpr int kLoads = 8;
  for (int t = t0; t < end; t += kLoads * kSortThreads) {
    uint32_t v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) v[k] = id_at(ids, t + k * kSortThreads + threadIdx.x, end);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (v[k] - lo < span) atomicAdd(&n[v[k] - lo], 1);
      under += __popcll(__ballot(v[k] < lo));
    }
  }
  return under;
}

template <typename Id>
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(const Id* __restrict__ ids, int T, int64_t V,
                                                             int seg_tokens, int32_t* __restrict__ cnt,
                                                             int32_t* __restrict__ below) {
  __shared__ __align__(16) int32_t n[kRange];
  __shared__ int32_t under;
  const int tid = threadIdx.x;
  const int64_t range = blockIdx.x;
  const int seg = blockIdx.y;
  const uint32_t lo = (uint32_t)(range * kRange), span = (uint32_t)min<int64_t>(kRange, V - lo);
  reinterpret_cast<int4*>(n)[tid] = int4{};
  if (tid == 0) under = 0;
  __syncthreads();
  const int mine = count_tokens(ids, seg * seg_tokens, min(T, (seg + 1) * seg_tokens), lo, span, n);
  if ((tid & 63) == 0) atomicAdd(&under, mine);
  __syncthreads();
  reinterpret_cast<int4*>(cnt)[(seg * gridDim.x + range) * kSortThreads + tid] = reinterpret_cast<const int4*>(n)[tid];
  if (tid == 0) below[seg * gridDim.x + range] = under;
}

template <typename Id, bool SELF>
__global__ __launch_bounds__(kSortThreads) void embed_place_kernel(const Id* __restrict__ ids, int T, int64_t V,
                                                             int seg_tokens, const int32_t* __restrict__ cnt,
                                                             const int32_t* __restrict__ below,
                                                             int32_t* __restrict__ start, int2* __restrict__ sorted) {
  // ids in fours, four to a thread
  __shared__ __align__(16) int32_t n[kWaves][kRange];   // counts of each wave's tokens, then where its next one goes
  __shared__ __align__(16) int32_t others[SELF ? 2 : 1][SELF ? kRange : 4];
  __shared__ int32_t wave_sum[kWaves], under;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t range = blockIdx.x, ranges = gridDim.x;
  const int seg = blockIdx.y, segs = gridDim.y;
  const uint32_t lo = (uint32_t)(range * kRange), span = (uint32_t)min<int64_t>(kRange, V - lo);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) reinterpret_cast<int4*>(n[w])[tid] = int4{};
  if constexpr (SELF) {
    reinterpret_cast<int4*>(others[0])[tid] = reinterpret_cast<int4*>(others[1])[tid] = int4{};
    if (tid == 0) under = 0;
  }
  __syncthreads();
  const int per_wave = seg_tokens / kWaves;
  const int t0 = seg * seg_tokens + wave * per_wave, end = min(t0 + per_wave, T);
  uint32_t v[kGroups];
  auto load = [&](int t) {
#pragma unroll
    for (int k = 0; k < kGroups; ++k) v[k] = id_at(ids, t + k * 64 + lane, end);
  };
  int mine = 0;
  for (int t = t0; t < end; t += kGroups * 64) {
    load(t);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (v[k] - lo < span) atomicAdd(&n[wave][v[k] - lo], 1);
      if constexpr (SELF) mine += __popcll(__ballot(v[k] < lo));
    }
  }
  // this thread's ids in the segments before and in all
  int total[kEach] = {}, before[kEach] = {}, base = 0;
  const auto add = [](int (&to)[kEach], const int4& v) {
    to[0] += v.x;
    to[1] += v.y;
    to[2] += v.z;
    to[3] += v.w;
  };
  if constexpr (SELF) {
    mine += count_tokens(ids, 0, min(T, seg * seg_tokens), lo, span, others[0]);
    mine += count_tokens(ids, (seg + 1) * seg_tokens, T, lo, span, others[1]);
    if (lane == 0) atomicAdd(&under, mine);
    __syncthreads();
    add(before, reinterpret_cast<const int4*>(others[0])[tid]);
    add(total, reinterpret_cast<const int4*>(others[0])[tid]);
    add(total, reinterpret_cast<const int4*>(others[1])[tid]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) add(total, reinterpret_cast<const int4*>(n[w])[tid]);
    base = under;
  } else {
    int4 c[kMaxSegs];   // all loads in flight
    int u[kMaxSegs];
#pragma unroll
    for (int s = 0; s < kMaxSegs; ++s) {
      const int k = min(s, segs - 1);
      c[s] = reinterpret_cast<const int4*>(cnt)[(k * ranges + range) * kSortThreads + tid];
      u[s] = below[k * ranges + range];
    }
#pragma unroll
    for (int s = 0; s < kMaxSegs; ++s) {
      if (s < segs) {
        add(total, c[s]);
        base += u[s];
      }
      if (s < seg) add(before, c[s]);
    }
  }
  // exclusive scan of the totals over the range's ids
  const int sum = total[0] + total[1] + total[2] + total[3];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();   // the wave counts are complete as well
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  int first = base + incl - sum, run[kEach];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    const int i = tid * kEach + q;
    if (seg == 0 && i < (int)span) {
      start[lo + i] = first;
      if ((int64_t)lo + i == V - 1) start[V] = first + total[q];
    }
    run[q] = first + before[q];
    first += total[q];
  }
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    int4* const at = reinterpret_cast<int4*>(n[w]) + tid;
    const int4 c = *at;
    *at = make_int4(run[0], run[1], run[2], run[3]);
    add(run, c);
  }
  __syncthreads();
  for (int t = t0; t < end; t += kGroups * 64) {
    load(t);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const uint32_t i = v[k] - lo;
      const bool in = i < span;
      uint64_t same = __ballot(in);
      if (same == 0) continue;
      // lanes with this lane's id, by one ballot a bit
#pragma unroll
      for (int b = 0; b < kIdBits; ++b) {
        const bool bit = (i >> b) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1));
      if (in) sorted[n[wave][i] + rank] = make_int2(t + k * 64 + lane, (int)v[k]);
      wave_sync();   // every lane has read its counter
      if (in && rank == 0) n[wave][i] += __popcll(same);
      wave_sync();
    }
  }
}

// Sums of runs.  The sorted tokens are cut into chunks; a team of threads sums
// a chunk's rows in order, VEC columns a thread, kAhead rows in flight.  A run
// inside one chunk goes to its row of the gradient.  A run that came from the
// chunk before leaves its part in parts[2 chunk], one that starts here and goes
// on in parts[2 chunk + 1]; embed_join_kernel adds those.  The workgroups past
// the chunks' clear the rows of ids that no token has, kClearRows each, so that
// these writes run beside the sums' reads.
constexpr int kAhead = 8, kClearRows = 16;

// VEC values of a row of dout; read once, so they need not stay in the caches
// (74 to 61 us for 16384 rows of 1600 beside the writes of 322 MB).
template <int VEC>
struct Row;
template <>
struct Row<8> {
  h8 x;
  __device__ __forceinline__ void load(const _Float16* p) { x = __builtin_nontemporal_load(reinterpret_cast<const h8u*>(p)); }
  __device__ __forceinline__ float at(int e) const { return (float)x[e]; }
};
template <>
struct Row<1> {
  _Float16 x;
  __device__ __forceinline__ void load(const _Float16* p) { x = *p; }
  __device__ __forceinline__ float at(int) const { return (float)x; }
};

// VEC values of fp32, 16 bytes at a time
template <int VEC>
__device__ __forceinline__ void load_sum(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const f4 x = *reinterpret_cast<const f4u*>(p), y = *reinterpret_cast<const f4u*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = x[e];
      v[4 + e] = y[e];
    }
  } else {
    v[0] = p[0];
  }
}
template <int VEC>
__device__ __forceinline__ void store_sum(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<f4u*>(p) = f4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f4u*>(p + 4) = f4{v[4], v[5], v[6], v[7]};
  } else {
    p[0] = v[0];
  }
}

// blockIdx.x: teams of chunks, then the rows to clear; blockIdx.y: slices of
// team * VEC columns.  With ADD the gradient's old values are loaded with the
// rows that end their runs: loaded at the end of each run, one after the other,
// they made up most of the kernel's time.
template <int VEC, bool ADD>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(const int2* __restrict__ sorted,
                                                             const int32_t* __restrict__ start,
                                                             const _Float16* __restrict__ dout, int64_t V, int64_t d,
                                                             float scale, int team, int chunk_tokens, int sum_blocks,
                                                             float* __restrict__ parts, float* __restrict__ dtable) {
  if ((int)blockIdx.x >= sum_blocks) {
    // kClearRows rows are one run of memory that starts 64-byte aligned, whatever
    // the width: zeros in 16-byte pieces, an element at a time only where a piece
    // holds entries of two rows
    __shared__ bool absent[kClearRows + 1];
    const int64_t v0 = (int64_t)(blockIdx.x - sum_blocks) * kClearRows;
    const int rows = (int)min<int64_t>(kClearRows, V - v0);
    if (threadIdx.x <= kClearRows) absent[threadIdx.x] = (int)threadIdx.x < rows && start[v0 + threadIdx.x] == start[v0 + threadIdx.x + 1];
    __syncthreads();
    float* const to = dtable + v0 * d;
    const uint32_t width = (uint32_t)d, entries = (uint32_t)rows * width, pieces = (entries + 3) / 4;
    const uint32_t first = (uint32_t)((uint64_t)pieces * blockIdx.y / gridDim.y), last = (uint32_t)((uint64_t)pieces * (blockIdx.y + 1) / gridDim.y);
    for (uint32_t i = first + threadIdx.x; i < last; i += kThreads) {
      const uint32_t r = 4 * i / width, r3 = (4 * i + 3) / width;   // past the last row: kClearRows or a row that is not there
      if (r == r3) {
        if (absent[r]) *reinterpret_cast<f4*>(to + 4 * i) = f4{};
      } else {
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const uint32_t re = (4 * i + e) / width;
          if (re < (uint32_t)rows && absent[re]) to[4 * i + e] = 0.0f;
        }
      }
    }
    return;
  }
  const int total = start[V];
  const int64_t chunk = (int64_t)blockIdx.x * (kThreads / team) + threadIdx.x / team;
  const int64_t mine = ((int64_t)blockIdx.y * team + threadIdx.x % team) * VEC, col = min<int64_t>(mine, d - VEC);
  const int shared = (int)(mine - col);   // columns that the thread before has too
  const int64_t p0 = chunk * chunk_tokens;
  if (p0 >= total || mine >= d) return;
  const int count = (int)min<int64_t>(chunk_tokens, total - p0);
  const int id_before = p0 > 0 ? sorted[p0 - 1].y : -1, id_after = p0 + count < total ? sorted[p0 + count].y : -1;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
  int2 at[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) at[k] = sorted[p0 + min(k, count - 1)];
  bool head = at[0].y == id_before;   // in a run that came from the chunk before
  for (int i = 0; i < count; i += kAhead) {
    Row<VEC> v[kAhead];
    float old[ADD ? kAhead : 1][VEC];
    int ids[kAhead + 1];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      v[k].load(dout + (int64_t)at[k].x * d + col);
      ids[k] = at[k].y;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) at[k] = sorted[p0 + min(i + kAhead + k, count - 1)];
    ids[kAhead] = at[0].y;
    bool ends[kAhead];   // row i + k is its run's last, or the chunk's
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      ends[k] = i + k + 1 >= count || ids[k + 1] != ids[k];
      if (ADD && ends[k] && i + k < count) load_sum<VEC>(dtable + (int64_t)ids[k] * d + col, old[ADD ? k : 0]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= count) break;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[k].at(e);
      if (!ends[k]) continue;
      if (head) {
        store_sum<VEC>(parts + 2 * chunk * d + col, acc);
      } else if (i + k + 1 >= count && ids[k] == id_after) {
        store_sum<VEC>(parts + (2 * chunk + 1) * d + col, acc);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = ADD ? old[ADD ? k : 0][e] + acc[e] * scale : acc[e] * scale;
        float* const to = dtable + (int64_t)ids[k] * d + col;
        if (!ADD || shared == 0) {
          store_sum<VEC>(to, acc);
        } else {   // its neighbour's columns are added to once
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e >= shared) to[e] = acc[e];
        }
      }
      head = false;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
    }
  }
}

// Of the chunk in which a run that goes on has started, adds up the run's
// parts: every wave takes every kJoinWaves-th part after the first, in order,
// and the waves' sums are added in theirs.  256 columns a workgroup.
constexpr int kJoinWaves = 8;
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(const int2* __restrict__ sorted,
                                                                     const int32_t* __restrict__ start, int64_t V,
                                                                     int64_t d, float scale, int chunk_tokens, int add,
                                                                     const float* __restrict__ parts,
                                                                     float* __restrict__ dtable) {
  __shared__ float sums[kJoinWaves][256];
  const int total = start[V];
  const int64_t chunk = blockIdx.x, last = (chunk + 1) * chunk_tokens - 1;
  if (last + 1 >= total) return;
  const int id = sorted[last].y;
  if (sorted[last + 1].y != id || start[id] < chunk * chunk_tokens) return;
  const int64_t end = (start[id + 1] - 1) / chunk_tokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.y * 256 + lane;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto part = [&](int64_t row, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = c0 + 64 * e < d ? parts[row * d + c0 + 64 * e] : 0.0f;
  };
  if (wave == 0) part(2 * chunk + 1, v);
#pragma unroll 4
  for (int64_t k = chunk + 1 + wave; k <= end; k += kJoinWaves) {
    float x[4];
    part(2 * k, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[wave][lane + 64 * e] = v[e];
  __syncthreads();
  const int c = threadIdx.x;
  const int64_t col = (int64_t)blockIdx.y * 256 + c;
  if (c >= 256 || col >= d) return;
  float s = sums[0][c];
#pragma unroll
  for (int w = 1; w < kJoinWaves; ++w) s += sums[w][c];
  s *= scale;
  float* o = dtable + (int64_t)id * d + col;
  *o = add ? *o + s : s;
}

struct BwdPlan {
  int64_t ranges, segs, seg_tokens, chunk_tokens, chunks;
  int64_t cnt, below, start, sorted, parts, bytes;   // byte offsets in the workspace
};

BwdPlan bwd_plan(int64_t T, int64_t V, int64_t d) {
  BwdPlan p;
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  p.ranges = (V + kRange - 1) / kRange;
  const int64_t unit = 64 * kWaves;
  p.seg_tokens = (T + kMaxSegs * unit - 1) / (kMaxSegs * unit) * unit;
  if (p.seg_tokens < kMinSeg) p.seg_tokens = kMinSeg;
  p.segs = T == 0 ? 1 : (T + p.seg_tokens - 1) / p.seg_tokens;
  // shorter chunks where there are few: 517 tokens' sums wait for 16 rows each,
  // not for 64; longer ones leave fewer parts to join
  p.chunk_tokens = T >= 65536 ? 64 : T >= 8192 ? 32 : 16;
  p.chunks = (T + p.chunk_tokens - 1) / p.chunk_tokens;
  p.cnt = 0;
  p.below = p.cnt + up(p.segs * p.ranges * kRange * 4);
  p.start = p.below + up(p.segs * p.ranges * 4);
  p.sorted = p.start + up((V + 1) * 4);
  p.parts = p.sorted + up(T * 8);
  p.bytes = p.parts + up(2 * p.chunks * d * 4);
  return p;
}

template <typename Id>
hipError_t launch_bwd(const Id* ids, int64_t T, const _Float16* dout, int64_t V, int64_t d, float scale, bool add,
                      float* dtable, unsigned char* ws, hipStream_t s) {
  const BwdPlan p = bwd_plan(T, V, d);
  int32_t* cnt = reinterpret_cast<int32_t*>(ws + p.cnt);
  int32_t* below = reinterpret_cast<int32_t*>(ws + p.below);
  int32_t* start = reinterpret_cast<int32_t*>(ws + p.start);
  int2* sorted = reinterpret_cast<int2*>(ws + p.sorted);
  float* parts = reinterpret_cast<float*>(ws + p.parts);
  const dim3 grid((unsigned)p.ranges, (unsigned)p.segs);
  if (T <= kSelfCount) {
    hipLaunchKernelGGL((embed_place_kernel<Id, true>), grid, dim3(kSortThreads), 0, s, ids, (int)T, V, (int)p.seg_tokens, nullptr, nullptr,
                       start, sorted);
  } else {
    hipLaunchKernelGGL((embed_count_kernel<Id>), grid, dim3(kSortThreads), 0, s, ids, (int)T, V, (int)p.seg_tokens, cnt, below);
    hipLaunchKernelGGL((embed_place_kernel<Id, false>), grid, dim3(kSortThreads), 0, s, ids, (int)T, V, (int)p.seg_tokens, cnt, below, start,
                       sorted);
  }
  const int vec = d >= 8 ? 8 : 1;
  int team = 8;
  while (team < kThreads && team * vec < d) team *= 2;
  const int sum_blocks = (int)((p.chunks + kThreads / team - 1) / (kThreads / team));
  const int64_t clear_blocks = add ? 0 : (V + kClearRows - 1) / kClearRows;
  const dim3 sums((unsigned)(sum_blocks + clear_blocks), (unsigned)((d + team * vec - 1) / (team * vec)));
  const int chunk = (int)p.chunk_tokens;
  auto sum = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, sums, dim3(kThreads), 0, s, sorted, start, dout, V, d, scale, team, chunk, sum_blocks, parts,
                       dtable);
  };
  if (vec == 8)
    add ? sum(embed_sum_kernel<8, true>) : sum(embed_sum_kernel<8, false>);
  else
    add ? sum(embed_sum_kernel<1, true>) : sum(embed_sum_kernel<1, false>);
  if (p.chunks > 1)
    hipLaunchKernelGGL(embed_join_kernel, dim3((unsigned)(p.chunks - 1), (unsigned)((d + 255) / 256)), dim3(64 * kJoinWaves),
                       0, s, sorted, start, V, d, scale, chunk, (int)add, parts, dtable);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const void* ids, bool ids64, const void* table, bool table32, int64_t T, int64_t V, int64_t d,
                            float scale, uint16_t* out, hipStream_t s) {
  if (table32)
    return ids64 ? launch_fwd<float, int64_t>(ids, table, T, V, d, scale, out, s)
                 : launch_fwd<float, int32_t>(ids, table, T, V, d, scale, out, s);
  return ids64 ? launch_fwd<_Float16, int64_t>(ids, table, T, V, d, scale, out, s)
               : launch_fwd<_Float16, int32_t>(ids, table, T, V, d, scale, out, s);
}

int64_t embed_bwd_workspace(int64_t T, int64_t V, int64_t d) { return bwd_plan(T, V, d).bytes; }

hipError_t launch_embed_bwd(const void* ids, bool ids64, int64_t T, const uint16_t* dout, int64_t V, int64_t d,
                            float scale, bool add, float* dtable, void* ws, hipStream_t s) {
  const _Float16* g = reinterpret_cast<const _Float16*>(dout);
  unsigned char* w = static_cast<unsigned char*>(ws);
  return ids64 ? launch_bwd<int64_t>(static_cast<const int64_t*>(ids), T, g, V, d, scale, add, dtable, w, s)
               : launch_bwd<int32_t>(static_cast<const int32_t*>(ids), T, g, V, d, scale, add, dtable, w, s);
}

}  // namespace sp24
