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
// ids.  No atomics on floating point, no dense [T, V] anything.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kItems = 4;   // row chunks per thread of the forward: that many gathers in flight

template <typename T>
__device__ __forceinline__ void load_row8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load_row8<_Float16>(const _Float16* p, float (&v)[8]) {
  const h8 x = *reinterpret_cast<const h8*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
}
template <>
__device__ __forceinline__ void load_row8<float>(const float* p, float (&v)[8]) {
  const f4 x = *reinterpret_cast<const f4*>(p), y = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = x[e];
    v[4 + e] = y[e];
  }
}

// A row is d / VEC chunks; a workgroup takes kThreads * kItems consecutive
// chunks of the flattened [T, d / VEC] output.
template <typename Table, typename Id, int VEC>
__global__ __launch_bounds__(kThreads) void embed_fwd_kernel(const Id* __restrict__ ids, const Table* __restrict__ table,
                                                              int64_t T, int64_t V, int64_t d, float scale,
                                                              _Float16* __restrict__ out) {
  const uint32_t chunks = (uint32_t)(d / VEC);
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kItems);
  const int64_t t0 = first / chunks;
  const uint32_t c0 = (uint32_t)(first - t0 * chunks);
  int64_t t[kItems], id[kItems];
  uint32_t c[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = c0 + threadIdx.x + k * kThreads;   // c0 < chunks <= 2^31
    const uint32_t q = i / chunks;
    t[k] = t0 + q;
    c[k] = i - q * chunks;
    id[k] = t[k] < T ? (int64_t)ids[t[k]] : -1;
  }
  float v[kItems][VEC];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[k][e] = 0.0f;
    if (id[k] >= 0 && id[k] < V) {
      const Table* row = table + id[k] * d + (int64_t)c[k] * VEC;
      if constexpr (VEC == 8)
        load_row8<Table>(row, v[k]);
      else
        v[k][0] = (float)row[0];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] *= scale;
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (t[k] >= T) continue;
    _Float16* o = out + t[k] * d + (int64_t)c[k] * VEC;
    if constexpr (VEC == 8) {
      h8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[k][e];
      *reinterpret_cast<h8*>(o) = h;
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
  const int vec = d % 8 == 0 ? 8 : 1;   // rows of other widths are not 16-byte aligned
  const int64_t items = T * (d / vec);
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
// tokens in at most kMaxSegs segments of a multiple of kSegStep.  A workgroup
// reads all ids of its segment and keeps those of its range; each wave has a
// contiguous part of the segment and its own counters, so that tokens of one
// id are placed in token order.
//   count: cnt[seg][v] and below[seg][range], the segment's tokens of each id
//          and with ids below the range
//   place: start[v], where id v's run begins in sorted order, and
//          sorted[p] = (token, id)
constexpr int kRange = 1024, kWaves = kRange / 64, kSegStep = 4096, kMaxSegs = 32;
constexpr int kGroups = kSegStep / kWaves / 64;   // groups of 64 tokens that a wave loads at once
static_assert(kGroups * kWaves * 64 == kSegStep, "whole waves of tokens");

// What one lane of a wave has written to LDS is read by the others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The id of token t relative to the range [lo, lo + kRange); -1 for one below
// it, kRange for one above or padding.
template <typename Id>
__device__ __forceinline__ int in_range(const Id* ids, int64_t t, int64_t end, int64_t lo, int64_t V) {
  if (t >= end) return kRange;
  const int64_t id = (int64_t)ids[t];
  if (id < 0 || id >= V) return kRange;
  if (id < lo) return -1;
  return id - lo < kRange ? (int)(id - lo) : kRange;
}

template <typename Id>
__global__ __launch_bounds__(kRange) void embed_count_kernel(const Id* __restrict__ ids, int64_t T, int64_t V,
                                                             int64_t seg_tokens, int32_t* __restrict__ cnt,
                                                             int32_t* __restrict__ below) {
  __shared__ int32_t n[kRange];
  __shared__ int32_t under;
  const int tid = threadIdx.x;
  const int64_t range = blockIdx.x, seg = blockIdx.y, lo = range * kRange;
  n[tid] = 0;
  if (tid == 0) under = 0;
  __syncthreads();
  const int64_t end = min<int64_t>((seg + 1) * seg_tokens, T);
  int mine = 0;
  for (int64_t t = seg * seg_tokens; t < end; t += kSegStep) {
#pragma unroll
    for (int k = 0; k < kSegStep / kRange; ++k) {
      const int v = in_range(ids, t + k * kRange + tid, end, lo, V);
      if (v >= 0 && v < kRange) atomicAdd(&n[v], 1);
      mine += __popcll(__ballot(v < 0));   // the wave's count, in every lane
    }
  }
  if ((tid & 63) == 0) atomicAdd(&under, mine);
  __syncthreads();
  cnt[(seg * gridDim.x + range) * kRange + tid] = n[tid];
  if (tid == 0) below[seg * gridDim.x + range] = under;
}

template <typename Id>
__global__ __launch_bounds__(kRange) void embed_place_kernel(const Id* __restrict__ ids, int64_t T, int64_t V,
                                                             int64_t seg_tokens, const int32_t* __restrict__ cnt,
                                                             const int32_t* __restrict__ below,
                                                             int32_t* __restrict__ start, int2* __restrict__ sorted) {
  __shared__ int32_t n[kWaves][kRange];   // counts of each wave's tokens, then where its next one goes
  __shared__ int32_t wave_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t range = blockIdx.x, seg = blockIdx.y, ranges = gridDim.x, segs = gridDim.y, lo = range * kRange;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) n[w][tid] = 0;
  __syncthreads();
  const int64_t per_wave = seg_tokens / kWaves;
  const int64_t t0 = seg * seg_tokens + wave * per_wave, end = min<int64_t>(t0 + per_wave, T);
  int v[kGroups];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < kGroups; ++k) v[k] = in_range(ids, t + k * 64 + lane, end, lo, V);
  };
  for (int64_t t = t0; t < end; t += kGroups * 64) {
    load(t);
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
      if (v[k] >= 0 && v[k] < kRange) atomicAdd(&n[wave][v[k]], 1);
  }
  // this thread's id over all segments, the earlier ones apart
  int total = 0, before = 0;
  for (int64_t s = 0; s < segs; ++s) {
    const int c = cnt[(s * ranges + range) * kRange + tid];
    total += c;
    if (s < seg) before += c;
  }
  int base = 0;
  for (int64_t s = 0; s < segs; ++s) base += below[s * ranges + range];
  // exclusive scan of the totals over the range's ids
  int incl = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();   // the wave counts are complete as well
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  const int first = base + incl - total;
  if (seg == 0 && lo + tid < V) {
    start[lo + tid] = first;
    if (lo + tid == V - 1) start[V] = first + total;
  }
  int run = first + before;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int c = n[w][tid];
    n[w][tid] = run;
    run += c;
  }
  __syncthreads();
  for (int64_t t = t0; t < end; t += kGroups * 64) {
    load(t);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const bool in = v[k] >= 0 && v[k] < kRange;
      uint64_t same = __ballot(in);
      if (same == 0) continue;
      // lanes with this lane's id, by one ballot a bit
#pragma unroll
      for (int b = 0; b < 10; ++b) {
        const bool bit = (v[k] >> b) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1));
      if (in) sorted[n[wave][v[k]] + rank] = make_int2((int)(t + k * 64 + lane), (int)(lo + v[k]));
      wave_sync();   // every lane has read its counter
      if (in && rank == 0) n[wave][v[k]] += __popcll(same);
      wave_sync();
    }
  }
}

// Sums of runs.  The sorted tokens are cut into chunks of kChunk; a team of
// threads sums a chunk's rows in order, kVec columns a thread.  A run inside
// one chunk goes to its row of the gradient.  A run that came from the chunk
// before leaves its part in head[chunk], one that starts here and goes on in
// tail[chunk]; embed_join_kernel adds those.
constexpr int kChunk = 64, kAhead = 8;

template <int VEC>
__device__ __forceinline__ void add_row(const _Float16* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const h8 x = *reinterpret_cast<const h8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
  } else {
    v[0] = (float)p[0];
  }
}

template <int VEC>
__device__ __forceinline__ void store_sum(float* p, const float (&v)[VEC], float scale, bool add) {
  if constexpr (VEC == 8) {
    f4 x, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = v[e] * scale;
      y[e] = v[4 + e] * scale;
    }
    if (add) {
      x += *reinterpret_cast<const f4*>(p);
      y += *reinterpret_cast<const f4*>(p + 4);
    }
    *reinterpret_cast<f4*>(p) = x;
    *reinterpret_cast<f4*>(p + 4) = y;
  } else {
    p[0] = add ? p[0] + v[0] * scale : v[0] * scale;
  }
}

// blockIdx.x: teams of chunks; blockIdx.y: slices of team * VEC columns
template <int VEC>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(const int2* __restrict__ sorted,
                                                             const int32_t* __restrict__ start,
                                                             const _Float16* __restrict__ dout, int64_t V, int64_t d,
                                                             float scale, int team, int add, float* __restrict__ parts,
                                                             float* __restrict__ dtable) {
  const int total = start[V];
  const int64_t chunk = (int64_t)blockIdx.x * (kThreads / team) + threadIdx.x / team;
  const int64_t col = ((int64_t)blockIdx.y * team + threadIdx.x % team) * VEC;
  const int64_t p0 = chunk * kChunk;
  if (p0 >= total || col >= d) return;
  const int count = (int)min<int64_t>(kChunk, total - p0);
  const bool from_before = p0 > 0 && sorted[p0 - 1].y == sorted[p0].y;
  const bool goes_on = p0 + count < total && sorted[p0 + count].y == sorted[p0 + count - 1].y;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
  int id = sorted[p0].y;
  bool first = true;   // still in the chunk's first run
  for (int i = 0; i < count; i += kAhead) {
    int2 at[kAhead];
    float v[kAhead][VEC];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) at[k] = sorted[p0 + min(i + k, count - 1)];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) add_row<VEC>(dout + (int64_t)at[k].x * d + col, v[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= count) break;
      if (at[k].y != id) {
        if (first && from_before)
          store_sum<VEC>(parts + (2 * chunk) * d + col, acc, 1.0f, false);
        else
          store_sum<VEC>(dtable + (int64_t)id * d + col, acc, scale, add != 0);
        first = false;
        id = at[k].y;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[k][e];
    }
  }
  if (first && from_before)
    store_sum<VEC>(parts + (2 * chunk) * d + col, acc, 1.0f, false);
  else if (goes_on)
    store_sum<VEC>(parts + (2 * chunk + 1) * d + col, acc, 1.0f, false);
  else
    store_sum<VEC>(dtable + (int64_t)id * d + col, acc, scale, add != 0);
}

// The chunk in which a run that goes on has started adds up its parts, in
// order.  One thread a column.
__global__ __launch_bounds__(kThreads) void embed_join_kernel(const int2* __restrict__ sorted,
                                                              const int32_t* __restrict__ start, int64_t V, int64_t d,
                                                              float scale, int add, const float* __restrict__ parts,
                                                              float* __restrict__ dtable) {
  const int total = start[V];
  const int64_t chunk = blockIdx.x, last = (chunk + 1) * kChunk - 1;
  if (last + 1 >= total) return;
  const int id = sorted[last].y;
  if (sorted[last + 1].y != id || start[id] < chunk * kChunk) return;
  const int64_t end = (start[id + 1] - 1) / kChunk;
  for (int64_t c = threadIdx.x; c < d; c += kThreads) {
    float v = parts[(2 * chunk + 1) * d + c];
    for (int64_t k = chunk + 1; k <= end; ++k) v += parts[2 * k * d + c];
    v *= scale;
    float* o = dtable + (int64_t)id * d + c;
    *o = add ? *o + v : v;
  }
}

// Rows of ids that no token has, kClearRows a workgroup.
constexpr int kClearRows = 16;
__global__ __launch_bounds__(kThreads) void embed_clear_kernel(const int32_t* __restrict__ start, int64_t V, int64_t d,
                                                               float* __restrict__ dtable) {
  const int64_t v0 = (int64_t)blockIdx.x * kClearRows, v1 = min<int64_t>(v0 + kClearRows, V);
  for (int64_t v = v0; v < v1; ++v) {
    if (start[v] != start[v + 1]) continue;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) dtable[v * d + c] = 0.0f;
  }
}

struct BwdPlan {
  int64_t ranges, segs, seg_tokens, chunks;
  int64_t cnt, below, start, sorted, parts, bytes;   // byte offsets in the workspace
};

BwdPlan bwd_plan(int64_t T, int64_t V, int64_t d) {
  BwdPlan p;
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  p.ranges = (V + kRange - 1) / kRange;
  p.seg_tokens = (T + (int64_t)kMaxSegs * kSegStep - 1) / ((int64_t)kMaxSegs * kSegStep) * kSegStep;
  if (p.seg_tokens == 0) p.seg_tokens = kSegStep;
  p.segs = T == 0 ? 1 : (T + p.seg_tokens - 1) / p.seg_tokens;
  p.chunks = (T + kChunk - 1) / kChunk;
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
  hipLaunchKernelGGL((embed_count_kernel<Id>), grid, dim3(kRange), 0, s, ids, T, V, p.seg_tokens, cnt, below);
  hipLaunchKernelGGL((embed_place_kernel<Id>), grid, dim3(kRange), 0, s, ids, T, V, p.seg_tokens, cnt, below, start,
                     sorted);
  if (T > 0) {
    const int vec = d % 8 == 0 ? 8 : 1;
    int team = 8;
    while (team < kThreads && team * vec < d) team *= 2;
    const dim3 sums((unsigned)((p.chunks + kThreads / team - 1) / (kThreads / team)),
                    (unsigned)((d + team * vec - 1) / (team * vec)));
    if (vec == 8)
      hipLaunchKernelGGL((embed_sum_kernel<8>), sums, dim3(kThreads), 0, s, sorted, start, dout, V, d, scale, team,
                         (int)add, parts, dtable);
    else
      hipLaunchKernelGGL((embed_sum_kernel<1>), sums, dim3(kThreads), 0, s, sorted, start, dout, V, d, scale, team,
                         (int)add, parts, dtable);
    hipLaunchKernelGGL(embed_join_kernel, dim3((unsigned)p.chunks), dim3(kThreads), 0, s, sorted, start, V, d, scale,
                       (int)add, parts, dtable);
  }
  if (!add)
    hipLaunchKernelGGL(embed_clear_kernel, dim3((unsigned)((V + kClearRows - 1) / kClearRows)), dim3(kThreads), 0, s,
                       start, V, d, dtable);
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
