// What the kernels share that run the 2:4 sparse products' fast path
// (sp24_spmm.hip, sp24_linear.hip): the tile's geometry and its LDS layouts.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "sp24_device.hpp"
#include "sp24_internal.hpp"

namespace sp24 {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16 __attribute__((ext_vector_type(16)));
typedef float f16v __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Fast path (K a multiple of 64, every operand below 2 GiB).
//
// Workgroup tile BM features x BN tokens in waves of WM x WN (launched as
// 256 x 256 with 8 waves of 128 x 64, two waves per SIMD).  A 3-stage LDS ring is filled by direct global->LDS buffer
// loads (no VGPR round trip), two stages ahead of the one being computed, so
// HBM/L2 latency hides behind two stages of MFMA work.  Rows past N or T read
// as zero (buffer bounds); they only feed outputs that are not stored.
//
// LDS layouts (per stage), both XOR-swizzled so that ds_read_b128 is free of
// bank conflicts for 8- and 16-lane groups:
//   S  [BM rows][4 chunks of 16 B]: chunk c of row r at slot c ^ fS(r)
//   B  [BN rows][8 chunks of 16 B]: chunk c of row r at slot c ^ fB(r)
//   meta [BM rows][2 dwords]
// A direct load writes 64 consecutive 16-byte LDS slots, one per lane, so each
// lane fetches the global chunk whose swizzled slot is its own lane index.

__device__ __forceinline__ int swz_s(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }
__device__ __forceinline__ int swz_b(int r) { return (r & 7) ^ ((r >> 3) & 1); }

template <int BM, int BN, int WM, int WN>
struct FastCfg {
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN;
  static constexpr int WAVES = WAVES_M * WAVES_N;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int TM = WM / 32, TN = WN / 32;
  static constexpr int S_BYTES = BM * 64, B_BYTES = BN * 128, M_BYTES = BM * 8;
  static constexpr int S_LOADS = S_BYTES / 1024 / WAVES;   // 16-byte direct loads per wave per stage
  static constexpr int B_LOADS = B_BYTES / 1024 / WAVES;
  static constexpr int M_LOADS = M_BYTES / 256 / WAVES;    // 4-byte direct loads
  static constexpr int LOADS = S_LOADS + B_LOADS + M_LOADS;
  static_assert(S_BYTES % (1024 * WAVES) == 0 && B_BYTES % (1024 * WAVES) == 0 && M_BYTES % (256 * WAVES) == 0,
                "tile does not split evenly into direct loads");
  static_assert(LOADS <= 63, "vmcnt range");
};

}  // namespace
}  // namespace sp24
