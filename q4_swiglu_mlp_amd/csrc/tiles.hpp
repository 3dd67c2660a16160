// What the tiled products share: buffer loads bounded by a tile's part of a matrix, copies straight to
// LDS, and the row tiles of grouped rows (offsets on the GPU, as zinc_moe_sort writes them).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace zinc {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Buffer loads bounded by a matrix's `bytes` from p: bytes behind them read as zero
// and touch no memory.
using Buffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buffer tile_buffer(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00020000);
}
// Sixteen bytes a lane to LDS, lane after lane from dst.
__device__ __forceinline__ void to_lds(Buffer b, int off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}
// A bounded buffer as its four words (the same for the wave).
__device__ __forceinline__ i32x4_t buffer_words(const uint8_t* p, int bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
// to_lds out of the compiler's sight, which would wait for all copies before every transposing read: whoever
// reads the tile waits for them by count.  (m0 is for such copies alone on gfx950; a kernel has them of one kind.)
__device__ __forceinline__ void copy_to_lds(i32x4_t b, int off, const uint8_t* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)dst;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(b), "s"(__builtin_amdgcn_readfirstlane(at)));
}
__device__ __forceinline__ i32x4_t load_piece(Buffer b, int off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
}

// The rows [first, first + rows) of tile `tile` (TM rows each) of the experts'
// row ranges, and its expert; rows <= 0 past the last tile.  Offsets outside
// [0, total] or not ascending are cut to that range.
struct RowTile {
  int expert, first, rows;
};

template <int TM>
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ offsets, int E, int total, int tile) {
  if (!offsets) return {0, tile * TM, min(TM, total - tile * TM)};
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = e < E ? min(max(offsets[e], 0), total) : 0;
    const int hi = e < E ? min(max(offsets[e + 1], lo), total) : 0;
    const int n = (hi - lo + TM - 1) / TM;
    int scan = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(scan, d, 64);
      if (lane >= d) scan += o;
    }
    const uint64_t here = __ballot(seen + scan > tile);
    if (here) {
      const int l = (int)__builtin_ctzll(here);
      const int before = seen + __builtin_amdgcn_readlane(scan - n, l);
      const int first = __builtin_amdgcn_readlane(lo, l) + (tile - before) * TM;
      return {e0 + l, first, min(TM, __builtin_amdgcn_readlane(hi, l) - first)};
    }
    seen += __builtin_amdgcn_readlane(scan, 63);
  }
  return {0, 0, 0};
}

// Row tiles a grouped product can have: every expert's last one may be partly filled.
inline long long max_row_tiles(long long rows, int experts, int TM) {
  return experts ? (rows + TM - 1) / TM + (experts < rows ? experts : rows) : (rows + TM - 1) / TM;
}

// Row tiles of all experts, and the tables; offsets are cut to [0, M] and, where
// they do not ascend, the range is empty.
template <int TM, typename ARGS>
__device__ __forceinline__ int make_tables(const ARGS& g, int32_t* starts, int32_t* ends) {
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = e < g.E ? min(max(g.offsets[e], 0), g.M) : 0;
    const int hi = e < g.E ? min(max(g.offsets[e + 1], lo), g.M) : 0;
    const int n = (hi - lo + TM - 1) / TM;
    int scan = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(scan, d, 64);
      if (lane >= d) scan += o;
    }
    if (threadIdx.x < 64 && e < g.E) {
      starts[e] = lo;
      if (e == g.E - 1) starts[g.E] = hi;
      ends[e] = seen + scan;
    }
    seen += __builtin_amdgcn_readlane(scan, 63);
  }
  return seen;
}

// Row tile mt by those tables: its expert and rows, into r.
template <int TM, typename ARGS, typename UNIT>
__device__ __forceinline__ void tile_rows(const ARGS& g, const int32_t* starts, const int32_t* ends, int mt, UNIT& r) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    const int end = e < g.E ? ends[e] : 0x7FFFFFFF;
    const uint64_t here = __ballot(end > mt);
    if (here) {
      r.expert = e0 + (int)__builtin_ctzll(here);
      break;
    }
  }
  r.expert = __builtin_amdgcn_readfirstlane(r.expert);
  const int before = r.expert ? ends[r.expert - 1] : 0, lo = starts[r.expert];
  r.first = __builtin_amdgcn_readfirstlane(lo + (mt - before) * TM);
  r.rows = __builtin_amdgcn_readfirstlane(min(TM, max(lo, starts[r.expert + 1]) - r.first));
}

// Raises the kernel's LDS limit, once a device.  The kernel itself is the argument, so that no two share a flag.
template <auto KERNEL>
hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> ready{0};   // devices whose limit is raised
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

constexpr int kLds = 160 * 1024;

// Compute units of the current device (looked up once a device).
inline hipError_t compute_units(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  *n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*n) return hipSuccess;
  e = hipDeviceGetAttribute(n, hipDeviceAttributeMultiprocessorCount, dev);
  if (e == hipSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}

}  // namespace zinc
