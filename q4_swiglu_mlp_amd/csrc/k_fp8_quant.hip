// Block quantiser to e4m3 (fp8_device.hpp has the arithmetic): one scale per
// row and 128 columns, or per 128 x 128 tile; rows may be written to the
// places an expert sort gives them (the FP8 gather).
//
// Bound by HBM: one read of x, one write of q.  A row's block is 16 lanes of
// eight values, so its maximum is four DPP steps and x is read once.  Measured, bf16, input and
// output in HBM: 11008 x 4096 by tiles 29 us into a fresh output, 32.6 over outputs in turn (4.2 TB/s;
// a large copy 5.2), rows of 8192 x 4096 23 us (4.4), 4096 x 2048 to eight places each 17.3 us (4.9).
// On the tensors of the call before, in the last-level cache: 24, 18 and 15 us.  A few rows cost a
// launch, 2.3 us.
#include "fp8_device.hpp"
#include "launch.hpp"

namespace zinc {
namespace {

// One 16-lane group per (row, block of 128 columns).  GATHER: row t goes to
// rows slot_row[t * top_k + s] (values outside [0, M * top_k) are skipped).
template <typename T, bool GATHER>
__global__ __launch_bounds__(256) void k_quant_rows(const T* __restrict__ x, long long groups, int C, int nblk,
                                                    const int32_t* __restrict__ slot_row, int top_k, int n_rows,
                                                    uint8_t* __restrict__ q, float* __restrict__ scales) {
  const int l = threadIdx.x & 15;
  for (long long g = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); g < groups; g += (long long)gridDim.x * 16) {
    const long long r = g / nblk;
    const int b = (int)(g - r * nblk);
    const int c = b * 128 + l * 8;
    float v[8] = {};
    if (c < C) load8(x + r * C + c, v);
    bool whole;
    const uint32_t f = scale_field(max16(max_finite(v, whole)));
    const uint2 w = to_e4m3(v, inverse_scale_of(f), whole);
    if constexpr (GATHER) {
      for (int s0 = 0; s0 < top_k; s0 += 8) {
        int row[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) row[s] = s0 + s < top_k ? slot_row[r * top_k + s0 + s] : -1;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if ((unsigned)row[s] >= (unsigned)n_rows) continue;
          if (c < C) *reinterpret_cast<uint2*>(q + (long long)row[s] * C + c) = w;
          if (l == 0) scales[(long long)row[s] * nblk + b] = scale_of(f);
        }
      }
    } else {
      if (c < C) *reinterpret_cast<uint2*>(q + r * C + c) = w;
      if (l == 0) scales[r * nblk + b] = scale_of(f);
    }
  }
}

// One workgroup per 128 x 128 tile, neighbours along a row block (tiles past 2^22 in
// turn); a thread holds eight columns of eight rows.
template <typename T>
__global__ __launch_bounds__(256) void k_quant_tiles(const T* __restrict__ x, int R, int C, int nblk,
                                                     uint8_t* __restrict__ q, float* __restrict__ scales) {
  __shared__ uint32_t part[4];
  const long long tiles = ((long long)R + 127) / 128 * nblk;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long rb = tile / nblk;
    const int c = (int)(tile - rb * nblk) * 128 + (int)(threadIdx.x & 15) * 8;
    const long long r0 = rb * 128 + (threadIdx.x >> 4);
    float v[8][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long r = r0 + 16 * j;
      if (r < R && c < C) {
        load8(x + r * C + c, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      }
    }
    uint32_t m = 0;
    bool whole[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, max_finite(v[j], whole[j]));
    m = max16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    const uint32_t f = scale_field(max(max(part[0], part[1]), max(part[2], part[3])));
    const float inv = inverse_scale_of(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long r = r0 + 16 * j;
      if (r < R && c < C) *reinterpret_cast<uint2*>(q + r * C + c) = to_e4m3(v[j], inv, whole[j]);
    }
    if (threadIdx.x == 0) scales[tile] = scale_of(f);
    if (tile + gridDim.x < tiles) __syncthreads();   // part is read before it is written again
  }
}

// Workgroups of 16 groups of lanes; groups past 2^22 workgroups are taken in
// turn (a grid holds fewer than 2^32 threads).
dim3 group_grid(long long groups) {
  const long long b = (groups + 15) / 16;
  return dim3((unsigned)(b < (1 << 22) ? b : (1 << 22)));
}

template <typename T>
void rows(const void* x, int R, int C, const int32_t* slot_row, int top_k, uint8_t* q, float* scales,
          hipStream_t stream) {
  const int nblk = (C + 127) / 128;
  const long long groups = (long long)R * nblk;
  const dim3 grid = group_grid(groups);
  if (slot_row)
    hipLaunchKernelGGL((k_quant_rows<T, true>), grid, dim3(256), 0, stream, static_cast<const T*>(x), groups, C, nblk,
                       slot_row, top_k, R * top_k, q, scales);
  else
    hipLaunchKernelGGL((k_quant_rows<T, false>), grid, dim3(256), 0, stream, static_cast<const T*>(x), groups, C,
                       nblk, nullptr, 1, R, q, scales);
}

template <typename T>
void tiles(const void* x, int R, int C, uint8_t* q, float* scales, hipStream_t stream) {
  const int nblk = (C + 127) / 128;
  const long long n = ((long long)R + 127) / 128 * nblk;
  hipLaunchKernelGGL(k_quant_tiles<T>, dim3((unsigned)(n < (1 << 22) ? n : (1 << 22))), dim3(256), 0, stream,
                     static_cast<const T*>(x), R, C, nblk, q, scales);
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int type, int R, int C, int block_rows, void* q, float* scales,
                               hipStream_t stream) {
  uint8_t* qb = static_cast<uint8_t*>(q);
  if (block_rows == 1) {
    if (type == 0) rows<_Float16>(x, R, C, nullptr, 1, qb, scales, stream);
    if (type == 1) rows<__bf16>(x, R, C, nullptr, 1, qb, scales, stream);
    if (type == 2) rows<float>(x, R, C, nullptr, 1, qb, scales, stream);
  } else {
    if (type == 0) tiles<_Float16>(x, R, C, qb, scales, stream);
    if (type == 1) tiles<__bf16>(x, R, C, qb, scales, stream);
    if (type == 2) tiles<float>(x, R, C, qb, scales, stream);
  }
  return hipGetLastError();
}

hipError_t launch_moe_gather_fp8(const void* x, int type, int M, int top_k, int C, const int32_t* slot_row, void* q,
                                 float* scales, hipStream_t stream) {
  uint8_t* qb = static_cast<uint8_t*>(q);
  if (type == 0) rows<_Float16>(x, M, C, slot_row, top_k, qb, scales, stream);
  if (type == 1) rows<__bf16>(x, M, C, slot_row, top_k, qb, scales, stream);
  if (type == 2) rows<float>(x, M, C, slot_row, top_k, qb, scales, stream);
  return hipGetLastError();
}

}  // namespace zinc
