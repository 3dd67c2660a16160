// The launches of a 16-bit product by expert.
#pragma once

#include "gemm16_plan.hpp"
#include "gemm16_tile.hpp"
#include "launch.hpp"

namespace zinc {

// The queues' first numbers, behind the units that the workgroups start with.
static __global__ void k_gemm16_queue(int32_t* queue, int first) { queue[32 * threadIdx.x] = first; }

// As many persistent workgroups as the CUs hold, a multiple of the eight XCDs.
template <typename KERNEL>
unsigned gemm16_blocks(const Gemm16Args& g, int shape, int cus) {
  const int bytes = (int)KERNEL::smem_bytes(g.E), TM = kGemm16Shapes[shape].TM, TN = kGemm16Shapes[shape].TN;
  const int cols = KERNEL::kProduct == kForward ? g.N : g.K;
  const long long row_tiles =
      KERNEL::kProduct == kWeight ? (long long)g.E * ((g.N + TM - 1) / TM) : max_row_tiles(g.M, g.E, TM);
  const int held = kLds / bytes < KERNEL::HELD ? kLds / bytes : KERNEL::HELD;
  const long long units = row_tiles * ((cols + TN - 1) / TN) * g.splits, room = (long long)cus * held;
  return (unsigned)(((units < room ? units : room) + 7) / 8 * 8);
}

// The launch's grid and LDS, whose limit is raised for FUNCTION (KERNEL's kernel, or one that KERNEL stands for).
template <typename KERNEL, auto FUNCTION>
hipError_t gemm16_grid(const Gemm16Args& g, int shape, unsigned* grid, int* bytes) {
  *bytes = (int)KERNEL::smem_bytes(g.E);
  hipError_t e = allow_lds<FUNCTION>(kLds);
  int cus = 0;
  if (e == hipSuccess) e = compute_units(&cus);
  if (e != hipSuccess) return e;
  *grid = gemm16_blocks<KERNEL>(g, shape, cus);
  return hipSuccess;
}

template <typename KERNEL>
hipError_t run_gemm16(const Gemm16Args& g, int shape, hipStream_t stream) {
  unsigned grid = 0;
  int bytes = 0;
  hipError_t e = gemm16_grid<KERNEL, &k_gemm16<KERNEL>>(g, shape, &grid, &bytes);
  if (e != hipSuccess) return e;
  if (g.queue) {
    hipLaunchKernelGGL(k_gemm16_queue, dim3(1), dim3(8), 0, stream, g.queue, (int)grid / 8);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  timing_begin(stream);
  hipLaunchKernelGGL(k_gemm16<KERNEL>, dim3(grid), dim3(KERNEL::THREADS), bytes, stream, g);
  timing_end(stream);
  return hipGetLastError();
}

template <Product F, typename T, typename O>
hipError_t run_gemm16(const Gemm16Args& g, int shape, hipStream_t stream) {
  if (shape == 0) return run_gemm16<Gemm16<F, 256, 256, 2, 4, 2, T, O>>(g, 0, stream);
  if (shape == 1) return run_gemm16<Gemm16<F, 128, 256, 2, 4, 3, T, O>>(g, 1, stream);
  if (shape == 2) return run_gemm16<Gemm16<F, 128, 128, 2, 2, 2, T, O>>(g, 2, stream);
  return run_gemm16<Gemm16<F, 64, 128, 1, 4, F == kForward ? 3 : 2, T, O>>(g, 3, stream);
}

// f(T, O) for the type codes of the operands (0 fp16, 1 bf16) and of the output (the same, or 2 fp32).
template <typename F>
hipError_t by_types(int type, int out_type, F f) {
  if (type == 0) return out_type == 2 ? f(_Float16{}, 0.0f) : f(_Float16{}, _Float16{});
  return out_type == 2 ? f(__bf16{}, 0.0f) : f(__bf16{}, __bf16{});
}

// c = the sum of the parts of the summed dimension, in their order, for the rows inside the experts' ranges
// (offsets null: for all `total` values).
template <typename O>
__global__ __launch_bounds__(256) void k_gemm16_join(const float* __restrict__ parts, size_t part, int splits,
                                                     const int32_t* __restrict__ offsets, int E, int M, int cols,
                                                     size_t total, O* __restrict__ c) {
  size_t from = 0;
  if (offsets) {
    const int lo = min(max(offsets[0], 0), M), hi = min(max(offsets[E], lo), M);
    from = (size_t)lo * cols;
    total = (size_t)hi * cols;
  }
  for (size_t i = from + ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total; i += (size_t)gridDim.x * 1024) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(parts + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(parts + s * part + i);
    typedef O O4 __attribute__((ext_vector_type(4)));
    O4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (O)v[r];
    *reinterpret_cast<O4*>(c + i) = o;
  }
}

// The whole product: one launch, or the parts and their sum.  ws: the queue, then the parts.
template <Product F>
hipError_t launch_gemm16(const void* p, const void* q, int type, const int32_t* offsets, int E, int M, int N, int K,
                         int out_type, void* c, void* ws, hipStream_t stream) {
  const Gemm16Plan plan = plan_gemm16(F, M, E, N, K);
  Gemm16Args g{p, q, offsets, E, M, N, K, c, plan.splits, plan.part, plan.queue ? static_cast<int32_t*>(ws) : nullptr};
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kQueueBytes);
  if (plan.splits > 1) g.c = parts;
  hipError_t e = by_types(type, plan.splits > 1 ? 2 : out_type, [&](auto t, auto o) {
    return run_gemm16<F, decltype(t), decltype(o)>(g, plan.shape, stream);
  });
  if (e != hipSuccess || plan.splits == 1) return e;
  return by_types(type, out_type, [&](auto, auto o) {
    using O = decltype(o);
    const int cols = F == kForward ? N : K;
    const size_t total = F == kWeight ? (size_t)E * N * K : (size_t)M * cols, blocks = (total + 1023) / 1024;
    hipLaunchKernelGGL(k_gemm16_join<O>, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream, parts,
                       plan.part, plan.splits, F == kWeight ? nullptr : offsets, E, M, cols, total,
                       static_cast<O*>(c));
    return hipGetLastError();
  });
}

}  // namespace zinc
