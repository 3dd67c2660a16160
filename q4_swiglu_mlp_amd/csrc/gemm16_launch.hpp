// How a 16-bit product by expert is cut, by its sizes alone, and its launches.
#pragma once

#include "gemm16_tile.hpp"
#include "launch.hpp"

namespace zinc {

constexpr size_t kQueueBytes = 8 * 32 * 4;

// The tiles, with the workgroups of each that a CU holds, and what a step of 64 takes a CU in us: one
// workgroup alone, and each of as many as it holds (dense 8192 x 4096 x 4096: 265, 267, 274 and 336 us;
// 2331 rows of 7 experts, 520 x 1032, 17 steps: 29, 19, 16 and 12).
struct Gemm16Shape {
  int TM, TN, held;
  double alone, full;
};
constexpr Gemm16Shape kGemm16Shapes[] = {
    {256, 256, 1, 1.5, 1.85}, {128, 256, 1, 0.9, 1.04}, {128, 128, 2, 0.72, 0.56}, {64, 128, 3, 0.47, 0.33}};

struct Gemm16Plan {
  int shape, splits;
  bool queue;        // the units are more than the CUs hold at once, and uneven
  size_t part;       // values from one part of the summed dimension to the next
};

// The cut with the least time by the figures above: rounds of units times their steps, and for more than one
// part of the summed dimension 3 us for the launch that joins them and its traffic at 4 TB/s.  An expert's
// last row tile counts as half full.  (Experts of uneven sizes: as if they were even.)
inline Gemm16Plan plan_gemm16(Product f, int M, int E, int N, int K, int cus = 256) {
  const int used = E < M ? E : (M ? M : 1);
  const double out = f == kForward ? (double)M * N : f == kInput ? (double)M * K : (double)E * N * K;
  const int steps = f == kWeight ? (M / used + 95) / 64 : ((f == kForward ? K : N) + 63) / 64;
  Gemm16Plan best{3, 1, false, 0};
  double least = 1e30;
  for (int i = 0; i < 4; ++i) {
    const Gemm16Shape& s = kGemm16Shapes[i];
    const int cols = f == kForward ? N : K, col_tiles = (cols + s.TN - 1) / s.TN;
    const double row_tiles = f == kWeight ? (double)E * ((N + s.TM - 1) / s.TM)
                                          : (M <= used ? M : (double)M / s.TM + 0.5 * used > used ? (double)M / s.TM + 0.5 * used : used);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      const int each = (steps + splits - 1) / splits;
      if (splits > 1 && (each < 4 || (steps + each - 1) / each != splits || splits * out > (1 << 25))) continue;
      const double units = row_tiles * col_tiles * splits, a_cu = units / cus;
      const int at_once = a_cu >= s.held ? s.held : a_cu <= 1 ? 1 : (int)(a_cu + 0.999);
      const double step = s.full * at_once > s.alone ? s.full * at_once : s.alone;
      double rounds = units / (cus * (double)at_once);
      rounds = rounds <= 1 ? 1 : (double)(long long)(rounds + 0.95);
      const double us = rounds * (each + 2) * step + (splits > 1 ? 3 + splits * out * 8 / 4e6 : 0);
      if (us < least) {
        least = us;
        best = {i, splits, units > 1.5 * cus * s.held && i < 2, ((size_t)out + 7) / 8 * 8};
      }
    }
  }
  if (best.splits > 1) best.queue = false;
  return best;
}
inline size_t gemm16_part_bytes(const Gemm16Plan& p) { return p.splits > 1 ? p.splits * p.part * sizeof(float) : 0; }

// The queues' first numbers, behind the units that the workgroups start with.
static __global__ void k_gemm16_queue(int32_t* queue, int first) { queue[32 * threadIdx.x] = first; }

// As many persistent workgroups as the CUs hold, a multiple of the eight XCDs.
template <typename KERNEL>
hipError_t gemm16_grid(const Gemm16Args& g, const void* kernel, int shape, unsigned* grid, int* bytes) {
  *bytes = (int)KERNEL::smem_bytes(g.E);
  hipError_t e = allow_lds<KERNEL>(kernel, kLds);
  int cus = 0;
  if (e == hipSuccess) e = compute_units(&cus);
  if (e != hipSuccess) return e;
  const int cols = KERNEL::kProduct == kForward ? g.N : g.K, TM = kGemm16Shapes[shape].TM;
  const long long row_tiles =
      KERNEL::kProduct == kWeight ? (long long)g.E * ((g.N + TM - 1) / TM) : max_row_tiles(g.M, g.E, TM);
  const int held = kLds / *bytes < KERNEL::HELD ? kLds / *bytes : KERNEL::HELD, TN = kGemm16Shapes[shape].TN;
  const long long units = row_tiles * ((cols + TN - 1) / TN) * g.splits, room = (long long)cus * held;
  const long long blocks = units < room ? units : room;
  *grid = (unsigned)((blocks + 7) / 8 * 8);
  return hipSuccess;
}

template <typename KERNEL>
hipError_t run_gemm16(const Gemm16Args& g, int shape, hipStream_t stream) {
  unsigned grid = 0;
  int bytes = 0;
  hipError_t e = gemm16_grid<KERNEL>(g, reinterpret_cast<const void*>(&k_gemm16<KERNEL>), shape, &grid, &bytes);
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
  return run_gemm16<Gemm16<F, 64, 128, 1, 4, 2, T, O>>(g, 3, stream);
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
