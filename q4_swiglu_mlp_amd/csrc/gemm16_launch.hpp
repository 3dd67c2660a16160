// How a 16-bit product by expert is cut, by its sizes alone, and its launches.
#pragma once

#include <cmath>

#include "gemm16_tile.hpp"
#include "launch.hpp"

namespace zinc {

constexpr size_t kQueueBytes = 8 * 32 * 4;

// The tiles: workgroups a CU holds, steps a unit has at least, and what a model of the time (us) takes: a step of
// 64 of one workgroup alone on a CU, a CU's time for one where it is full, the steps that a unit's beginning
// costs, and the TB/s at which the chip stores outputs.
struct Gemm16Shape {
  int TM, TN, held, least;
  double alone, full, begin, stores;
};
constexpr Gemm16Shape kGemm16Shapes[] = {{256, 256, 1, 3, 1.08, 0.49, 1.54, 5.2},
                                         {128, 256, 1, 4, 0.57, 0.96, 0.46, 6.1},
                                         {128, 128, 2, 3, 0.65, 0.51, 1.6, 4.7},
                                         {64, 128, 3, 3, 0.48, 0.34, 1.66, 7.7},
                                         {64, 128, 2, 4, 0.2, 0.4, 0.52, 3.8}};   // the last one's, of c: three buffers

struct Gemm16Plan {
  int shape, splits;
  bool queue;        // units dealt out as CUs fall free, for the launch that their queues cost
  size_t part;       // values from one part of the summed dimension to the next
  double us;         // the model's time
};

// Experts with rows, if any may have any.
inline double gemm16_used(int M, int E) { return M == 0 ? 1 : E * (1 - std::pow(1 - 1.0 / E, M)); }

// Parts of the summed dimension at most (of four steps, in dw of two of the mean expert's), and values in all of them
// (64 MB: of 300 drawn sizes with four times as many none took less).  With the rows neither falls.
constexpr double kPartValues = 1 << 24;
inline int gemm16_most_parts(Product f, int M, int E, int N, int K) {
  const double most = f == kWeight ? M / gemm16_used(M, E) / 128 : ((f == kForward ? K : N) + 63) / 64 / 4;
  return most < 1 ? 1 : most > 16 ? 16 : (int)most;
}
// A workspace's bytes for the parts of any product of up to M rows.
inline size_t gemm16_part_bytes(Product f, int M, int E, int N, int K) {
  const int parts = gemm16_most_parts(f, M, E, N, K);
  const double out = f == kForward ? (double)M * N : f == kInput ? (double)M * K : (double)E * N * K;
  return parts == 1 ? 0 : 4 * (size_t)(parts * out < kPartValues ? parts * out : kPartValues);
}

// The cut with the least time by a model fitted to 4388 timings: 90 products of 1 - 256 experts of uneven sizes, 1 -
// 30000 rows, each with its gradients, in every tile, in 1 - 16 parts, dealt out or not.  It is off by 17 % on average;
// what it picks takes 4 % more than the best on average (c 3.5 %, da 2 %, dw 5 %), 48 % in the worst of 360.
// Examples, us, in the order of the tiles, in one part: 32768 rows of 64 x 768 x 2048 124, 132, 150 and 171, dw in
// fp32 178, 191, 203 and 250; 2331 of 7 x 520 x 1032 31, 21, 19 and 13; 64 of 64 x 768 x 2048 49, 34, 38 and 32,
// and 27 in two parts of the last.  For 256 CUs.
// small: the smallest tile, in one part, dealt out in turn.
inline Gemm16Plan plan_gemm16(Product f, int M, int E, int N, int K, bool small = false) {
  constexpr int kCus = 256;
  const bool weight = f == kWeight;
  const int cols = f == kForward ? N : K;
  const double used = gemm16_used(M, E);
  const double out = f == kForward ? (double)M * N : f == kInput ? (double)M * K : (double)E * N * K;
  const double read = 2.0 * M * (f == kInput ? N : K) + (weight ? 2.0 * M * N : 2.0 * used * N * K);
  const double several = 1 - 1.0 / E;   // how far experts' sizes can differ
  const int parts = small ? 1 : gemm16_most_parts(f, M, E, N, K);
  Gemm16Plan best{3, 1, false, 0, 0};
  if (M == 0) return best;   // (dw of no rows)
  double least = 1e30;
  for (int i = small ? 3 : 0; i < 4; ++i) {
    const Gemm16Shape& s = kGemm16Shapes[i == 3 && f == kForward ? 4 : i];
    const double col_tiles = (cols + s.TN - 1) / s.TN;
    double row_tiles = used * ((N + s.TM - 1) / s.TM);
    if (!weight) {   // an expert's last tile is partly filled
      row_tiles = E == 1 ? (M + s.TM - 1) / s.TM : M / (double)s.TM + 0.77 * used;
      if (row_tiles < used) row_tiles = used;
    }
    const double alone = !weight && M < used * s.TM ? 1.5 * s.alone : s.alone;   // weights that are read only once
    const int all = weight ? 0 : ((f == kForward ? K : N) + 63) / 64;
    const double mean = M / used / 64;   // an expert's steps in dw; the largest's 1 + 1.1 times as many
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > parts || (splits > 1 && splits * out > kPartValues)) break;
      double steps, most;
      if (weight) {
        steps = mean / splits + 0.5;
        most = (1 + 1.1 * several) * mean / splits + 0.5;
      } else {
        const int each = (all + splits - 1) / splits;
        if ((all + each - 1) / each != splits) continue;   // no part is empty
        steps = most = each;
      }
      const double bytes = splits > 1 ? 4 : weight ? 3 : 2;   // (not by the call's types: the plan goes by sizes)
      steps = steps < s.least ? s.least : steps;
      most = most < s.least ? s.least : most;
      const double units = row_tiles * col_tiles * splits, rounds = units / kCus;
      const int c = rounds > s.held ? s.held : rounds <= 1.05 ? 1 : (int)(rounds + 0.95);   // workgroups a CU has
      const double step = s.full * c > alone ? s.full * c : alone;
      const double store = s.TM * s.TN * bytes * kCus / (s.stores * 1e6), work = (steps + s.begin) * step / c;
      const double unit = s.held == 1 ? work + store
                          : work > store ? work + 0.49 * store : store + 0.49 * work;   // others compute meanwhile
      const double longest = (most + s.begin) * step;
      for (int queue = 0; queue < (splits == 1 && rounds > 1 && !small ? 2 : 1); ++queue) {
        double us = longest + store * (rounds < 1 ? rounds : 1);
        if (rounds > 1) {
          us = rounds * unit;
          if (weight && !queue) us *= 1 + 0.53 * several * (mean < 2.6 ? 0.21 : mean < 12.5 ? mean / 12.5 : 1);
          if (!weight && !queue) us = (double)(long long)(rounds / c + 0.9) * c * unit;
          if (us < longest) us = longest;
        }
        if (weight) us += (1 - used / E) * out * bytes * splits / 5.3e6;   // zeros for experts without rows
        const double memory = (read + bytes * splits * out) / (rounds <= 1.05 ? 5.5e6 : 6.4e6);
        if (us < memory) us = memory;
        if (us < 8) us = 7.2 + 0.1 * us;   // the host's time for one launch, which another adds to
        us += (queue ? 6 : 0) + (splits > 1 ? 2.8 + (splits * 4 + 3) * out / 4.9e6 : 0);
        if (us < least) {
          least = us;
          best = {i, splits, queue != 0, ((size_t)out + 7) / 8 * 8, us};
        }
      }
    }
  }
  return best;
}

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
