// How a 16-bit product by expert is cut, by its sizes alone.  Plain C++, without the device's code.
#pragma once

#include <cmath>
#include <cstddef>
#include <initializer_list>

namespace zinc {

enum Product { kForward, kInput, kWeight };

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
// Examples (bf16, the kernel's us by trace, operands from HBM), in the order of the tiles, in one part, dealt out in
// turn: 32768 rows of 64 x 768 x 2048 c 126, 137, 158 and 178, da 137, 151, 168 and 202, dw in fp32 205, 229, 232 and
// 302, and 170 from queues in the largest; 2331 of 7 x 520 x 1032 (fp16, from the caches) 32, 20, 15 and 13; 64 of 64 x
// 768 x 2048 45, 32, 36 and 26, and 22 + 4 in two parts of the last.  For 256 CUs.
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

// Both gradients in one launch: one after the other where both are dealt out in the largest tile, or side by side in the
// smallest, by the model's times as if four fifths of the shorter were added to the longer (over 200 drawn sizes 6 %
// less on average).  A call, us, so and in two launches: 1111 rows of 7 x 520 x 1032, fp16 15 and 24; 500 of 64 x 256 x
// 512 20 and 23; 8 of 256 x 312 x 4152 142 and 153; 64 of 64 x 768 x 2048 119 and 108 (it takes two).  The model
// misses 47 of 16 x 1752 x 696: 41 in two, which it takes, and 27 side by side.
struct BackwardPlan {
  Gemm16Plan input, weight;
  bool together, beside;
};
inline BackwardPlan plan_backward(int M, int E, int N, int K) {
  BackwardPlan p{plan_gemm16(kInput, M, E, N, K), plan_gemm16(kWeight, M, E, N, K), false, false};
  p.together = p.input.queue && p.weight.queue && p.input.shape == 0 && p.weight.shape == 0;
  const double a = plan_gemm16(kInput, M, E, N, K, true).us, w = plan_gemm16(kWeight, M, E, N, K, true).us;
  p.beside = !p.together && (a > w ? a + 0.8 * w : w + 0.8 * a) < p.input.us + p.weight.us;
  return p;
}

}  // namespace zinc
