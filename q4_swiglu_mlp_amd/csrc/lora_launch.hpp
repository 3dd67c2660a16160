// How the adapters' products are cut, by their sizes alone, and their launches (lora_device.hpp).
#pragma once

#include "lora_device.hpp"
#include "launch.hpp"

namespace zinc {

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Row tiles of 16 a workgroup takes: one where adapters have few rows, else as many as the registers hold
// with two workgroups a CU.  8192 rows, eight adapters, 4096 to 11008, us: the second product through the
// caches of rank 16 74 with two, 80 with four, 75 with one; of rank 32 78 and 81; of rank 64 104 with two, 91 with
// four, but 101 and 115 where its matrix is turned (dx); the first of rank 16 15 - 17 with any, of rank 64 27 with
// two, 40 with one.
// Of the forward call's first product, 23 with four in one workgroup a CU.
inline int lora_row_tiles(int M, int E, int rank, bool forward) {
  if (M / E <= 24 || rank > 128) return 1;
  return forward && rank > 32 && rank <= 64 ? 4 : 2;
}

// Rows times splits of the first products' parts, at most, wherever there is more than one.
constexpr int kPartRows = 16384;

// Parts of the columns in a first product: enough for two workgroups a CU, of 512 columns or more.
inline int shrink_splits(int M, int E, int rank, int C, bool forward) {
  if (M == 0) return 1;
  const long long tiles = max_row_tiles(M, E, 16 * lora_row_tiles(M, E, rank, forward));
  long long s = 512 / (tiles < 512 ? tiles : 512);
  const int by_columns = ceil_div(C, 512), by_rows = kPartRows / (M < kPartRows ? M : kPartRows);
  s = s < by_columns ? s : by_columns;
  s = s < by_rows ? s : by_rows;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}
inline size_t lora_part_bytes(int M, int rank) { return (size_t)(M > kPartRows ? M : kPartRows) * rank * 4; }

inline ShrinkArgs shrink_of(bool forward, const LoraPlan& plan, const void* z, const void* w, int C, int rank,
                            float* parts) {
  const int splits = shrink_splits(plan.M, plan.E, rank, C, forward);
  return {plan, z, w, C, rank, splits, ceil_div(ceil_div(C, splits), 32) * 32, parts};
}
inline long long shrink_blocks(bool forward, const ShrinkArgs& s) {
  return max_row_tiles(s.plan.M, s.plan.E, 16 * lora_row_tiles(s.plan.M, s.plan.E, s.rank, forward)) * s.splits;
}

// Spans of the columns in a second product: 1024 columns (8192 x 11008, rank 64 84 us, 512 columns 88, 768 92,
// 2816 92), down to 256 where there are fewer than two workgroups a CU.
inline ExpandArgs expand_of(bool forward, const ShrinkArgs& f, const void* w, int N, const float* scales,
                            const void* base, void* y) {
  ExpandArgs s{f.plan, f.parts, f.splits, f.rank, N, w, scales, base, y, 0, 0, 0, 0};
  s.row_tiles = (int)max_row_tiles(f.plan.M, f.plan.E, 16 * lora_row_tiles(f.plan.M, f.plan.E, f.rank, forward));
  const int least = ceil_div(N, 1024), most = ceil_div(N, 256);
  int spans = 512 / (s.row_tiles ? s.row_tiles : 1);
  spans = spans < least ? least : spans > most ? most : spans;
  s.span = ceil_div(ceil_div(N, spans), 256) * 256;
  s.spans = ceil_div(N, s.span);
  s.copies = base == y ? 0 : ceil_div(f.plan.M, kCopied);
  return s;
}
inline long long expand_blocks(const ExpandArgs& s) {
  return ((long long)s.row_tiles + s.copies) * s.spans;
}

// Parts of an adapter's rows in the gradients of A and B: as many as make two workgroups a CU at least, of 128 rows
// or more if the rows are even (4060 rows of 8, 5784 columns: the second launch 55 us with two parts, 74 with one).
inline int grad_splits(int M, int E, int C) {
  const long long tiles = (long long)E * ceil_div(C, 128);
  long long s = ceil_div(512, tiles);
  const int by_rows = M / E / 128;
  s = s < by_rows ? s : by_rows;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}
inline size_t grad_bytes(int M, int E, int rank, int C) {
  const int s = grad_splits(M, E, C);
  return s > 1 ? (size_t)s * E * rank * C * 4 : 0;
}
inline long long grad_blocks(const LoraGradArgs& s) { return (long long)s.plan.E * s.splits * ceil_div(s.C, 128); }

// Workgroups a CU that a kernel's registers are held to.
constexpr int lora_held(int JT) { return JT <= 8 ? 2 : 1; }
constexpr int lora_forward_tiles(int JT, int R) { return R == 2 && JT == 4 ? 4 : R; }

template <int V>
struct Int {
  static constexpr int value = V;
};

// f(T, JT, R): the type, the tiles of 16 that hold the rank, and the backward call's row tiles.
template <typename T, int JT, typename F>
hipError_t by_rows(bool few, F f) {
  if constexpr (JT <= 8)
    if (!few) return f(T{}, Int<JT>{}, Int<2>{});
  return f(T{}, Int<JT>{}, Int<1>{});
}
template <typename T, typename F>
hipError_t by_rank(int rank, bool few, F f) {
  if (rank <= 16) return by_rows<T, 1>(few, f);
  if (rank <= 32) return by_rows<T, 2>(few, f);
  if (rank <= 64) return by_rows<T, 4>(few, f);
  if (rank <= 128) return by_rows<T, 8>(few, f);
  constexpr int kMost = 16;
  static_assert(kLoraMaxRank == 16 * kMost, "the largest rank fills the most tiles");
  return by_rows<T, kMost>(few, f);
}
template <typename F>
hipError_t by_kind(int type, int M, int E, int rank, F f) {
  const bool few = lora_row_tiles(M, E, rank, false) == 1;
  return type == 0 ? by_rank<_Float16>(rank, few, f) : by_rank<__bf16>(rank, few, f);
}

}  // namespace zinc
