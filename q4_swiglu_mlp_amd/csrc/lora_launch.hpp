// How the adapters' products are cut, by their sizes alone, and their launches (lora_device.hpp).
#pragma once

#include "lora_device.hpp"
#include "launch.hpp"

namespace zinc {

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Row tiles of 16 a workgroup takes: one where adapters have few rows, else as many as the registers hold
// with two workgroups a CU.  8192 rows, eight adapters, 4096 to 11008, bf16, us by trace, with one, two and four: the
// forward call's second product of rank 16 76, 71 and 78, of rank 32 84, 74 and 79, of rank 64 123, 96 and 90, its first
// of rank 16 22, 20 and 17, of rank 64 41, 28 and 23; all of the gradients of rank 16 147, 142 and 168, of rank 64 244,
// 235 and 445 (registers spill).
inline int lora_row_tiles(int M, int E, int rank, bool forward) {
  if (M / E <= 24 || rank > 128) return 1;
  return forward && rank > 32 && rank <= 64 ? 4 : 2;
}

// Rows times splits of the first products' parts, at most, wherever there is more than one.
constexpr int kPartRows = 16384;

// Parts of the columns in a first product: as many as leave at most two workgroups a CU, of 512 columns or more.
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

// Spans of the columns in a second product: 1024 columns (8192 x 11008, bf16, 512, 768, 1024 and 2816 columns: rank 16
// 71, 69, 71 and 75 us, rank 32 74, 74, 74 and 77, rank 64 95, 96, 90 and 85), down to 256 where there are fewer than two
// workgroups a CU.
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
// or more if the rows are even.  They pay for their sum where the rows are uneven or the adapters few: a call on uneven
// rows, bf16, us, in 1, 2, 4 and 8 parts: 4096 rows of 4, rank 16, 4096 to 4096 72, 57, 55 (the rule's) and 59; 2000 of
// 2, rank 16, 2048 to 2048 57, 37, 27 and 26 (seven: 26); 4060 of 8, rank 64, 5784 to 1032 106, 101 (the rule's), 110 and
// 130, but 5784 to 5784 127, 144 (the rule's), 163 and 200.
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
