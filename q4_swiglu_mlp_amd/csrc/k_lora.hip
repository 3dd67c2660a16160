// The low-rank adapters' calls: which launches, their splits and their workspace.
#include "lora_launch.hpp"

namespace zinc {

hipError_t launch_lora_join(const float* parts, int splits, size_t each, size_t n, const float* scales, int type,
                            void* out, hipStream_t stream);

namespace {

// Rows times splits of the first products' parts, at most, wherever there is more than one.
constexpr int kPartRows = 16384;

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Parts of the columns in a first product: enough for two workgroups a CU, of 512 columns or more.
int shrink_splits(int M, int E, int rank, int C) {
  if (M == 0) return 1;
  const long long tiles = max_row_tiles(M, E, 16 * lora_row_tiles(M, E, rank));
  long long s = 512 / (tiles < 512 ? tiles : 512);
  const int by_columns = ceil_div(C, 512), by_rows = kPartRows / (M < kPartRows ? M : kPartRows);
  s = s < by_columns ? s : by_columns;
  s = s < by_rows ? s : by_rows;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

// Parts of an adapter's rows in the gradients of A and B: as many as make two workgroups a CU, of 256 rows
// or more if the rows are even.
int grad_splits(int M, int E, int C) {
  const long long tiles = (long long)E * ceil_div(C, 64);
  long long s = 512 / (tiles < 512 ? tiles : 512);
  const int by_rows = M / E / 256;
  s = s < by_rows ? s : by_rows;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

size_t part_bytes(int M, int rank) { return (size_t)(M > kPartRows ? M : kPartRows) * rank * 4; }
size_t grad_bytes(int M, int E, int rank, int C) {
  const int s = grad_splits(M, E, C);
  return s > 1 ? (size_t)s * E * rank * C * 4 : 0;
}

ShrinkArgs shrink_of(const LoraPlan& plan, const void* z, const void* w, int C, int rank, float* parts) {
  const int splits = shrink_splits(plan.M, plan.E, rank, C);
  return {plan, z, w, C, rank, splits, ceil_div(ceil_div(C, splits), 32) * 32, parts};
}

hipError_t gradient(const LoraPlan& plan, const void* z, const float* f, int f_splits, int rank, int C,
                    const float* scales, int type, bool j_first, float* parts, void* out, hipStream_t stream) {
  const int splits = grad_splits(plan.M, plan.E, C);
  const LoraGradArgs g{plan, z, f, f_splits, rank, C, scales, splits, splits > 1 ? static_cast<void*>(parts) : out};
  const hipError_t e = launch_lora_grad(g, type, j_first, stream);
  if (e != hipSuccess || splits == 1) return e;
  const size_t each = (size_t)rank * C;
  return launch_lora_join(parts, splits, each, each * plan.E, scales, type, out, stream);
}

}  // namespace

size_t lora_workspace_bytes(int M, int rank) { return part_bytes(M, rank); }

hipError_t launch_lora(const void* x, const void* a, const void* b, const float* scales, const int32_t* offsets,
                       const int32_t* slot_row, const int32_t* row_slot, int E, int M, int K, int N, int rank, int type,
                       const void* base, void* y, void* ws, hipStream_t stream) {
  const LoraPlan plan{offsets, slot_row, row_slot, E, M};
  const ShrinkArgs s = shrink_of(plan, x, a, K, rank, static_cast<float*>(ws));
  const hipError_t e = launch_lora_shrink(s, type, false, stream);
  if (e != hipSuccess) return e;
  return launch_lora_expand({plan, s.parts, s.splits, rank, N, b, scales, base, y, 0}, type, false, stream);
}

size_t lora_backward_workspace_bytes(int M, int E, int K, int N, int rank) {
  return 2 * part_bytes(M, rank) + grad_bytes(M, E, rank, K) + grad_bytes(M, E, rank, N);
}

hipError_t launch_lora_backward(const void* dy, const void* x, const void* a, const void* b, const float* scales,
                                const int32_t* offsets, const int32_t* slot_row, const int32_t* row_slot, int E, int M,
                                int K, int N, int rank, int type, const void* base, void* dx, void* da, void* db,
                                void* ws, hipStream_t stream) {
  const LoraPlan plan{offsets, slot_row, row_slot, E, M};
  char* at = static_cast<char*>(ws);
  float* h = reinterpret_cast<float*>(at);
  float* dh = reinterpret_cast<float*>(at + part_bytes(M, rank));
  float* parts_a = reinterpret_cast<float*>(at + 2 * part_bytes(M, rank));
  float* parts_b = reinterpret_cast<float*>(at + 2 * part_bytes(M, rank) + grad_bytes(M, E, rank, K));
  hipError_t e = hipSuccess;
  const ShrinkArgs sh = shrink_of(plan, x, a, K, rank, h), sd = shrink_of(plan, dy, b, N, rank, dh);
  if (M && db) e = launch_lora_shrink(sh, type, false, stream);
  if (e == hipSuccess && M && (dx || da)) e = launch_lora_shrink(sd, type, true, stream);
  if (e == hipSuccess && dx)
    e = launch_lora_expand({plan, dh, sd.splits, rank, K, a, scales, base, dx, 0}, type, true, stream);
  if (e == hipSuccess && da)
    e = gradient(plan, x, dh, sd.splits, rank, K, scales, type, true, parts_a, da, stream);
  if (e == hipSuccess && db)
    e = gradient(plan, dy, h, sh.splits, rank, N, scales, type, false, parts_b, db, stream);
  return e;
}

}  // namespace zinc
