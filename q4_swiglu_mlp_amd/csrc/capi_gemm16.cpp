// C ABI of the 16-bit products by group, SwiGLU and the low-rank adapters (include/zinc_mlp.h): host-side
// argument checks, then the launchers.  Every check runs before the first HIP call.
#include "../../include/zinc_mlp.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "launch.hpp"

namespace {

constexpr int kMaxGroups = 1024;
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxCols = 65536;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool cols_ok(int32_t c) { return c > 0 && c % 8 == 0 && c <= kMaxCols; }
bool rows_ok(int32_t M) { return M >= 0 && M <= kMaxRows; }
bool groups_ok(int32_t E) { return E >= 1 && E <= kMaxGroups; }
bool half_type(int32_t t) { return t == ZINC_F16 || t == ZINC_BF16; }
bool out_ok(int32_t type, int32_t out) { return out == type || out == ZINC_F32; }

// A workspace of `need` bytes; none is asked for where need is 0.
int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ZINC_OK;
  if (!ws) return ZINC_ERR_NULL;
  if (!aligned(ws, 16)) return ZINC_ERR_ALIGN;
  return bytes < need ? ZINC_ERR_WORKSPACE : ZINC_OK;
}

hipStream_t begin(void* stream) {
  (void)hipGetLastError();
  return static_cast<hipStream_t>(stream);
}

bool gemm_ok(int32_t rows, int32_t E, int32_t N, int32_t K) {
  return rows_ok(rows) && groups_ok(E) && cols_ok(N) && cols_ok(K);
}
bool lora_shape_ok(int32_t K, int32_t N, int32_t rank) {
  return cols_ok(K) && cols_ok(N) && rank > 0 && rank % 8 == 0 && rank <= zinc::kLoraMaxRank;
}

}  // namespace

extern "C" {

size_t zinc_moe_gemm_workspace_size(int32_t rows, int32_t n_experts, int32_t N, int32_t K) {
  if (!gemm_ok(rows, n_experts, N, K)) return 0;
  return zinc::gemm16_workspace_bytes(rows, n_experts, N, K);
}

int zinc_moe_gemm(const void* a, const void* w, int32_t type, const int32_t* offsets, int32_t n_experts, int32_t rows,
                  int32_t N, int32_t K, int32_t out_type, void* c, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (!cols_ok(N) || !cols_ok(K)) return ZINC_ERR_SHAPE;
  if (!gemm_ok(rows, n_experts, N, K) || !half_type(type) || !out_ok(type, out_type)) return ZINC_ERR_ARG;
  if (rows == 0) return ZINC_OK;
  if (!a || !w || !offsets || !c) return ZINC_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(c, 16) || !aligned(offsets, 4)) return ZINC_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes, zinc::gemm16_workspace_bytes(rows, n_experts, N, K));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(
      zinc::launch_gemm16_forward(a, w, type, offsets, n_experts, rows, N, K, out_type, c, workspace, begin(stream)));
}

size_t zinc_moe_gemm_backward_workspace_size(int32_t rows, int32_t n_experts, int32_t N, int32_t K) {
  if (!gemm_ok(rows, n_experts, N, K)) return 0;
  return zinc::gemm16_backward_workspace_bytes(rows, n_experts, N, K);
}

int zinc_moe_gemm_backward(const void* dc, const void* a, const void* w, int32_t type, const int32_t* offsets,
                           int32_t n_experts, int32_t rows, int32_t N, int32_t K, int32_t da_type, void* da,
                           int32_t dw_type, void* dw, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cols_ok(N) || !cols_ok(K)) return ZINC_ERR_SHAPE;
  if (!gemm_ok(rows, n_experts, N, K) || !half_type(type) || (da && !out_ok(type, da_type)) ||
      (dw && !out_ok(type, dw_type)))
    return ZINC_ERR_ARG;
  if (!da && !dw) return ZINC_ERR_NULL;
  if (rows == 0 && !dw) return ZINC_OK;
  if (!offsets || (rows > 0 && (!dc || (da && !w) || (dw && !a)))) return ZINC_ERR_NULL;
  if (!aligned(dc, 16) || !aligned(a, 16) || !aligned(w, 16) || !aligned(da, 16) || !aligned(dw, 16) ||
      !aligned(offsets, 4))
    return ZINC_ERR_ALIGN;
  const int st =
      check_workspace(workspace, workspace_bytes, zinc::gemm16_backward_workspace_bytes(rows, n_experts, N, K));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(zinc::launch_gemm16_backward(dc, a, w, type, offsets, n_experts, rows, N, K, da_type, da,
                                                            dw_type, dw, workspace, begin(stream)));
}

int zinc_swiglu(const void* gate, const void* up, int32_t type, int32_t rows, int32_t cols, void* h, void* stream) {
  if (!cols_ok(cols)) return ZINC_ERR_SHAPE;
  if (!rows_ok(rows) || (!half_type(type) && type != ZINC_F32)) return ZINC_ERR_ARG;
  if (rows == 0) return ZINC_OK;
  if (!gate || !up || !h) return ZINC_ERR_NULL;
  if (!aligned(gate, 16) || !aligned(up, 16) || !aligned(h, 16)) return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(zinc::launch_swiglu(gate, up, type, (size_t)rows * cols, h, begin(stream)));
}

int zinc_swiglu_backward(const void* dh, const void* gate, const void* up, int32_t type, int32_t rows, int32_t cols,
                         void* dgate, void* dup, void* stream) {
  if (!cols_ok(cols)) return ZINC_ERR_SHAPE;
  if (!rows_ok(rows) || (!half_type(type) && type != ZINC_F32)) return ZINC_ERR_ARG;
  if (rows == 0) return ZINC_OK;
  if (!dh || !gate || !up || !dgate || !dup) return ZINC_ERR_NULL;
  if (!aligned(dh, 16) || !aligned(gate, 16) || !aligned(up, 16) || !aligned(dgate, 16) || !aligned(dup, 16))
    return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(
      zinc::launch_swiglu_backward(dh, gate, up, type, (size_t)rows * cols, dgate, dup, begin(stream)));
}

size_t zinc_lora_workspace_size(int32_t M, int32_t n_adapters, int32_t K, int32_t N, int32_t rank) {
  if (!lora_shape_ok(K, N, rank) || !rows_ok(M) || !groups_ok(n_adapters) || M == 0) return 0;
  return zinc::lora_workspace_bytes(M, rank);
}

int zinc_lora(const void* x, int32_t type, int32_t M, int32_t K, const void* a, const void* b, int32_t rank,
              int32_t n_adapters, int32_t N, const float* scales, const int32_t* offsets, const int32_t* slot_row,
              const int32_t* row_slot, const void* base, void* y, void* workspace, size_t workspace_bytes,
              void* stream) {
  if (!lora_shape_ok(K, N, rank)) return ZINC_ERR_SHAPE;
  if (!rows_ok(M) || !groups_ok(n_adapters) || !half_type(type)) return ZINC_ERR_ARG;
  if (M == 0) return ZINC_OK;
  if (!x || !a || !b || !offsets || !slot_row || !row_slot || !y) return ZINC_ERR_NULL;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || !aligned(y, 16) ||
      !aligned(scales, 4) || !aligned(offsets, 4) || !aligned(slot_row, 4) || !aligned(row_slot, 4))
    return ZINC_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes, zinc::lora_workspace_bytes(M, rank));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(zinc::launch_lora(x, a, b, scales, offsets, slot_row, row_slot, n_adapters, M, K, N,
                                                 rank, type, base, y, workspace, begin(stream)));
}

size_t zinc_lora_backward_workspace_size(int32_t M, int32_t n_adapters, int32_t K, int32_t N, int32_t rank) {
  if (!lora_shape_ok(K, N, rank) || !rows_ok(M) || !groups_ok(n_adapters) || M == 0) return 0;
  return zinc::lora_backward_workspace_bytes(M, n_adapters, K, N, rank);
}

int zinc_lora_backward(const void* dy, const void* x, int32_t type, int32_t M, int32_t K, const void* a, const void* b,
                       int32_t rank, int32_t n_adapters, int32_t N, const float* scales, const int32_t* offsets,
                       const int32_t* slot_row, const int32_t* row_slot, const void* base, void* dx, void* da, void* db,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!lora_shape_ok(K, N, rank)) return ZINC_ERR_SHAPE;
  if (!rows_ok(M) || !groups_ok(n_adapters) || !half_type(type)) return ZINC_ERR_ARG;
  if (!dx && !da && !db) return ZINC_ERR_NULL;
  if (M == 0 && !da && !db) return ZINC_OK;
  if (!offsets || (M > 0 && (!dy || !x || !a || !b || !slot_row || !row_slot))) return ZINC_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) ||
      !aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16) || !aligned(scales, 4) || !aligned(offsets, 4) ||
      !aligned(slot_row, 4) || !aligned(row_slot, 4))
    return ZINC_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes,
                                 M ? zinc::lora_backward_workspace_bytes(M, n_adapters, K, N, rank) : 0);
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(zinc::launch_lora_backward(dy, x, a, b, scales, offsets, slot_row, row_slot, n_adapters,
                                                          M, K, N, rank, type, base, M ? dx : nullptr, da, db,
                                                          workspace, begin(stream)));
}

}  // extern "C"
