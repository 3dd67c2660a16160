// C ABI of the FP8 expert layer (include/zinc_mlp.h): host-side argument checks,
// then the launchers.  Every check runs before the first HIP call.
#include "../../include/zinc_mlp.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "launch.hpp"

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 1024;
constexpr long long kMaxSlots = 1 << 24;
constexpr int kMaxCols = 65536;
constexpr int kMaxN = 1 << 20;
constexpr int kMaxHidden = 16384;
constexpr int kMaxInter = 65536;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool type_ok(int32_t t) { return t == ZINC_F16 || t == ZINC_BF16 || t == ZINC_F32; }
bool slots_ok(int32_t M, int32_t top_k) {
  return M >= 0 && top_k >= 1 && top_k <= kMaxTopK && (long long)M * top_k <= kMaxSlots;
}
bool cols_ok(int32_t c, int32_t unit) { return c > 0 && c % unit == 0 && c <= kMaxCols; }

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

// What the calls on routed rows share.
int check_rows(int32_t type, int32_t M, int32_t top_k, int32_t hidden, int32_t unit) {
  if (!cols_ok(hidden, unit)) return ZINC_ERR_SHAPE;
  return type_ok(type) && slots_ok(M, top_k) ? ZINC_OK : ZINC_ERR_ARG;
}

bool gemm_shape_ok(int32_t N, int32_t K) { return N >= 1 && N <= kMaxN && cols_ok(K, 16); }
bool gemm_sizes_ok(int32_t M, int32_t E) { return M >= 0 && M <= kMaxSlots && E >= 1 && E <= kMaxExperts; }

int gemm(const void* a, const float* sa, const void* w, const float* sw, const int32_t* offsets, int32_t E, int32_t M,
         int32_t N, int32_t K, int32_t out_type, void* c, void* ws, size_t ws_bytes, void* stream) {
  if (!gemm_shape_ok(N, K)) return ZINC_ERR_SHAPE;
  if (!gemm_sizes_ok(M, E) || !type_ok(out_type)) return ZINC_ERR_ARG;
  if (M == 0) return ZINC_OK;
  if (!a || !sa || !w || !sw || !c) return ZINC_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(c, 16) || !aligned(sa, 4) || !aligned(sw, 4) ||
      !aligned(offsets, 4))
    return ZINC_ERR_ALIGN;
  const int st = check_workspace(ws, ws_bytes, zinc::gemm_fp8_workspace_bytes(M, offsets ? E : 0, N, K));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(
      zinc::launch_gemm_fp8(a, sa, w, sw, offsets, E, M, N, K, out_type, c, ws, begin(stream)));
}

bool experts_ok(int32_t M, int32_t top_k, int32_t E) {
  return E >= 1 && E <= kMaxExperts && top_k <= E && slots_ok(M, top_k);
}
bool dims_ok(int32_t hidden, int32_t inter) {
  return hidden > 0 && hidden % 128 == 0 && hidden <= kMaxHidden && inter > 0 && inter % 128 == 0 &&
         inter <= kMaxInter;
}

}  // namespace

extern "C" {

size_t zinc_moe_sort_workspace_size(int32_t M, int32_t top_k, int32_t n_experts) {
  if (!slots_ok(M, top_k) || n_experts < 1 || n_experts > kMaxExperts) return 0;
  return zinc::moe_sort_workspace_bytes(M * top_k, n_experts);
}

int zinc_moe_sort(const int32_t* expert_ids, int32_t M, int32_t top_k, int32_t n_experts, int32_t* offsets,
                  int32_t* slot_row, int32_t* row_slot, void* workspace, size_t workspace_bytes, int32_t* dev_error,
                  void* stream) {
  if (!slots_ok(M, top_k) || n_experts < 1 || n_experts > kMaxExperts) return ZINC_ERR_ARG;
  if (!offsets || (M > 0 && (!expert_ids || !slot_row || !row_slot))) return ZINC_ERR_NULL;
  if (!aligned(expert_ids, 4) || !aligned(offsets, 4) || !aligned(slot_row, 4) || !aligned(row_slot, 4) ||
      !aligned(dev_error, 4))
    return ZINC_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes, zinc::moe_sort_workspace_bytes(M * top_k, n_experts));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(zinc::launch_moe_sort(expert_ids, M * top_k, n_experts, offsets, slot_row, row_slot,
                                                     workspace, dev_error, begin(stream)));
}

int zinc_moe_gather(const void* x, int32_t type, int32_t M, int32_t top_k, int32_t hidden, const int32_t* slot_row,
                    void* xs, void* stream) {
  const int st = check_rows(type, M, top_k, hidden, 8);
  if (st != ZINC_OK || M == 0) return st;
  if (!x || !slot_row || !xs) return ZINC_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(slot_row, 4)) return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(
      zinc::launch_moe_gather(x, hidden * (type == ZINC_F32 ? 4 : 2), M, top_k, slot_row, xs, begin(stream)));
}

int zinc_moe_gather_fp8(const void* x, int32_t type, int32_t M, int32_t top_k, int32_t hidden,
                        const int32_t* slot_row, void* q, float* scales, void* stream) {
  const int st = check_rows(type, M, top_k, hidden, 16);
  if (st != ZINC_OK || M == 0) return st;
  if (!x || !slot_row || !q || !scales) return ZINC_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(slot_row, 4)) return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(
      zinc::launch_moe_gather_fp8(x, type, M, top_k, hidden, slot_row, q, scales, begin(stream)));
}

int zinc_moe_combine(const void* ys, int32_t type, int32_t M, int32_t top_k, int32_t hidden, const int32_t* slot_row,
                     const float* expert_weights, void* y, void* stream) {
  const int st = check_rows(type, M, top_k, hidden, 8);
  if (st != ZINC_OK || M == 0) return st;
  if (!ys || !slot_row || !y) return ZINC_ERR_NULL;
  if (!aligned(ys, 16) || !aligned(y, 16) || !aligned(slot_row, 4) || !aligned(expert_weights, 4))
    return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(
      zinc::launch_moe_combine(ys, type, M, top_k, hidden, slot_row, expert_weights, y, begin(stream)));
}

int zinc_moe_combine_backward(const void* dy, const void* ys, int32_t type, int32_t M, int32_t top_k, int32_t hidden,
                              const int32_t* slot_row, const float* expert_weights, void* dys, float* dweights,
                              void* stream) {
  const int st = check_rows(type, M, top_k, hidden, 8);
  if (st != ZINC_OK || M == 0) return st;
  if (!dy || !ys || !slot_row || !expert_weights || !dys || !dweights) return ZINC_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(slot_row, 4) ||
      !aligned(expert_weights, 4) || !aligned(dweights, 4))
    return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(zinc::launch_moe_combine_backward(dy, ys, type, M, top_k, hidden, slot_row,
                                                                 expert_weights, dys, dweights, begin(stream)));
}

int zinc_fp8_quantize(const void* x, int32_t type, int32_t rows, int32_t cols, int32_t block_rows, void* q,
                      float* scales, void* stream) {
  if (!cols_ok(cols, 16)) return ZINC_ERR_SHAPE;
  if (!type_ok(type) || rows < 0 || (block_rows != 1 && block_rows != 128)) return ZINC_ERR_ARG;
  if (rows == 0) return ZINC_OK;
  if (!x || !q || !scales) return ZINC_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4)) return ZINC_ERR_ALIGN;
  return zinc::status_from_hip(zinc::launch_fp8_quantize(x, type, rows, cols, block_rows, q, scales, begin(stream)));
}

size_t zinc_gemm_fp8_workspace_size(int32_t M, int32_t N, int32_t K) {
  return gemm_shape_ok(N, K) && gemm_sizes_ok(M, 1) ? zinc::gemm_fp8_workspace_bytes(M, 0, N, K) : 0;
}

int zinc_gemm_fp8(const void* a, const float* a_scales, const void* w, const float* w_scales, int32_t M, int32_t N,
                  int32_t K, int32_t out_type, void* c, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm(a, a_scales, w, w_scales, nullptr, 1, M, N, K, out_type, c, workspace, workspace_bytes, stream);
}

size_t zinc_moe_gemm_fp8_workspace_size(int32_t rows, int32_t n_experts, int32_t N, int32_t K) {
  return gemm_shape_ok(N, K) && gemm_sizes_ok(rows, n_experts)
             ? zinc::gemm_fp8_workspace_bytes(rows, n_experts, N, K)
             : 0;
}

int zinc_moe_gemm_fp8(const void* a, const float* a_scales, const void* w, const float* w_scales,
                      const int32_t* offsets, int32_t n_experts, int32_t rows, int32_t N, int32_t K,
                      int32_t out_type, void* c, void* workspace, size_t workspace_bytes, void* stream) {
  if (!offsets && rows > 0) return ZINC_ERR_NULL;
  return gemm(a, a_scales, w, w_scales, offsets, n_experts, rows, N, K, out_type, c, workspace, workspace_bytes,
              stream);
}

size_t zinc_moe_fp8_experts_workspace_size(int32_t M, int32_t top_k, int32_t n_experts, int32_t hidden, int32_t inter,
                                           int32_t type) {
  if (!dims_ok(hidden, inter) || !type_ok(type) || !experts_ok(M, top_k, n_experts)) return 0;
  return zinc::moe_fp8_workspace_bytes(M, top_k, n_experts, hidden, inter);
}

int zinc_moe_fp8_experts(const void* w_gate, const float* gate_scales, const void* w_up, const float* up_scales,
                         const void* w_down, const float* down_scales, int32_t n_experts, int32_t hidden,
                         int32_t inter, const void* x, int32_t type, int32_t M, const int32_t* expert_ids,
                         const float* expert_weights, int32_t top_k, void* y, void* workspace, size_t workspace_bytes,
                         int32_t* dev_error, void* stream) {
  if (!dims_ok(hidden, inter)) return ZINC_ERR_SHAPE;
  if (!type_ok(type) || !experts_ok(M, top_k, n_experts)) return ZINC_ERR_ARG;
  if (M == 0) return ZINC_OK;
  if (!w_gate || !gate_scales || !w_up || !up_scales || !w_down || !down_scales || !x || !expert_ids ||
      !expert_weights || !y)
    return ZINC_ERR_NULL;
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || !aligned(x, 16) || !aligned(y, 16) ||
      !aligned(gate_scales, 4) || !aligned(up_scales, 4) || !aligned(down_scales, 4) || !aligned(expert_ids, 4) ||
      !aligned(expert_weights, 4) || !aligned(dev_error, 4))
    return ZINC_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes,
                                 zinc::moe_fp8_workspace_bytes(M, top_k, n_experts, hidden, inter));
  if (st != ZINC_OK) return st;
  return zinc::status_from_hip(zinc::launch_moe_fp8(w_gate, gate_scales, w_up, up_scales, w_down, down_scales,
                                                    n_experts, hidden, inter, x, type, M, expert_ids, expert_weights,
                                                    top_k, y, workspace, dev_error, begin(stream)));
}

}  // extern "C"
