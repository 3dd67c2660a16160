// Host-side launchers of the library's kernels.  Every launcher assumes its
// arguments were validated by the C ABI layer (capi.cpp): shapes are
// multiples of 256, pointers are 16-byte aligned, sizes fit the workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace zinc {

// ZINC_OK for hipSuccess; otherwise ZINC_ERR_HIP, and `e` becomes the text
// that zinc_hip_error_string() returns on this thread (capi.cpp).
int status_from_hip(hipError_t e);

// Kernel timing hook (timing.cpp): no-ops unless zinc_timing_enable() was called.
void timing_begin(hipStream_t stream);
void timing_end(hipStream_t stream);

hipError_t launch_q4k_dequant_f32(const void* blocks, int rows, int cols, float* out, hipStream_t stream);
// fmt 1: Q5_K (cols % 256 == 0), 2: Q5_1 (cols % 32 == 0).
hipError_t launch_q5_dequant_f32(int fmt, const void* blocks, int rows, int cols, float* out, hipStream_t stream);

// Fused prefill.
size_t prefill_workspace_bytes(int M, int hidden, int inter);
// mlp_scale multiplies the MLP output; res (nullable, [M x hidden] fp16, may be
// y) is added at the output scale: y = fp16((res + mlp_scale * MLP(x)) * 2^-out_shift).
hipError_t launch_prefill(const void* wg, const void* wu, const void* wd, int hidden, int inter,
                          const void* x, void* y, int M, int inter_shift, int out_shift, void* ws,
                          hipStream_t stream, float mlp_scale = 1.0f, const void* res = nullptr);

// The staged comparison baseline of the prefill: the same units with the
// gate/up outputs and the intermediate in device memory (four main launches).
size_t prefill_staged_workspace_bytes(int M, int hidden, int inter);
hipError_t launch_prefill_staged(const void* wg, const void* wu, const void* wd, int hidden, int inter,
                                 const void* x, void* y, int M, int inter_shift, int out_shift, void* ws,
                                 hipStream_t stream);

// Decode, 1 <= M <= 8: row-streaming dot products for M = 1 (k_decode.hip),
// 16x16x32 MFMA tiles for M >= 2 (k_decode_mfma.hip); both write the fp16
// intermediate [M x inter] into the workspace between their two kernels.
size_t decode_workspace_bytes(int M, int hidden, int inter);
// gamma (nullable): the pre-MLP RMS norm of x with weight gamma and eps is the
// MLP's input; xn ([M x hidden] fp16 scratch) receives it where a kernel of its
// own computes it.
hipError_t launch_decode(const void* wg, const void* wu, const void* wd, int hidden, int inter,
                         const void* x, void* y, int M, int inter_shift, int out_shift, void* ws,
                         hipStream_t stream, float mlp_scale = 1.0f, const void* res = nullptr,
                         const void* gamma = nullptr, float eps = 0.0f, void* xn = nullptr);
hipError_t launch_decode_mfma(const void* wg, const void* wu, const void* wd, int hidden, int inter,
                              const void* x, void* y, int M, int inter_shift, int out_shift, void* ws,
                              hipStream_t stream, float mlp_scale = 1.0f, const void* res = nullptr);

// Batched-expert MoE.
size_t moe_workspace_bytes(int M, int top_k, int n_experts, int hidden, int inter);
// down_fmt: 0 Q4_K, 1 Q5_K, 2 Q5_1 (W_down's block format; gate and up are Q4_K).
hipError_t launch_moe(const void* wg, const void* wu, const void* wd, int n_experts, int hidden, int inter,
                      const void* x, int M, const int32_t* ids, const float* p, int top_k, void* y,
                      int inter_shift, int out_shift, void* ws, int32_t* dev_error, hipStream_t stream,
                      int down_fmt = 0);

// MoE router: per token the top_k largest logits' experts and their softmax
// weights (k_router.hip).  1 <= top_k <= min(64, n_experts), n_experts <= 1024.
hipError_t launch_route_topk(const float* logits, int M, int n_experts, int top_k, int32_t* ids, float* p,
                             hipStream_t stream);

// Expert-layer token permutation (k_moe_tokens.hip).  S = M * top_k slots; type
// codes: 0 fp16, 1 bf16, 2 fp32.
size_t moe_sort_workspace_bytes(int S, int E);
hipError_t launch_moe_sort(const int32_t* ids, int S, int E, int32_t* offsets, int32_t* slot_row, int32_t* row_slot,
                           void* ws, int32_t* dev_error, hipStream_t stream);
hipError_t launch_moe_gather(const void* x, int row_bytes, int M, int top_k, const int32_t* slot_row, void* xs,
                             hipStream_t stream);
hipError_t launch_moe_combine(const void* ys, int type, int M, int top_k, int H, const int32_t* slot_row,
                              const float* p, void* y, hipStream_t stream);
// The same of fp32 rows; `type` is y's, p is given.
hipError_t launch_moe_combine_rows(const float* ys, int type, int M, int top_k, int H, const int32_t* slot_row,
                                   const float* p, void* y, hipStream_t stream);
hipError_t launch_moe_combine_backward(const void* dy, const void* ys, int type, int M, int top_k, int H,
                                       const int32_t* slot_row, const float* p, void* dys, float* dp,
                                       hipStream_t stream);

// e4m3 with a scale per block of 128 (k_fp8_quant.hip).
hipError_t launch_fp8_quantize(const void* x, int type, int R, int C, int block_rows, void* q, float* scales,
                               hipStream_t stream);
hipError_t launch_moe_gather_fp8(const void* x, int type, int M, int top_k, int C, const int32_t* slot_row, void* q,
                                 float* scales, hipStream_t stream);

// Products of block-scaled e4m3 matrices and the FP8 expert layer (k_fp8_gemm.hip).
// offsets: nullptr for one dense product (E = 1), else the experts' row ranges.
size_t gemm_fp8_workspace_bytes(int M, int E, int N, int K);
hipError_t launch_gemm_fp8(const void* a, const float* sa, const void* w, const float* sw, const int32_t* offsets,
                           int E, int M, int N, int K, int out_type, void* c, void* ws, hipStream_t stream);
size_t moe_fp8_workspace_bytes(int M, int top_k, int E, int H, int I);
hipError_t launch_moe_fp8(const void* wg, const float* sg, const void* wu, const float* su, const void* wd,
                          const float* sd, int E, int H, int I, const void* x, int type, int M, const int32_t* ids,
                          const float* p, int top_k, void* y, void* ws, int32_t* dev_error, hipStream_t stream);

// 16-bit products by group (k_gemm16_*.hip): rows offsets[e] .. offsets[e + 1] - 1 of M take group e's matrix
// [N x K].  type: the operands' (0 or 1); out_type: the same or 2.
//   forward  c [M x N] = a [M x K] w^T;  input  c = da [M x K] = dc [M x N] w;  weight  c = dw [E x N x K] = dc^T a
hipError_t launch_gemm16_forward(const void* a, const void* w, int type, const int32_t* offsets, int E, int M, int N,
                                 int K, int out_type, void* c, void* ws, hipStream_t stream);
hipError_t launch_gemm16_input(const void* dc, const void* w, int type, const int32_t* offsets, int E, int M, int N,
                               int K, int out_type, void* c, void* ws, hipStream_t stream);
hipError_t launch_gemm16_weight(const void* dc, const void* a, int type, const int32_t* offsets, int E, int M, int N,
                                int K, int out_type, void* c, void* ws, hipStream_t stream);

size_t gemm16_workspace_bytes(int M, int E, int N, int K);
// Both gradients, or one where the other's output is null.
size_t gemm16_backward_workspace_bytes(int M, int E, int N, int K);
hipError_t launch_gemm16_backward(const void* dc, const void* a, const void* w, int type, const int32_t* offsets, int E,
                                  int M, int N, int K, int da_type, void* da, int dw_type, void* dw, void* ws,
                                  hipStream_t stream);

// SwiGLU and its gradients over n values, a multiple of eight (k_swiglu.hip).
hipError_t launch_swiglu(const void* gate, const void* up, int type, size_t n, void* h, hipStream_t stream);
hipError_t launch_swiglu_backward(const void* dh, const void* gate, const void* up, int type, size_t n, void* dgate,
                                  void* dup, hipStream_t stream);

// Low-rank adapters beside a projection (k_lora_*.hip).  base may be null or y (dx); dx, da, db may be null.
constexpr int kLoraMaxRank = 256;   // what the kernels' most tiles of 16 hold
size_t lora_workspace_bytes(int M, int rank);
hipError_t launch_lora(const void* x, const void* a, const void* b, const float* scales, const int32_t* offsets,
                       const int32_t* slot_row, const int32_t* row_slot, int E, int M, int K, int N, int rank, int type,
                       const void* base, void* y, void* ws, hipStream_t stream);
size_t lora_backward_workspace_bytes(int M, int E, int K, int N, int rank);
hipError_t launch_lora_backward(const void* dy, const void* x, const void* a, const void* b, const float* scales,
                                const int32_t* offsets, const int32_t* slot_row, const int32_t* row_slot, int E, int M,
                                int K, int N, int rank, int type, const void* base, void* dx, void* da, void* db,
                                void* ws, hipStream_t stream);

}  // namespace zinc
