#include "gemm16_launch.hpp"

namespace zinc {

hipError_t launch_gemm16_forward(const void* p, const void* q, int type, const int32_t* offsets, int E, int M, int N,
                               int K, int out_type, void* c, void* ws, hipStream_t stream) {
  return launch_gemm16<kForward>(p, q, type, offsets, E, M, N, K, out_type, c, ws, stream);
}

size_t gemm16_workspace_bytes(int M, int E, int N, int K) {
  return M == 0 ? 0 : kQueueBytes + gemm16_part_bytes(kForward, M, E, N, K);
}

}  // namespace zinc
