#include "gemm16_launch.hpp"

namespace zinc {

hipError_t launch_gemm16_weight(const void* p, const void* q, int type, const int32_t* offsets, int E, int M, int N,
                               int K, int out_type, void* c, void* ws, hipStream_t stream) {
  return launch_gemm16<kWeight>(p, q, type, offsets, E, M, N, K, out_type, c, ws, stream);
}

}  // namespace zinc
