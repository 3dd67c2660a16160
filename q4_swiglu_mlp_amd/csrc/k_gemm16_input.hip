#include "gemm16_launch.hpp"

namespace zinc {

hipError_t launch_gemm16_input(const void* p, const void* q, int type, const int32_t* offsets, int E, int M, int N,
                               int K, int out_type, void* c, hipStream_t stream) {
  const Gemm16Args g{p, q, offsets, E, M, N, K, c};
  const int mean = M / E;
  return by_types(type, out_type, [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    if (mean <= 160) return run_gemm16<kInput, 64, 128, 1, 4, T, O>(g, stream);
    if (mean <= 320) return run_gemm16<kInput, 128, 128, 2, 2, T, O>(g, stream);
    return run_gemm16<kInput, 256, 256, 2, 4, T, O>(g, stream);
  });
}

}  // namespace zinc
