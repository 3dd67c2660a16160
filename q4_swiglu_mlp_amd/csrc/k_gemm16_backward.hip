// Both gradients of a 16-bit product by expert.  Where both are many units of the largest tile, one launch
// computes them: a workgroup that finds no more units of da goes on with those of dw, the experts with most
// rows first, so the last round of the one is work for the same CUs (32768 rows of 64 experts, 768 x 2048, dw in
// fp32, operands from HBM: 310 us, in two launches 323; where every second workgroup begins with dw 330).
#include "gemm16_launch.hpp"

namespace zinc {
namespace {

template <typename INPUT, typename WEIGHT>
__global__ __launch_bounds__(INPUT::THREADS) void k_gemm16_both(Gemm16Args a, Gemm16Args w) {
  extern __shared__ __align__(16) uint8_t smem[];
  INPUT::run(a, smem);
  __syncthreads();
  WEIGHT::run(w, smem);
}

// What the launch asks of a kernel, for the two together.
template <typename INPUT, typename WEIGHT>
struct Both {
  static constexpr Product kProduct = kInput;
  static constexpr int HELD = 1;
  static size_t smem_bytes(int E) { return INPUT::smem_bytes(E); }
};

struct BackwardPlan {
  Gemm16Plan input, weight;
  bool together;
};
BackwardPlan plan_backward(int M, int E, int N, int K) {
  BackwardPlan p{plan_gemm16(kInput, M, E, N, K), plan_gemm16(kWeight, M, E, N, K), false};
  p.together = p.input.queue && p.weight.queue && p.input.shape == 0 && p.weight.shape == 0;
  return p;
}

template <typename T, typename OA, typename OW>
hipError_t run_both(const Gemm16Args& a, const Gemm16Args& w, hipStream_t stream) {
  using INPUT = Gemm16<kInput, 256, 256, 2, 4, 2, T, OA>;
  using WEIGHT = Gemm16<kWeight, 256, 256, 2, 4, 2, T, OW>;
  const void* kernel = reinterpret_cast<const void*>(&k_gemm16_both<INPUT, WEIGHT>);
  unsigned grid = 0;
  int bytes = 0;
  hipError_t e = gemm16_grid<Both<INPUT, WEIGHT>>(a, kernel, 0, &grid, &bytes);
  if (e != hipSuccess) return e;
  for (int32_t* q : {a.queue, w.queue}) {
    hipLaunchKernelGGL(k_gemm16_queue, dim3(1), dim3(8), 0, stream, q, (int)grid / 8);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  timing_begin(stream);
  hipLaunchKernelGGL((k_gemm16_both<INPUT, WEIGHT>), dim3(grid), dim3(INPUT::THREADS), bytes, stream, a, w);
  timing_end(stream);
  return hipGetLastError();
}

}  // namespace

size_t gemm16_backward_workspace_bytes(int M, int E, int N, int K) {
  const BackwardPlan p = plan_backward(M, E, N, K);
  const size_t a = M ? gemm16_part_bytes(p.input) : 0, w = gemm16_part_bytes(p.weight);
  return (M && (p.input.queue || a)) || p.weight.queue || w ? 2 * kQueueBytes + (a > w ? a : w) : 0;
}

hipError_t launch_gemm16_backward(const void* dc, const void* a, const void* w, int type, const int32_t* offsets, int E,
                                  int M, int N, int K, int da_type, void* da, int dw_type, void* dw, void* ws,
                                  hipStream_t stream) {
  const BackwardPlan p = plan_backward(M, E, N, K);
  int32_t* queue = static_cast<int32_t*>(ws);
  if (da && dw && p.together) {
    const Gemm16Args ga{dc, w, offsets, E, M, N, K, da, 1, 0, queue};
    const Gemm16Args gw{dc, a, offsets, E, M, N, K, dw, 1, 0, queue + kQueueBytes / 4};
    return by_types(type, da_type, [&](auto t, auto oa) {
      using T = decltype(t);
      using OA = decltype(oa);
      return dw_type == 2 ? run_both<T, OA, float>(ga, gw, stream) : run_both<T, OA, T>(ga, gw, stream);
    });
  }
  hipError_t e = hipSuccess;
  if (da && M) e = launch_gemm16_input(dc, w, type, offsets, E, M, N, K, da_type, da, ws, stream);
  if (e == hipSuccess && dw) e = launch_gemm16_weight(dc, a, type, offsets, E, M, N, K, dw_type, dw, ws, stream);
  return e;
}

}  // namespace zinc
