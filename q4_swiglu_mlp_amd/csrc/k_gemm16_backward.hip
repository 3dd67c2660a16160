// Both gradients of a 16-bit product by expert, in one launch where that is less.  Where both are many units of the
// largest tile, a workgroup that finds no more units of da goes on with those of dw, the experts with most
// rows first, so the last round of the one is work for the same CUs (32768 rows of 64 experts, 768 x 2048, dw in
// fp32, operands from HBM: a call 300 us, in two launches 311, of which the kernels are 140 - 143 and 174 - 180; where
// every second workgroup began with dw 6 % more).
// Where both are a few units, or bound by memory, the smallest tile's workgroups for da and for dw lie side by side
// (plan_backward).
#include "gemm16_launch.hpp"

namespace zinc {
namespace {

template <typename INPUT, typename WEIGHT>
__global__ __launch_bounds__(INPUT::THREADS) void k_gemm16_both(Gemm16Args a, Gemm16Args w) {
  extern __shared__ __align__(16) uint8_t smem[];
  INPUT::run(a, smem, blockIdx.x, gridDim.x);
  __syncthreads();
  WEIGHT::run(w, smem, blockIdx.x, gridDim.x);
}

// What the launch asks of a kernel, for the two together.
template <typename INPUT, typename WEIGHT>
struct Both {
  static constexpr Product kProduct = kInput;
  static constexpr int HELD = 1;
  static size_t smem_bytes(int E) { return INPUT::smem_bytes(E); }
};

// The workgroups before `first` compute da, the others dw.
template <typename INPUT, typename WEIGHT>
__global__ __launch_bounds__(INPUT::THREADS) void k_gemm16_beside(Gemm16Args a, Gemm16Args w, int first) {
  extern __shared__ __align__(16) uint8_t smem[];
  if ((int)blockIdx.x < first)
    INPUT::run(a, smem, blockIdx.x, first);
  else
    WEIGHT::run(w, smem, blockIdx.x - first, gridDim.x - first);
}

template <typename T, typename OA, typename OW>
hipError_t run_beside(const Gemm16Args& a, const Gemm16Args& w, hipStream_t stream) {
  using INPUT = Gemm16<kInput, 64, 128, 1, 4, 2, T, OA>;
  using WEIGHT = Gemm16<kWeight, 64, 128, 1, 4, 2, T, OW>;
  int cus = 0;
  hipError_t e = allow_lds<&k_gemm16_beside<INPUT, WEIGHT>>(kLds);
  if (e == hipSuccess) e = compute_units(&cus);
  if (e != hipSuccess) return e;
  const unsigned first = gemm16_blocks<INPUT>(a, 3, cus), behind = gemm16_blocks<WEIGHT>(w, 3, cus);
  timing_begin(stream);
  hipLaunchKernelGGL((k_gemm16_beside<INPUT, WEIGHT>), dim3(first + behind), dim3(INPUT::THREADS),
                     INPUT::smem_bytes(a.E), stream, a, w, (int)first);
  timing_end(stream);
  return hipGetLastError();
}

template <typename T, typename OA, typename OW>
hipError_t run_both(const Gemm16Args& a, const Gemm16Args& w, hipStream_t stream) {
  using INPUT = Gemm16<kInput, 256, 256, 2, 4, 2, T, OA>;
  using WEIGHT = Gemm16<kWeight, 256, 256, 2, 4, 2, T, OW>;
  unsigned grid = 0;
  int bytes = 0;
  hipError_t e = gemm16_grid<Both<INPUT, WEIGHT>, &k_gemm16_both<INPUT, WEIGHT>>(a, 0, &grid, &bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_gemm16_queue, dim3(1), dim3(16), 0, stream, a.queue, (int)grid / 8);   // both: w's follows
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  timing_begin(stream);
  hipLaunchKernelGGL((k_gemm16_both<INPUT, WEIGHT>), dim3(grid), dim3(INPUT::THREADS), bytes, stream, a, w);
  timing_end(stream);
  return hipGetLastError();
}

}  // namespace

size_t gemm16_backward_workspace_bytes(int M, int E, int N, int K) {
  if (M == 0) return 0;
  const size_t a = gemm16_part_bytes(kInput, M, E, N, K), w = gemm16_part_bytes(kWeight, M, E, N, K);
  return 2 * kQueueBytes + (a > w ? a : w);
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
  if (da && dw && M && p.beside) {
    const Gemm16Args ga{dc, w, offsets, E, M, N, K, da, 1, 0, nullptr};
    const Gemm16Args gw{dc, a, offsets, E, M, N, K, dw, 1, 0, nullptr};
    return by_types(type, da_type, [&](auto t, auto oa) {
      using T = decltype(t);
      using OA = decltype(oa);
      return dw_type == 2 ? run_beside<T, OA, float>(ga, gw, stream) : run_beside<T, OA, T>(ga, gw, stream);
    });
  }
  hipError_t e = hipSuccess;
  if (da && M) e = launch_gemm16_input(dc, w, type, offsets, E, M, N, K, da_type, da, ws, stream);
  if (e == hipSuccess && dw) e = launch_gemm16_weight(dc, a, type, offsets, E, M, N, K, dw_type, dw, ws, stream);
  return e;
}

}  // namespace zinc
