#include "lora_launch.hpp"

namespace zinc {
namespace {

template <typename KERNEL>
__global__ __launch_bounds__(256, KERNEL::TM == 64 ? 1 : lora_held(KERNEL::kTiles)) void k_lora_shrink(ShrinkArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, blockIdx.x, smem);
}

template <typename KERNEL>
__global__ __launch_bounds__(256, 2) void k_lora_expand(ExpandArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, blockIdx.x, smem);
}

}  // namespace

size_t lora_workspace_bytes(int M, int rank) { return lora_part_bytes(M, rank); }

hipError_t launch_lora(const void* x, const void* a, const void* b, const float* scales, const int32_t* offsets,
                       const int32_t* slot_row, const int32_t* row_slot, int E, int M, int K, int N, int rank, int type,
                       const void* base, void* y, void* ws, hipStream_t stream) {
  const LoraPlan plan{offsets, slot_row, row_slot, E, M};
  const ShrinkArgs s = shrink_of(true, plan, x, a, K, rank, static_cast<float*>(ws));
  const ExpandArgs x2 = expand_of(true, s, b, N, scales, base, y);
  return by_kind(type, M, E, rank, [&](auto t, auto jt, auto r) {
    constexpr int JT = decltype(jt)::value, R = decltype(r)::value;
    using SHRINK = Shrink<decltype(t), JT, lora_forward_tiles(JT, R), false>;
    using EXPAND = Expand<decltype(t), JT, lora_forward_tiles(JT, R), false>;
    hipError_t e = allow_lds<&k_lora_shrink<SHRINK>>(kLds);
    if (e == hipSuccess) e = allow_lds<&k_lora_expand<EXPAND>>(kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_lora_shrink<SHRINK>, dim3((unsigned)shrink_blocks(true, s)), dim3(256), SHRINK::smem_bytes(),
                       stream, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_lora_expand<EXPAND>, dim3((unsigned)expand_blocks(x2)), dim3(256), EXPAND::smem_bytes(),
                       stream, x2);
    return hipGetLastError();
  });
}

}  // namespace zinc
