#include "lora_launch.hpp"

namespace zinc {
namespace {

template <typename KERNEL>
__global__ __launch_bounds__(256) void k_lora_shrink(ShrinkArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, smem);
}

template <typename KERNEL>
hipError_t run(const ShrinkArgs& s, hipStream_t stream) {
  const hipError_t e = allow_lds<KERNEL>(reinterpret_cast<const void*>(&k_lora_shrink<KERNEL>), kLds);
  if (e != hipSuccess) return e;
  const long long tiles = max_row_tiles(s.plan.M, s.plan.E, KERNEL::TM);
  hipLaunchKernelGGL(k_lora_shrink<KERNEL>, dim3((unsigned)(tiles * s.splits)), dim3(256), KERNEL::smem_bytes(),
                     stream, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_shrink(const ShrinkArgs& s, int type, bool w_t, hipStream_t stream) {
  const bool few = lora_row_tiles(s.plan.M, s.plan.E, s.rank) == 1;
  return by_type_and_rank(type, s.rank, [&](auto t, auto jt) {
    using T = decltype(t);
    constexpr int JT = decltype(jt)::value, RT = JT <= 4 ? 4 : JT == 8 ? 2 : 1;
    if (few) return w_t ? run<Shrink<T, JT, 1, true>>(s, stream) : run<Shrink<T, JT, 1, false>>(s, stream);
    return w_t ? run<Shrink<T, JT, RT, true>>(s, stream) : run<Shrink<T, JT, RT, false>>(s, stream);
  });
}

}  // namespace zinc
