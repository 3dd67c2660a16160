#include "lora_launch.hpp"

namespace zinc {
namespace {

template <typename KERNEL>
__global__ __launch_bounds__(256) void k_lora_expand(ExpandArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, smem);
}

template <typename KERNEL>
hipError_t run(ExpandArgs s, hipStream_t stream) {
  const hipError_t e = allow_lds<KERNEL>(reinterpret_cast<const void*>(&k_lora_expand<KERNEL>), kLds);
  if (e != hipSuccess) return e;
  s.row_tiles = (int)max_row_tiles(s.plan.M, s.plan.E, KERNEL::TM);
  const int copies = s.base == s.y ? 0 : (s.plan.M + kCopied - 1) / kCopied;
  hipLaunchKernelGGL(k_lora_expand<KERNEL>, dim3(s.row_tiles + copies, (s.N + kSpan - 1) / kSpan), dim3(256),
                     KERNEL::smem_bytes(), stream, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_expand(ExpandArgs s, int type, bool w_t, hipStream_t stream) {
  const bool few = lora_row_tiles(s.plan.M, s.plan.E, s.rank) == 1;
  return by_type_and_rank(type, s.rank, [&](auto t, auto jt) {
    using T = decltype(t);
    constexpr int JT = decltype(jt)::value, RT = JT <= 4 ? 4 : JT == 8 ? 2 : 1;
    if (few) return w_t ? run<Expand<T, JT, 1, true>>(s, stream) : run<Expand<T, JT, 1, false>>(s, stream);
    return w_t ? run<Expand<T, JT, RT, true>>(s, stream) : run<Expand<T, JT, RT, false>>(s, stream);
  });
}

}  // namespace zinc
