#include "lora_launch.hpp"

namespace zinc {
namespace {

template <typename KERNEL>
__global__ __launch_bounds__(256) void k_lora_grad(LoraGradArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, smem);
}

// out = s_e times the sum of the parts, in their order; `each` values an adapter.
template <typename T>
__global__ __launch_bounds__(256) void k_lora_join(const float* __restrict__ parts, int splits, size_t each, size_t n,
                                                   const float* __restrict__ scales, T* __restrict__ out) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (size_t)gridDim.x * 1024) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(parts + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(parts + s * n + i);
    const float scale = scales ? scales[i / each] : 1.0f;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (T)(scale * v[r]);
    *reinterpret_cast<T4*>(out + i) = o;
  }
}

template <typename KERNEL>
hipError_t run(const LoraGradArgs& s, hipStream_t stream) {
  const hipError_t e = allow_lds<KERNEL>(reinterpret_cast<const void*>(&k_lora_grad<KERNEL>), kLds);
  if (e != hipSuccess) return e;
  const long long blocks = (long long)s.plan.E * s.splits * ((s.C + 63) / 64);
  hipLaunchKernelGGL(k_lora_grad<KERNEL>, dim3((unsigned)blocks), dim3(256), KERNEL::smem_bytes(), stream, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_grad(const LoraGradArgs& s, int type, bool j_first, hipStream_t stream) {
  return by_type_and_rank(type, s.rank, [&](auto t, auto jt) {
    using T = decltype(t);
    constexpr int JT = decltype(jt)::value;
    return j_first ? run<LoraGrad<T, JT, true>>(s, stream) : run<LoraGrad<T, JT, false>>(s, stream);
  });
}

hipError_t launch_lora_join(const float* parts, int splits, size_t each, size_t n, const float* scales, int type,
                            void* out, hipStream_t stream) {
  const size_t blocks = (n + 1023) / 1024;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
  if (type == 0)
    hipLaunchKernelGGL(k_lora_join<_Float16>, grid, dim3(256), 0, stream, parts, splits, each, n, scales,
                       static_cast<_Float16*>(out));
  else
    hipLaunchKernelGGL(k_lora_join<__bf16>, grid, dim3(256), 0, stream, parts, splits, each, n, scales,
                       static_cast<__bf16*>(out));
  return hipGetLastError();
}

}  // namespace zinc
