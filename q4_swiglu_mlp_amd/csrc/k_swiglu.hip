// SwiGLU of rows and its gradients, elementwise:
//   h = silu(g) u,   dg = dh u s (1 + g (1 - s)),   du = dh g s,   s = 1 / (1 + e^-g)
// in fp32, rounded once to the rows' type.  Bound by the memory: one read of each input and one write of
// each output, eight values a lane at a time.
#include "fp8_device.hpp"
#include "launch.hpp"
#include "silu.hpp"

namespace zinc {
namespace {

template <typename T, bool STREAMED>
__global__ __launch_bounds__(256) void k_swiglu(const T* __restrict__ gate, const T* __restrict__ up, size_t n,
                                                T* __restrict__ h) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (size_t)gridDim.x * 2048) {
    float g[8], u[8], v[8];
    load8(gate + i, g);
    load8(up + i, u);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const Sigmoid s = sigmoid(g[r]);
      v[r] = (u[r] * s.factor) * (g[r] * s.value) * s.factor;
    }
    store8<STREAMED>(h + i, v);
  }
}

template <typename T, bool STREAMED>
__global__ __launch_bounds__(256) void k_swiglu_backward(const T* __restrict__ dh, const T* __restrict__ gate,
                                                         const T* __restrict__ up, size_t n, T* __restrict__ dgate,
                                                         T* __restrict__ dup) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (size_t)gridDim.x * 2048) {
    float d[8], g[8], u[8], dg[8], du[8];
    load8(dh + i, d);
    load8(gate + i, g);
    load8(up + i, u);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const Sigmoid s = sigmoid(g[r]);
      // dh, up and s^2 may each leave what fp32 holds of the others' product: their exponents are added apart.  (0 g
      // is NaN for an infinite gate, as s g is.)
      const float slope = fmaf(g[r], 0.0f, s.value * fmaf(g[r], s.rest, 1.0f));
      const int exponent = __builtin_amdgcn_frexp_expf(d[r]) + __builtin_amdgcn_frexp_expf(u[r]) - 2 * s.half;
      dg[r] = __builtin_amdgcn_ldexpf(
          __builtin_amdgcn_frexp_mantf(d[r]) * __builtin_amdgcn_frexp_mantf(u[r]) * slope, exponent);
      du[r] = (d[r] * s.factor) * (g[r] * s.value) * s.factor;
    }
    store8<STREAMED>(dgate + i, dg);
    store8<STREAMED>(dup + i, du);
  }
}

// Outputs that the last-level cache (256 MB) does not hold beside the inputs are stored past the caches: 8192 x
// 11008 bf16 90.0 us against 91.1, its gradients 156.7 against 157.7; fp32 182.8 against 179.3, 312.3 against 313.9
// (and just above the size, 32768 x 768 fp32, 52.5 against 46.3).
template <typename T>
void forward(const void* gate, const void* up, size_t n, void* h, unsigned blocks, hipStream_t stream) {
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, stream, static_cast<const T*>(gate),
                       static_cast<const T*>(up), n, static_cast<T*>(h));
  };
  if (3 * n * sizeof(T) > (256u << 20))
    run(k_swiglu<T, true>);
  else
    run(k_swiglu<T, false>);
}
template <typename T>
void backward(const void* dh, const void* gate, const void* up, size_t n, void* dgate, void* dup, unsigned blocks,
              hipStream_t stream) {
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, stream, static_cast<const T*>(dh),
                       static_cast<const T*>(gate), static_cast<const T*>(up), n, static_cast<T*>(dgate),
                       static_cast<T*>(dup));
  };
  if (5 * n * sizeof(T) > (256u << 20))
    run(k_swiglu_backward<T, true>);
  else
    run(k_swiglu_backward<T, false>);
}

// One round of 2048 values a workgroup (8192 x 11008 bf16 90 us, its gradients 157; eight rounds 98 and 172).
unsigned blocks_for(size_t n) {
  const size_t blocks = (n + 2047) / 2048;
  return (unsigned)(blocks < 65536 ? blocks : 65536);
}

}  // namespace

hipError_t launch_swiglu(const void* gate, const void* up, int type, size_t n, void* h, hipStream_t stream) {
  const unsigned blocks = blocks_for(n);
  if (type == 0)
    forward<_Float16>(gate, up, n, h, blocks, stream);
  else if (type == 1)
    forward<__bf16>(gate, up, n, h, blocks, stream);
  else
    forward<float>(gate, up, n, h, blocks, stream);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* dh, const void* gate, const void* up, int type, size_t n, void* dgate,
                                  void* dup, hipStream_t stream) {
  const unsigned blocks = blocks_for(n);
  if (type == 0)
    backward<_Float16>(dh, gate, up, n, dgate, dup, blocks, stream);
  else if (type == 1)
    backward<__bf16>(dh, gate, up, n, dgate, dup, blocks, stream);
  else
    backward<float>(dh, gate, up, n, dgate, dup, blocks, stream);
  return hipGetLastError();
}

}  // namespace zinc
