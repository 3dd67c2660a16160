// The adapters' gradients in two launches: both first products (A x and B^T dy), then everything that
// is made of them, dx and the gradients of A and B; and a third where those of few columns are summed in parts.
#include "lora_launch.hpp"

namespace zinc {
namespace {

template <typename H, typename DH>
__global__ __launch_bounds__(256, lora_held(H::kTiles)) void k_lora_firsts(ShrinkArgs h, ShrinkArgs dh, int h_blocks) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int block = blockIdx.x;
  if (block < h_blocks)
    H::run(h, block, smem);
  else
    DH::run(dh, block - h_blocks, smem);
}

template <typename DX, typename DA, typename DB>
__global__ __launch_bounds__(256, lora_held(DX::kTiles)) void k_lora_seconds(ExpandArgs dx, LoraGradArgs da,
                                                                               LoraGradArgs db, int a_blocks,
                                                                               int b_blocks) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int block = blockIdx.x;
  if (block < a_blocks)
    DA::run(da, block, smem);
  else if (block < a_blocks + b_blocks)
    DB::run(db, block - a_blocks, smem);
  else
    DX::run(dx, block - a_blocks - b_blocks, smem);
}

// A gradient's parts, and what their sum times the adapter's scale goes to.
struct JoinArgs {
  const float* parts;
  int splits;
  size_t each, n;   // values an adapter, and in all; 0: nothing to join
  void* out;
};

template <typename T>
__global__ __launch_bounds__(256) void k_lora_join(JoinArgs a, JoinArgs b, LoraPlan plan,
                                                    const float* __restrict__ scales) {
  const JoinArgs& g = blockIdx.y ? b : a;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < g.n; i += (size_t)gridDim.x * 1024) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(g.parts + i);
    for (int s = 1; s < g.splits; ++s) v += *reinterpret_cast<const f32x4_t*>(g.parts + s * g.n + i);
    int lo, hi;
    positions_of(plan, (int)(i / g.each), lo, hi);
    const float scale = grad_scale(scales, (int)(i / g.each), hi > lo);
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (T)(scale * v[r]);
    *reinterpret_cast<T4*>(static_cast<T*>(g.out) + i) = o;
  }
}

}  // namespace

size_t lora_backward_workspace_bytes(int M, int E, int K, int N, int rank) {
  return 2 * lora_part_bytes(M, rank) + grad_bytes(M, E, rank, K) + grad_bytes(M, E, rank, N);
}

hipError_t launch_lora_backward(const void* dy, const void* x, const void* a, const void* b, const float* scales,
                                const int32_t* offsets, const int32_t* slot_row, const int32_t* row_slot, int E, int M,
                                int K, int N, int rank, int type, const void* base, void* dx, void* da, void* db,
                                void* ws, hipStream_t stream) {
  const LoraPlan plan{offsets, slot_row, row_slot, E, M};
  char* at = static_cast<char*>(ws);
  const size_t part = lora_part_bytes(M, rank);
  float* parts_a = reinterpret_cast<float*>(at + 2 * part);
  float* parts_b = reinterpret_cast<float*>(at + 2 * part + grad_bytes(M, E, rank, K));
  const ShrinkArgs h = shrink_of(false, plan, x, a, K, rank, reinterpret_cast<float*>(at));
  const ShrinkArgs dh = shrink_of(false, plan, dy, b, N, rank, reinterpret_cast<float*>(at + part));
  const ExpandArgs ex = expand_of(false, dh, a, K, scales, base, dx);
  const int sa = grad_splits(M, E, K), sb = grad_splits(M, E, N);
  const LoraGradArgs ga{plan, x, dh.parts, dh.splits, rank, K, scales, sa, sa > 1 ? static_cast<void*>(parts_a) : da};
  const LoraGradArgs gb{plan, dy, h.parts, h.splits, rank, N, scales, sb, sb > 1 ? static_cast<void*>(parts_b) : db};
  hipError_t e = by_kind(type, M, E, rank, [&](auto t, auto jt, auto r) {
    using T = decltype(t);
    constexpr int JT = decltype(jt)::value, R = decltype(r)::value;
    using H = Shrink<T, JT, R, false>;
    using DH = Shrink<T, JT, R, true>;
    using DX = Expand<T, JT, R, true>;
    using DA = LoraGrad<T, JT, true>;
    using DB = LoraGrad<T, JT, false>;
    const size_t first = H::smem_bytes() > DH::smem_bytes() ? H::smem_bytes() : DH::smem_bytes();
    const size_t second = DX::smem_bytes() > DA::smem_bytes() ? DX::smem_bytes() : DA::smem_bytes();
    hipError_t e = allow_lds<&k_lora_firsts<H, DH>>(kLds);
    if (e == hipSuccess) e = allow_lds<&k_lora_seconds<DX, DA, DB>>(kLds);
    if (e != hipSuccess) return e;
    const long long h_blocks = M && db ? shrink_blocks(false, h) : 0;
    const long long dh_blocks = M && (dx || da) ? shrink_blocks(false, dh) : 0;
    if (h_blocks + dh_blocks) {
      hipLaunchKernelGGL((k_lora_firsts<H, DH>), dim3((unsigned)(h_blocks + dh_blocks)), dim3(256), first, stream,
                         h, dh, (int)h_blocks);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const long long a_blocks = da ? grad_blocks(ga) : 0, b_blocks = db ? grad_blocks(gb) : 0;
    const long long x_blocks = dx ? expand_blocks(ex) : 0;
    if (a_blocks + b_blocks + x_blocks == 0) return e;
    hipLaunchKernelGGL((k_lora_seconds<DX, DA, DB>), dim3((unsigned)(a_blocks + b_blocks + x_blocks)), dim3(256),
                       second, stream, ex, ga, gb, (int)a_blocks, (int)b_blocks);
    return hipGetLastError();
  });
  const JoinArgs ja{parts_a, sa, (size_t)rank * K, da && sa > 1 ? (size_t)E * rank * K : 0, da};
  const JoinArgs jb{parts_b, sb, (size_t)rank * N, db && sb > 1 ? (size_t)E * rank * N : 0, db};
  const size_t most = ja.n > jb.n ? ja.n : jb.n;
  if (e != hipSuccess || most == 0) return e;
  const dim3 grid((unsigned)((most + 1023) / 1024 < 1024 ? (most + 1023) / 1024 : 1024), 2);
  if (type == 0)
    hipLaunchKernelGGL(k_lora_join<_Float16>, grid, dim3(256), 0, stream, ja, jb, plan, scales);
  else
    hipLaunchKernelGGL(k_lora_join<__bf16>, grid, dim3(256), 0, stream, ja, jb, plan, scales);
  return hipGetLastError();
}

}  // namespace zinc
