// Launches of the adapters' kernels (lora_device.hpp), by type and rank.
#pragma once

#include "lora_device.hpp"
#include "launch.hpp"

namespace zinc {

hipError_t launch_lora_shrink(const ShrinkArgs& s, int type, bool w_t, hipStream_t stream);
hipError_t launch_lora_expand(ExpandArgs s, int type, bool w_t, hipStream_t stream);
hipError_t launch_lora_grad(const LoraGradArgs& s, int type, bool j_first, hipStream_t stream);

// Row tiles of 16 a workgroup takes: four where an adapter has rows for them (fewer with the rank, by the
// registers that the sums and operands take).
inline int lora_row_tiles(int M, int E, int rank) {
  if (M / E <= 24) return 1;
  return rank <= 64 ? 4 : rank <= 128 ? 2 : 1;
}

template <int V>
struct Int {
  static constexpr int value = V;
};

// f(T, JT): the type and the tiles of 16 that hold the rank.
template <typename T, typename F>
hipError_t by_rank(int rank, F f) {
  if (rank <= 16) return f(T{}, Int<1>{});
  if (rank <= 32) return f(T{}, Int<2>{});
  if (rank <= 64) return f(T{}, Int<4>{});
  if (rank <= 128) return f(T{}, Int<8>{});
  return f(T{}, Int<16>{});
}
template <typename F>
hipError_t by_type_and_rank(int type, int rank, F f) {
  return type == 0 ? by_rank<_Float16>(rank, f) : by_rank<__bf16>(rank, f);
}

}  // namespace zinc
