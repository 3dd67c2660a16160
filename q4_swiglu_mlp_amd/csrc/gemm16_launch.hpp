// Launches of the 16-bit products by group (gemm16_tile.hpp), by types and shape.
#pragma once

#include "gemm16_tile.hpp"
#include "launch.hpp"

namespace zinc {

// As many persistent workgroups as the CUs hold, a multiple of the eight XCDs.
template <Product F, int TM, int TN, int WM, int WN, typename T, typename O>
hipError_t run_gemm16(const Gemm16Args& g, hipStream_t stream) {
  using KERNEL = Gemm16<F, TM, TN, WM, WN, T, O>;
  const int cols = F == kForward ? g.N : g.K, bytes = (int)KERNEL::smem_bytes(g.E);
  const long long row_tiles = F == kWeight ? (long long)g.E * ((g.N + TM - 1) / TM) : max_row_tiles(g.M, g.E, TM);
  hipError_t e = allow_lds<KERNEL>(reinterpret_cast<const void*>(&k_gemm16<KERNEL>), kLds);
  int cus = 0;
  if (e == hipSuccess) e = compute_units(&cus);
  if (e != hipSuccess) return e;
  const int held = kLds / bytes < KERNEL::HELD ? kLds / bytes : KERNEL::HELD;
  const long long units = row_tiles * ((cols + TN - 1) / TN), room = (long long)cus * held;
  const long long blocks = units < room ? units : room;
  timing_begin(stream);
  hipLaunchKernelGGL(k_gemm16<KERNEL>, dim3((unsigned)((blocks + 7) / 8 * 8)), dim3(KERNEL::THREADS), bytes, stream,
                     g);
  timing_end(stream);
  return hipGetLastError();
}

// f<T, O>() for the type codes of the operands (0 fp16, 1 bf16) and of the output (the same, or 2 fp32).
template <typename F>
hipError_t by_types(int type, int out_type, F f) {
  if (type == 0) return out_type == 2 ? f(_Float16{}, 0.0f) : f(_Float16{}, _Float16{});
  return out_type == 2 ? f(__bf16{}, 0.0f) : f(__bf16{}, __bf16{});
}

}  // namespace zinc
