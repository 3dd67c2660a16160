// Products of e4m3 matrices with one fp32 scale per block of 128:
//   c[m][n] = sum_kb sa[m][kb] sw[n / 128][kb] sum_{k in block kb} a[m][k] w[n][k]
// dense, or grouped: rows offsets[e] .. offsets[e + 1] - 1 of a take expert e's w.
//
// The MFMA (16x16x128, one block of 128 per instruction) runs with w as its
// row operand and a as its column operand: a lane then holds four columns n of
// one row m, its two scales are one product per 16x16 tile, and it stores four
// neighbouring outputs.  The block's partial sum starts from zero and is added
// to the fp32 accumulator with that product, so the scales cost one FMA per
// output and block.
//
// Precision.  The FP8 MFMA adds products in groups of eight neighbouring k: they
// are aligned to the group's largest (by operand exponents) and cut at 2^-13 of
// it; the groups then add in fp32.  Products have eight bits, so only those
// below 2^-6 of a group's largest lose any: measured 1.5e-5 of the result
// (2-norm, normal data, K = 128), far below the rounding of a 16-bit output (2e-4
// fp16, 1.7e-3 bf16).  fp32 outputs (the expert rows of an fp16 or fp32 layer too; a bf16
// layer's take the FP8 MFMA) and the products that feed an expert layer's second
// quantisation take the fp16 MFMA on exactly converted operands instead: half the rate, 7e-9
// of the result.  In that quantisation 1.5e-5 moves a value in 5000 to the next code, which is
// 1.2e-3 of y beside the 2e-4 and 1.7e-3 of its own rounding (a bf16 layer of 4001 tokens has
// 1.7e-3 in all, as in plain fp32; with the FP8 MFMA there, and 16-bit expert rows, 3.3e-3).
//
// What bounds it (TB/s and TFLOP/s of the whole call):
// - few rows, the pass over w: 1 x 11008 x 4096 12.7 us, 3.6 TB/s, with w in HBM;
// - many rows, the matrix units at the clock that the power limit leaves (about 1.9 GHz):
//   8192 x 11008 x 4096 bf16 330 us, 2240 TFLOP/s, 379 us with weights that come from HBM
//   (up to 5 % more on other cards); fp32 by fp16 MFMAs 480 us for 8192 x 8192 x 4096, 1145 TFLOP/s.
#include "fp8_stream.hpp"
#include "launch.hpp"

namespace zinc {
namespace {

// As many persistent workgroups as the CUs hold, a multiple of the eight XCDs.
template <typename KERNEL>
hipError_t run_tiles(GemmArgs g, int TM, int splits, hipStream_t stream) {
  g.row_tiles = (int)max_row_tiles(g.M, g.offsets ? g.E : 0, TM);
  g.col_tiles = (g.N + KERNEL::COLS - 1) / KERNEL::COLS;
  g.splits = splits;
  const int bytes = (int)KERNEL::smem_bytes(g.offsets ? g.E : 0);
  hipError_t e = allow_lds<&k_fp8_tile<KERNEL>>(kLds);
  int cus = 0;
  if (e == hipSuccess) e = compute_units(&cus);
  if (e != hipSuccess) return e;
  const int held = kLds / bytes < KERNEL::HELD ? kLds / bytes : KERNEL::HELD;
  const long long units = (long long)g.row_tiles * g.col_tiles * splits, room = (long long)cus * held;
  const long long blocks = units < room ? units : room;
  timing_begin(stream);
  hipLaunchKernelGGL(k_fp8_tile<KERNEL>, dim3((unsigned)((blocks + 7) / 8 * 8)), dim3(KERNEL::THREADS), bytes, stream,
                     g);
  timing_end(stream);
  return hipGetLastError();
}

// Weight streams: the blocks of 128 of a that fit LDS beside the rings, two
// workgroups a CU where all of them fit so, else one.
template <typename KERNEL>
hipError_t run_stream(StreamArgs s, int cols, hipStream_t stream) {
  GemmArgs& g = s.g;
  const int KB = (g.K + 127) / 128, all = (KB + s.ks - 1) / s.ks * s.ks;
  s.rows = g.M < KERNEL::TM ? g.M : KERNEL::TM;
  s.chunk = all;
  if (KERNEL::smem_bytes(s.rows, all) > kLds / 2) {
    while (KERNEL::smem_bytes(s.rows, s.chunk) > kLds) s.chunk -= s.ks;
  }
  const size_t bytes = KERNEL::smem_bytes(s.rows, s.chunk);
  g.row_tiles = (int)max_row_tiles(g.M, g.offsets ? g.E : 0, KERNEL::TM);
  g.col_tiles = (g.N + cols - 1) / cols;
  const hipError_t e = allow_lds<&k_fp8_stream<KERNEL>>(kLds);
  if (e != hipSuccess) return e;
  timing_begin(stream);
  hipLaunchKernelGGL(k_fp8_stream<KERNEL>, dim3((unsigned)((long long)g.row_tiles * g.col_tiles)),
                     dim3(KERNEL::THREADS), bytes, stream, s);
  timing_end(stream);
  return hipGetLastError();
}

// c = the sum of the parts of K, in their order.  A thread takes four values; bound by
// launch and HBM or L2: 3 us for eight parts of 64 x 4096.
template <typename T>
__global__ __launch_bounds__(256) void k_join_parts(const float* __restrict__ parts, size_t part, int splits,
                                                    size_t total, T* __restrict__ c) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total; i += (size_t)gridDim.x * 1024) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(parts + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(parts + s * part + i);
    if (i + 4 <= total) {
      typedef T T4 __attribute__((ext_vector_type(4)));
      T4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = (T)v[r];
      *reinterpret_cast<T4*>(c + i) = o;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (i + r < total) c[i + r] = (T)v[r];
    }
  }
}

// How a product is cut, by its sizes alone.  Times: us, 256 CUs, bf16 output, calls replayed; on one
// weight, which the last-level cache holds, where nothing else is said.
enum Shape { kStream, kSmall, kMiddle, kLarge, kLargest };
struct Cut {
  Shape shape;
  int splits;
};

// Dense.
// - Up to 4 rows the weight's stream: 11008 x 4096 12.1 against 12.8 for the best parts of
//   small tiles, 4096 x 11008 14.7 and 15.2, 4096 x 4096 7.8 and 9.9; with 8 rows 13.3
//   and 12.9, 18.2 and 15.3, 9.3 and 10.1; with 16 rows 16.1 and 13.2, 24 and 15.6.  Weights
//   from HBM: 14.2 and 16.0, 18.0 and 18.4, 8.8 and 12.0; 8 rows 15.3 and 16.2, 20.8 and
//   18.3, 9.9 and 12.1; 16 rows 17.7 and 16.6, 26.5 and 18.6, 12.5 and 12.4.
// - Else the largest tile (256 x 256, 128 x 256) with 160 units, five eighths of the CUs:
//   1024 x 11008 x 4096 53 with the first (172 units) against 74 with small tiles, 512 rows
//   35 with the second against 49 and 39, 2048 x 4096 x 11008 (128 and 256 units) 95 with
//   the second against 121 with the first.
// - Else small tiles (64 x 128), in parts of K that make one and a half units a CU, eight at
//   most, of five blocks or more: 64 x 11008 x 4096 16.2 in four parts, 17.1 in three
//   or five, 22 in one; 64 x 4096 x 11008 17.4 in eight, 18.2 in six, 20.3 in twelve, 52 in
//   one; 64 x 4096 x 4096 13.3 in six, 13.2 in four, 14.6 in eight.
Cut cut_dense(int M, int N, int K) {
  if (M <= 4) return {kStream, 1};
  const long long rows256 = (M + 255) / 256, cols256 = (N + 255) / 256, rows128 = (M + 127) / 128;
  if (rows256 * cols256 >= 160) return {kLargest, 1};
  if (rows128 * cols256 >= 160) return {kLarge, 1};
  const long long units = (long long)((M + 63) / 64) * ((N + 127) / 128);
  const int KB = (K + 127) / 128;
  int splits = (int)((380 + units / 2) / units);
  splits = splits > 8 ? 8 : splits;
  splits = splits > KB / 5 ? KB / 5 : splits;
  splits = splits < 1 ? 1 : splits;
  const int each = (KB + splits - 1) / splits;
  return {kSmall, (KB + each - 1) / each};   // no part is empty
}

// Grouped, by the mean rows of an expert.  64 experts of uneven sizes, 768 x 2048: 128 rows 43
// with small tiles, 46 with 128 x 128, 44 with 256 x 256; 192 rows 54, 52 and 66; 256 rows 61,
// 56 and 70; 384 rows 85, 80 and 76; 1024 rows 190, 164 and 142.  Where the sizes are even, an
// expert below 256 rows fills one tile of 256, which the mean cannot tell: 64 x 768 x 2048, 192 rows
// 51, 47 and 39, 256 rows 61, 59 and 73; 16 x 1536 x 4096, 192 rows 55, 52 and 66, 256 rows 72, 58
// and 71, 384 rows 81, 88 and 67; 128 x 512 x 2048, 192 rows 63, 55 and 47, 256 rows 78, 71 and 78;
// 8 x 14336 x 4096, 128 rows 183, 173 and 139, 256 rows 243, 248 and 209.
Shape cut_grouped(int rows, int E) {
  const int mean = rows / E;
  return mean <= 160 ? kSmall : mean <= 320 ? kMiddle : kLargest;
}

// Values from one part of K to the next, a multiple of eight.
size_t part_values(int M, int N) { return ((size_t)M * N + 7) / 8 * 8; }

template <bool EXACT, typename T>
hipError_t small_tiles(const GemmArgs& g, int splits, hipStream_t stream) {
  return run_tiles<TileKernel<64, 128, 1, 4, EXACT, false, T>>(g, 64, splits, stream);
}

// Twice the operand registers leave the fp16 MFMAs the 128 x 256 tile.
template <bool EXACT, typename T>
hipError_t largest_tiles(const GemmArgs& g, hipStream_t stream) {
  if constexpr (EXACT)
    return run_tiles<TileKernel<128, 256, 2, 4, true, false, T>>(g, 128, 1, stream);
  else
    return run_tiles<TileKernel<256, 256, 2, 4, false, false, T>>(g, 256, 1, stream);
}

template <bool EXACT, typename T>
hipError_t dense(GemmArgs g, void* ws, hipStream_t stream) {
  const Cut how = cut_dense(g.M, g.N, g.K);
  if (how.shape == kLargest) return largest_tiles<EXACT, T>(g, stream);
  if (how.shape == kLarge) return run_tiles<TileKernel<128, 256, 2, 4, EXACT, false, T>>(g, 128, 1, stream);
  if (how.shape == kStream) {
    // ks waves share 16 columns: as many as make 1280 waves, eight at most; one alone from 2048 on.
    // Weights from HBM, one row, K = 4096: N = 4096 8.1 us with eight, 8.7 with four, 11.5 with two;
    // 6144 10.7, 9.5 and 11.8; 11008 15.0 with four, 13.9 with two, 20.0 with one; 16384 19.9, 18.1 and
    // 20.9; 22016 24.7 with two, 23.5 with one; 32768 31.3 and 36.3 (four rows 34.2 and 35.8)
    StreamArgs s{};
    s.g = g;
    const int tiles = (g.N + 15) / 16;
    s.ks = tiles >= 2048 ? 1 : tiles >= 640 ? 2 : tiles >= 320 ? 4 : 8;
    return run_stream<StreamKernel<8, 4, false, float, T>>(s, 8 / s.ks * 16, stream);
  }
  if (how.splits == 1) return small_tiles<EXACT, T>(g, 1, stream);
  T* c = static_cast<T*>(g.c);
  g.c = ws;
  g.part = part_values(g.M, g.N);
  const hipError_t e = small_tiles<EXACT, float>(g, how.splits, stream);
  if (e != hipSuccess) return e;
  const size_t total = (size_t)g.M * g.N, blocks = (total + 1023) / 1024;
  hipLaunchKernelGGL(k_join_parts<T>, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream,
                     static_cast<const float*>(ws), g.part, how.splits, total, c);
  return hipGetLastError();
}

template <bool EXACT, typename T>
hipError_t grouped(const GemmArgs& g, hipStream_t stream) {
  const Shape shape = cut_grouped(g.M, g.E);
  if (shape == kSmall) return small_tiles<EXACT, T>(g, 1, stream);
  if (shape == kMiddle) return run_tiles<TileKernel<128, 128, 2, 2, EXACT, false, T>>(g, 128, 1, stream);
  return largest_tiles<EXACT, T>(g, stream);
}

template <bool EXACT, typename T>
hipError_t gemm(const GemmArgs& g, void* ws, hipStream_t stream) {
  return g.offsets ? grouped<EXACT, T>(g, stream) : dense<EXACT, T>(g, ws, stream);
}

template <typename T_IN>
hipError_t stream_gate_up(const StreamArgs& s, hipStream_t stream) {
  return run_stream<StreamKernel<16, 3, true, T_IN, float>>(s, 128, stream);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The expert call's workspace.  The experts' output rows are terms of y's sum: fp32, so that y's
// rounding is the only one to 16 bits, and no row leaves fp16's range before its weight.
struct ExpertsPlan {
  int32_t *offsets, *slot_row, *row_slot;
  void* sort_ws;
  uint8_t *xq, *hq;
  float *xs, *hs;
  float* ys;
};

ExpertsPlan carve(void* ws, int M, int top_k, int E, int H, int I, size_t* total) {
  ExpertsPlan p;
  char* base = static_cast<char*>(ws);
  size_t off = 0;
  const size_t S = (size_t)M * top_k;
  auto take = [&](size_t bytes) { char* r = base ? base + off : nullptr; off += align256(bytes); return r; };
  p.offsets = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * (E + 1)));
  p.slot_row = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * S));
  p.row_slot = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * S));
  p.sort_ws = take(moe_sort_workspace_bytes((int)S, E));
  p.xq = reinterpret_cast<uint8_t*>(take(S * H));
  p.xs = reinterpret_cast<float*>(take(S * (H / 128) * 4));
  p.hq = reinterpret_cast<uint8_t*>(take(S * I));
  p.hs = reinterpret_cast<float*>(take(S * (I / 128) * 4));
  p.ys = reinterpret_cast<float*>(take(S * H * 4));
  if (total) *total = off;
  return p;
}

}  // namespace

hipError_t launch_gemm_fp8(const void* a, const float* sa, const void* w, const float* sw, const int32_t* offsets,
                           int E, int M, int N, int K, int out_type, void* c, void* ws, hipStream_t stream) {
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.sa = sa;
  g.w = static_cast<const uint8_t*>(w);
  g.sw = sw;
  g.offsets = offsets;
  g.E = E;
  g.M = M;
  g.N = N;
  g.K = K;
  g.c = c;
  if (out_type == 0) return gemm<false, _Float16>(g, ws, stream);
  if (out_type == 1) return gemm<false, __bf16>(g, ws, stream);
  return gemm<true, float>(g, ws, stream);
}

size_t gemm_fp8_workspace_bytes(int M, int E, int N, int K) {
  if (M == 0 || E) return 0;
  const Cut how = cut_dense(M, N, K);
  return how.splits > 1 ? (size_t)how.splits * part_values(M, N) * sizeof(float) : 0;
}

size_t moe_fp8_workspace_bytes(int M, int top_k, int E, int H, int I) {
  size_t total = 0;
  carve(nullptr, M, top_k, E, H, I, &total);
  return total;
}

hipError_t launch_moe_fp8(const void* wg, const float* sg, const void* wu, const float* su, const void* wd,
                          const float* sd, int E, int H, int I, const void* x, int type, int M, const int32_t* ids,
                          const float* p, int top_k, void* y, void* ws, int32_t* dev_error, hipStream_t stream) {
  const ExpertsPlan pl = carve(ws, M, top_k, E, H, I, nullptr);
  const int S = M * top_k;
  hipError_t e = launch_moe_sort(ids, S, E, pl.offsets, pl.slot_row, pl.row_slot, pl.sort_ws, dev_error, stream);
  GemmArgs g{};
  g.a = pl.xq;
  g.sa = pl.xs;
  g.w = static_cast<const uint8_t*>(wg);
  g.sw = sg;
  g.w2 = static_cast<const uint8_t*>(wu);
  g.sw2 = su;
  g.offsets = pl.offsets;
  g.E = E;
  g.M = S;
  g.N = I;
  g.K = H;
  g.c = pl.hq;
  g.cs = pl.hs;
  if (e != hipSuccess) return e;
  // The gate and up products, by the mean rows of an expert (us of the whole call, bf16, experts
  // hit evenly, weights from HBM).  While no expert has more than 16 rows the weights stream past
  // tokens that are quantised on the way; then tiles of 64 rows while they hold any expert.
  //   64 experts, top-8, 2048 to 768: mean 13 82 with the stream, 91 with 64 rows, 100 with 128;
  //     20 103, 94 and 102; 44 102 with 64 rows, 111 with 128; 64 129 and 121
  //   16, top-2, 4096 to 1536: 13 84, 87 and 93; 20 116, 89 and 95; 44 98 and 102; 64 142 and 110
  //   128, top-8, 2048 to 512: 8 96, 101 and 108; 13 111, 106 and 112; 44 129 and 134; 64 157 and 151
  //   8, top-2, 4096 to 14336: 8 314, 314 and 334; 13 324, 316 and 337; 44 327 and 347; 64 425 and 389
  const int mean = S / E;
  if (mean <= 13) {
    StreamArgs s{};
    s.g = g;
    s.x = x;
    s.row_slot = pl.row_slot;
    s.top_k = top_k;
    s.tokens = M;
    s.ks = 1;
    e = type == 0 ? stream_gate_up<_Float16>(s, stream)
        : type == 1 ? stream_gate_up<__bf16>(s, stream)
                    : stream_gate_up<float>(s, stream);
  } else {
    e = launch_moe_gather_fp8(x, type, M, top_k, H, pl.slot_row, pl.xq, pl.xs, stream);
    if (e == hipSuccess)
      e = mean <= 43 ? run_tiles<TileKernel<64, 256, 1, 4, true, true, float>>(g, 64, 1, stream)
                     : run_tiles<TileKernel<128, 256, 2, 4, true, true, float>>(g, 128, 1, stream);
  }
  g.a = pl.hq;
  g.sa = pl.hs;
  g.w = static_cast<const uint8_t*>(wd);
  g.sw = sd;
  g.N = H;
  g.K = I;
  g.c = pl.ys;
  if (e != hipSuccess) return e;
  e = type == 1 ? grouped<false, float>(g, stream) : grouped<true, float>(g, stream);
  if (e == hipSuccess) e = launch_moe_combine_rows(pl.ys, type, M, top_k, H, pl.slot_row, p, y, stream);
  return e;
}

}  // namespace zinc
