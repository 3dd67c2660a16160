// The weight-streaming kernel of the block-scaled FP8 products for few rows:
// up to 16 rows of a against 16 rows of w a wave.  The work is the one pass
// over w; everything else is arranged around keeping its loads in flight.
//
// - A wave copies its 16 rows x 128 k (2 KB) straight to its own LDS ring, DEPTH
//   steps ahead (two buffer loads of eight whole 128-byte lines a step), and
//   waits for them by count, so there is no barrier in the stream.
// - The rows of a lie in LDS for all waves, a chunk of k at a time: copied, or
//   quantised on the way from a token's row (the gather and the quantiser of an
//   expert layer, without launches of their own).
// - KS waves share 16 rows of w, taking every KS-th block of 128; their sums are
//   joined in LDS in a fixed order.
// - The products run on the fp16 MFMA (16x16x32) after exact conversion: the
//   matrix rate does not matter here, and its sums lose nothing.
//
// Bound by the stream, from HBM: one row of 11008 x 4096 12.5 us (3.6 TB/s; a large copy moves 5.2;
// 11.7 us where the last-level cache holds w), gate and up of 32 tokens, top-8 of 64 experts,
// 2048 -> 768, 44.6 us (4.5 TB/s).
#pragma once

#include "fp8_tile.hpp"

namespace zinc {

struct StreamArgs {
  GemmArgs g;               // g.a / g.sa: e4m3 rows and scales
  const void* x;            // DUAL in their place: rows of type T_IN, row r being x[row_slot[r] / top_k]
  const int32_t* row_slot;
  int top_k, tokens;
  int ks;                   // waves per 16 rows of w
  int chunk;                // blocks of 128 of a held in LDS, a multiple of ks
  int rows;                 // rows of a held in LDS
};

// DUAL: the experts' gate and up products of token rows, quantised on the way in, and
// silu(gate) up quantised on the way out; else a dense product.
template <int NW, int DEPTH, bool DUAL, typename T_IN, typename T>
struct StreamKernel {
  static constexpr int TM = 16, THREADS = 64 * NW;
  static constexpr int RING = DEPTH * 2048;   // bytes a wave
  static_assert(!DUAL || NW == 16, "a quantised output block is 16 waves of 8 columns");

  // LDS: the waves' rings (reused for joining the sums), a's rows, its scales
  // [chunk][rows], w's scales [NW][2][chunk]
  static size_t smem_bytes(int rows, int chunk) {
    return (size_t)NW * RING + (size_t)rows * chunk * 128 + (size_t)chunk * rows * 4 + (size_t)NW * 2 * chunk * 4;
  }

  static __device__ __forceinline__ void run(const StreamArgs& s, uint8_t* smem) {
    const GemmArgs& g = s.g;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int mt = (int)(blockIdx.x / (unsigned)g.col_tiles), nt = (int)(blockIdx.x - (unsigned)mt * g.col_tiles);
    const RowTile rt = find_tile<TM>(g.offsets, g.E, g.M, mt);
    if (rt.rows <= 0) return;
    const int K = g.K, N = g.N, KB = (K + 127) / 128, NB = (N + 127) / 128;
    const int ks = s.ks, slice = wave % ks, tile = wave / ks;
    // the wave's columns: 16 from n0, or 8 of gate's and the same 8 of up's (whose waves do
    // not share columns: ks is 1)
    const int n0 = DUAL ? nt * 128 + wave * 8 : (nt * (NW / ks) + tile) * 16;
    const int cols = max(0, min(DUAL ? 8 : 16, N - n0));   // 0: past the last column
    const size_t w_at = ((size_t)rt.expert * N + (cols ? n0 : 0)) * K;
    const Buffer rw1 = tile_buffer(g.w + w_at, cols * K);
    const Buffer rw2 = tile_buffer((DUAL ? g.w2 : g.w) + w_at, cols * K);
    uint8_t* ring = smem + wave * RING;
    uint8_t* ta = smem + NW * RING;
    float* tsa = reinterpret_cast<float*>(ta + (size_t)s.rows * s.chunk * 128);
    float* tsw = tsa + s.chunk * s.rows;

    const int steps = cols ? (KB - slice + ks - 1) / ks : 0;   // this wave's blocks: slice, slice + ks, ...
    const int piece = (lane & 7) ^ (lane >> 3);
    const int v0 = (lane >> 3) * K + piece * 16;
    auto issue = [&](int j) {   // past the last step: a load outside the bound, which moves nothing
      const int off = j < steps ? v0 + (slice + j * ks) * 128 : 0x7FFFFFF0;
      const int off2 = j < steps ? (DUAL ? off : off + 8 * K) : 0x7FFFFFF0;
      uint8_t* dst = ring + (j % DEPTH) * 2048;
      to_lds(rw1, off, dst);
      to_lds(rw2, off2, dst + 1024);
    };
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) issue(j);

    f32x4_t acc = {0, 0, 0, 0};
    int j = 0;
    for (int c0 = 0; c0 < KB; c0 += s.chunk) {
      const int nb = min(s.chunk, KB - c0);
      if (c0) __syncthreads();
      load_a(s, rt, c0, nb, ta, tsa);
      {   // w's scales of the chunk, two rows a wave
        const int blk = min(n0 >> 7, NB - 1);
        const size_t at = ((size_t)rt.expert * NB + blk) * KB + c0;
        for (int b = lane; b < nb; b += 64) {
          tsw[(wave * 2) * s.chunk + b] = g.sw[at + b];
          tsw[(wave * 2 + 1) * s.chunk + b] = DUAL ? g.sw2[at + b] : g.sw[at + b];
        }
      }
      __syncthreads();
      for (; j < steps && slice + j * ks < c0 + nb; ++j) {
        const int kb = slice + j * ks, b = kb - c0;
        // this step's two loads done: at most those of the later steps are outstanding
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (DEPTH - 1)) : "memory");
        const uint8_t* tw = ring + (j % DEPTH) * 2048 + l16 * 128;
        i32x4_t pw[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pw[h] = *reinterpret_cast<const i32x4_t*>(tw + (((quad + 4 * h) ^ (lane & 7)) << 4));
        asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(pw[0]), "+v"(pw[1])::"memory");
        issue(j + DEPTH);
        if ((kb + 1) * 128 > K) {   // the last block, cut short: zeros behind K
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (kb * 128 + (quad + 4 * h) * 16 >= K) pw[h] = i32x4_t{0, 0, 0, 0};
        }
        half8_t fw[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          fw[2 * h] = e4m3_to_f16(pw[h][0], pw[h][1]);
          fw[2 * h + 1] = e4m3_to_f16(pw[h][2], pw[h][3]);
        }
        // a lane holds columns 4 quad .. + 3 of the 16: up's from 8 on
        const float t = tsw[(wave * 2 + (quad >> 1)) * s.chunk + b];
        const int m = min(l16, s.rows - 1);
        const uint8_t* row = ta + ((size_t)b * s.rows + m) * 128;
        f32x4_t d = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const i32x4_t p = *reinterpret_cast<const i32x4_t*>(row + (((quad + 4 * h) ^ (m & 7)) << 4));
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[2 * h], e4m3_to_f16(p[0], p[1]), d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[2 * h + 1], e4m3_to_f16(p[2], p[3]), d, 0, 0, 0);
        }
        const float st = t * tsa[b * s.rows + m];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(st, d[r], acc[r]);
      }
    }

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load to the ring is left
    if constexpr (DUAL) {
      __syncthreads();
      uint32_t* part = reinterpret_cast<uint32_t*>(smem);   // [NW][TM]
      // quads 0 and 1 hold gate's columns, 2 and 3 up's of the same rows
      float h[8] = {};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float u = __shfl_xor(acc[r], 32, 64);
        h[r] = __any(acc[r] < kTail) ? silu_times<true>(acc[r], u) : silu_times(acc[r], u);
      }
      bool whole;
      uint32_t top = max_finite(h, whole);
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      if (quad == 0) part[wave * TM + l16] = top;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int v = 0; v < NW; ++v) top = max(top, part[v * TM + l16]);
      const uint32_t f = scale_field(top);
      if (l16 < rt.rows && quad < 2) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g.c) + (size_t)(rt.first + l16) * N + n0 + 4 * quad) =
            to_e4m3(h, inverse_scale_of(f), whole).x;
        if (wave == 0 && quad == 0) g.cs[(size_t)(rt.first + l16) * NB + nt] = scale_of(f);
      }
    } else {
      if (ks > 1) {
        __syncthreads();
        f32x4_t* part = reinterpret_cast<f32x4_t*>(smem);   // [NW][64]
        part[wave * 64 + lane] = acc;
        __syncthreads();
        if (slice) return;
        for (int v = 1; v < ks; ++v) acc += part[(wave + v) * 64 + lane];
      }
      if (l16 >= rt.rows) return;
      const int n = n0 + 4 * quad;
      T* row = static_cast<T*>(g.c) + (size_t)(rt.first + l16) * N;
      if (N % 4 == 0) {
        typedef T T4 __attribute__((ext_vector_type(4)));
        T4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = (T)acc[r];
        if (n < N) *reinterpret_cast<T4*>(row + n) = o;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < N) row[n + r] = (T)acc[r];
      }
    }
  }

  // Blocks c0 .. c0 + nb - 1 of the tile's rows of a to LDS: [block][row][128 bytes],
  // a row's pieces in the order piece ^ (row & 7); zeros behind K.
  static __device__ __forceinline__ void load_a(const StreamArgs& s, const RowTile& rt, int c0, int nb, uint8_t* ta,
                                                float* tsa) {
    const GemmArgs& g = s.g;
    const int K = g.K, KB = (K + 127) / 128;
    if constexpr (!DUAL) {
      for (int i = threadIdx.x; i < nb * rt.rows * 8; i += THREADS) {
        const int p = i & 7, b = (i >> 3) % nb, m = (i >> 3) / nb;
        const int k = (c0 + b) * 128 + p * 16;
        i32x4_t v = {0, 0, 0, 0};
        if (k < K) v = *reinterpret_cast<const i32x4_t*>(g.a + (size_t)(rt.first + m) * K + k);
        *reinterpret_cast<i32x4_t*>(ta + ((size_t)b * s.rows + m) * 128 + ((p ^ (m & 7)) << 4)) = v;
        if (p == 0) tsa[b * s.rows + m] = g.sa[(size_t)(rt.first + m) * KB + c0 + b];
      }
    } else {
      // sixteen lanes a block, eight values a lane
      const int l = threadIdx.x & 15;
      for (int i = threadIdx.x >> 4; i < nb * rt.rows; i += THREADS / 16) {
        const int b = i % nb, m = i / nb;
        const int slot = s.row_slot[rt.first + m];
        const int tok = min(max(slot, 0) / s.top_k, s.tokens - 1);
        const int k = (c0 + b) * 128 + l * 8;
        float v[8] = {};
        if (k < K) load8(static_cast<const T_IN*>(s.x) + (size_t)tok * K + k, v);
        bool whole;
        const uint32_t f = scale_field(max16(max_finite(v, whole)));
        const uint2 q = to_e4m3(v, inverse_scale_of(f), whole);
        *reinterpret_cast<uint2*>(ta + ((size_t)b * s.rows + m) * 128 + (((l >> 1) ^ (m & 7)) << 4) + (l & 1) * 8) = q;
        if (l == 0) tsa[b * s.rows + m] = scale_of(f);
      }
    }
  }
};

template <typename KERNEL>
__global__ __launch_bounds__(KERNEL::THREADS) void k_fp8_stream(StreamArgs s) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(s, smem);
}

}  // namespace zinc
