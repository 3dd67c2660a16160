// The tiled kernel of the block-scaled FP8 products (k_fp8_gemm.hip): one
// workgroup computes TM x TN outputs, its waves a WM x WN grid of them, on
// 32x32 MFMAs with w as the row operand and a as the column operand (a lane
// holds 16 columns n of one row m).
//
// Per step of one block of 128 the two tiles, [TM x 128] and [TN x 128] bytes,
// are copied straight to LDS (16 bytes a lane, no registers in between) into
// one of two buffers while the waves multiply from the other; one barrier a
// step.  An LDS row is 128 bytes, its eight 16-byte pieces stored in the order
// piece ^ ((row >> 1) & 7), so that the lanes of a read, which run over rows,
// spread over all 64 banks (two rows fill them).  Which k a lane's piece holds is free as long as both
// operands agree: lane half h takes pieces h, h + 2, h + 4, h + 6.
#pragma once

#include "fp8_device.hpp"

namespace zinc {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

// Eight e4m3 bytes as fp16, exactly.
__device__ __forceinline__ half8_t e4m3_to_f16(int lo, int hi) {
  const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's share (64 bytes) of 32 rows x 128 k, as the MFMAs take it.
template <bool EXACT>
struct Frag {
  i32x8_t v[2];
  __device__ __forceinline__ void set(const i32x4_t (&p)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = __builtin_shufflevector(p[2 * h], p[2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Frag<true> {
  half8_t v[8];
  __device__ __forceinline__ void set(const i32x4_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = e4m3_to_f16(p[i][0], p[i][1]);
      v[2 * i + 1] = e4m3_to_f16(p[i][2], p[i][3]);
    }
  }
};

__device__ __forceinline__ f32x16_t mfma_block(const Frag<false>& a, const Frag<false>& b) {
  f32x16_t d = {};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v[h], b.v[h], d, 0, 0, 0, 0, 0, 0);
  return d;
}
__device__ __forceinline__ f32x16_t mfma_block(const Frag<true>& a, const Frag<true>& b) {
  f32x16_t d = {};
#pragma unroll
  for (int h = 0; h < 8; ++h) d = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.v[h], b.v[h], d, 0, 0, 0);
  return d;
}

// The rows [first, first + rows) of tile `tile` (TM rows each) of the experts'
// row ranges, and its expert; rows <= 0 past the last tile.  Offsets outside
// [0, total] or not ascending are cut to that range.
struct RowTile {
  int expert, first, rows;
};

template <int TM>
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ offsets, int E, int total, int tile) {
  if (!offsets) return {0, tile * TM, min(TM, total - tile * TM)};
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = e < E ? min(max(offsets[e], 0), total) : 0;
    const int hi = e < E ? min(max(offsets[e + 1], lo), total) : 0;
    const int n = (hi - lo + TM - 1) / TM;
    int scan = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(scan, d, 64);
      if (lane >= d) scan += o;
    }
    const uint64_t here = __ballot(seen + scan > tile);
    if (here) {
      const int l = (int)__builtin_ctzll(here);
      const int before = seen + __builtin_amdgcn_readlane(scan - n, l);
      const int first = __builtin_amdgcn_readlane(lo, l) + (tile - before) * TM;
      return {e0 + l, first, min(TM, __builtin_amdgcn_readlane(hi, l) - first)};
    }
    seen += __builtin_amdgcn_readlane(scan, 63);
  }
  return {0, 0, 0};
}

// Row tiles a grouped product can have: every expert's last one may be partly filled.
inline long long max_row_tiles(long long rows, int experts, int TM) {
  return experts ? (rows + TM - 1) / TM + (experts < rows ? experts : rows) : (rows + TM - 1) / TM;
}

struct GemmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;     // gate's, where two weights are multiplied
  const float* sw;
  const uint8_t* w2;    // up's
  const float* sw2;
  const int32_t* offsets;
  int E, M, N, K;
  int row_tiles, col_tiles;
  void* c;
  float* cs;            // scales of a quantised output
};

// Order of the workgroups: consecutive ids go to the eight XCDs in turn, so each
// XCD takes a contiguous run of tiles; within it eight row tiles are walked per
// column, which keeps both operands' tiles in its L2.
__device__ __forceinline__ bool tile_of_block(const GemmArgs& g, int& mt, int& nt) {
  constexpr int kBand = 8;
  const long long total = (long long)g.row_tiles * g.col_tiles, per = (total + 7) / 8;
  const long long t = (long long)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || t >= total) return false;
  const long long band = t / ((long long)kBand * g.col_tiles);
  const int in = (int)(t - band * kBand * g.col_tiles);
  const int size = min(kBand, g.row_tiles - (int)band * kBand);
  nt = in / size;
  mt = (int)band * kBand + in - nt * size;
  return true;
}

// Buffer loads bounded by a matrix's `bytes` from p: bytes behind them read as zero
// and touch no memory.
using Buffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buffer tile_buffer(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00020000);
}
// Sixteen bytes a lane to LDS, lane after lane from dst.
__device__ __forceinline__ void to_lds(Buffer b, int off, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ i32x4_t load_piece(Buffer b, int off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
}

// The same for the whole workgroup and not written by the kernel: scalar loads.
__device__ __forceinline__ const __attribute__((address_space(4))) float* uniform(const float* p) {
  return (const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

// DUAL: columns [0, TN / 2) of the tile are gate's rows, the others up's, and the
// output is silu(gate) up quantised to e4m3 (one block of 128 columns a tile).
template <int TM, int TN, int WM, int WN, bool EXACT, bool DUAL, typename T>
struct TileKernel {
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int MT = TM / WM / 32, NT = TN / WN / 32;
  static constexpr int COLS = DUAL ? TN / 2 : TN;   // output columns of a tile
  static constexpr int ROWS = TM + TN;              // LDS rows of a buffer
  static constexpr int PIECES = ROWS * 8 / THREADS; // 16-byte pieces a thread copies per step
  static constexpr int SB = TN / 128;               // w's scale blocks across the tile
  static_assert(TM % (8 * WAVES) == 0 && COLS % (8 * WAVES) == 0 && THREADS >= TM, "tile shape");
  static_assert(SB >= 1 && TN / WN <= 128 && WAVES % 2 == 0, "a wave's columns share one scale");
  static_assert(!DUAL || (NT == 2 && COLS == 128), "a quantised tile is one block wide");

  struct Smem {
    uint8_t tile[2][ROWS * 128];
    float scale[2][SB][4][TM];   // a's times w's, of four steps, two of them
  };

  static __device__ __forceinline__ void run(const GemmArgs& g, Smem& sm) {
    int mt, nt;
    if (!tile_of_block(g, mt, nt)) return;
    const RowTile rt = find_tile<TM>(g.offsets, g.E, g.M, mt);
    if (rt.rows <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, half = lane >> 5;
    const int K = g.K, N = g.N, KB = (K + 127) / 128, NB = (N + 127) / 128;
    const int n0 = nt * COLS;
    // Copy plan: instruction i of a wave carries LDS rows 8 (i WAVES + wave) .. + 7,
    // by buffer loads whose bound is the tile's part of the matrix: rows behind
    // its last are not read (their products go nowhere).
    const int piece = (lane & 7) ^ ((lane >> 4) + 4 * (wave & 1));
    const int row0 = 8 * wave + (lane >> 3);
    const uint8_t* a = g.a + (size_t)rt.first * K;
    const size_t w_at = ((size_t)rt.expert * N + n0) * K;
    const int cols = min(COLS, N - n0);
    const auto ra = tile_buffer(a, rt.rows * K);
    const auto rw1 = tile_buffer(g.w + w_at, cols * K);
    const auto rw2 = tile_buffer((DUAL ? g.w2 : g.w) + w_at, cols * K);
    const int v0 = row0 * K + piece * 16;
    auto stage = [&](int buf, int kb) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int r = i * WAVES * 8;   // the instruction's first row, less the wave's
        const int in = r < TM ? r : (r - TM) % COLS;
        const auto rs = r < TM ? ra : r < TM + COLS ? rw1 : rw2;
        uint8_t* dst = sm.tile[buf] + (i * WAVES + wave) * 1024;
        const int off = v0 + in * K + kb * 128;
        if ((kb + 1) * 128 <= K) {
          to_lds(rs, off, dst);
        } else {   // the last block, cut short: zeros behind K
          const bool is_in = kb * 128 + piece * 16 < K;
          const i32x4_t v = load_piece(rs, is_in ? off : 0);
          *reinterpret_cast<i32x4_t*>(dst + lane * 16) = is_in ? v : i32x4_t{0, 0, 0, 0};
        }
      }
    };
    // scales of four steps at a time, a's times w's: one thread a row.  a's are
    // loaded two steps before they are put, w's are scalar loads.
    const float* sa_row = g.sa + (size_t)(rt.first + min(tid, rt.rows - 1)) * KB;
    float s4[4];
    auto load_scales = [&](int kb) {
      if (tid < TM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s4[i] = sa_row[min(kb + i, KB - 1)];
      }
    };
    auto put_scales = [&](int kb) {
#pragma unroll
      for (int b = 0; b < SB; ++b) {
        const int blk = DUAL ? nt : min((n0 >> 7) + b, NB - 1);
        const auto sw = uniform((DUAL && b ? g.sw2 : g.sw) + ((size_t)rt.expert * NB + blk) * KB);
        float t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = sw[min(kb + i, KB - 1)];
        if (tid < TM) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sm.scale[(kb >> 2) & 1][b][i][tid] = s4[i] * t[i];
        }
      }
    };

    f32x16_t acc[MT][NT] = {};
    // byte offsets of the lane's four pieces in an LDS row block
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = l32 * 128 + (((half + 2 * j) ^ ((lane >> 1) & 7)) << 4);

    load_scales(0);
    put_scales(0);
    stage(0, 0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    for (int kb = 0; kb < KB; ++kb) {
      const int buf = kb & 1;
      if ((kb & 3) == 0 && kb + 4 < KB) load_scales(kb + 4);
      if (kb + 1 < KB) stage(buf ^ 1, kb + 1);
      const uint8_t* ta = sm.tile[buf] + wm * (TM / WM) * 128;
      const uint8_t* tw = sm.tile[buf] + TM * 128 + (DUAL ? wn * 32 : wn * (TN / WN)) * 128;
      const float* ts = sm.scale[(kb >> 2) & 1][DUAL ? 0 : wn * (TN / WN) / 128][kb & 3] + wm * (TM / WM) + l32;
      Frag<EXACT> fw[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        i32x4_t p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[q] = *reinterpret_cast<const i32x4_t*>(tw + (DUAL ? j * COLS : j * 32) * 128 + at[q]);
        fw[j].set(p);
      }
      // A step's MFMAs run while the previous step's block sums are scaled and
      // added: tile t = (i, j), its sums in d[t & 1].
      i32x4_t p[4];
      auto read_a = [&](int i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) p[q] = *reinterpret_cast<const i32x4_t*>(ta + i * 32 * 128 + at[q]);
      };
      Frag<EXACT> fa;
      f32x16_t d[2];
      float st[MT][DUAL ? NT : 1];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < (DUAL ? NT : 1); ++j) st[i][j] = ts[j * 4 * TM + i * 32];
      read_a(0);
#pragma unroll
      for (int t = 0; t <= MT * NT; ++t) {
        const int i = t / NT, j = t % NT;
        if (t < MT * NT) {
          if (j == 0) {
            fa.set(p);
            if (i + 1 < MT) read_a(i + 1);
          }
          d[t & 1] = mfma_block(fw[j], fa);
        }
        if (t > 0) {
          const int u = t - 1;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            acc[u / NT][u % NT][r] = fmaf(st[u / NT][DUAL ? u % NT : 0], d[u & 1][r], acc[u / NT][u % NT][r]);
          asm volatile("" : "+v"(acc[u / NT][u % NT]));   // here, not behind the loop's branches
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if ((kb & 3) == 2 && kb + 2 < KB) put_scales(kb + 2);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }

    if constexpr (!DUAL) {
      T* c = static_cast<T*>(g.c);
      const bool wide = N % 4 == 0;   // rows' outputs stay aligned to four
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 32 + l32;
        if (m >= rt.rows) continue;
        T* row = c + (size_t)(rt.first + m) * N;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int n = n0 + wn * (TN / WN) + j * 32 + 8 * q + 4 * half;
            if (wide) {
              typedef T T4 __attribute__((ext_vector_type(4)));
              T4 o;
#pragma unroll
              for (int r = 0; r < 4; ++r) o[r] = (T)acc[i][j][4 * q + r];
              if (n < N) *reinterpret_cast<T4*>(row + n) = o;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (n + r < N) row[n + r] = (T)acc[i][j][4 * q + r];
            }
          }
      }
    } else {
      // h = silu(gate) up; a row's maximum over the 128 columns: in the lane, over
      // the two lanes of the row, over the WN waves
      uint32_t* part = reinterpret_cast<uint32_t*>(&sm.tile[0][0]);   // [WN][TM]
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float z = acc[i][0][r];
          acc[i][0][r] = z / (1.0f + expf(-z)) * acc[i][1][r];
          m = max(m, finite_abs_bits(acc[i][0][r]));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (half == 0) part[wn * TM + wm * (TM / WM) + i * 32 + l32] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 32 + l32;
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < WN; ++v) top = max(top, part[v * TM + m]);
        const uint32_t f = scale_field(top);
        if (m >= rt.rows) continue;
        uint8_t* row = static_cast<uint8_t*>(g.c) + (size_t)(rt.first + m) * N + n0 + wn * 32 + 4 * half;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = acc[i][0][8 * q + r];
          const uint2 o = to_e4m3(v, inverse_scale_of(f));
          *reinterpret_cast<uint32_t*>(row + 16 * q) = o.x;
          *reinterpret_cast<uint32_t*>(row + 16 * q + 8) = o.y;
        }
        if (wn == 0 && half == 0) g.cs[(size_t)(rt.first + m) * NB + nt] = scale_of(f);
      }
    }
  }
};

template <typename KERNEL>
__global__ __launch_bounds__(KERNEL::THREADS) void k_fp8_tile(GemmArgs g) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(g, *reinterpret_cast<typename KERNEL::Smem*>(smem));
}

}  // namespace zinc
