// The tiled kernel of the block-scaled FP8 products (k_fp8_gemm.hip): one
// workgroup computes TM x TN outputs, its waves a WM x WN grid of them, on
// 16x16 MFMAs with w as the row operand and a as the column operand (a lane
// holds four neighbouring columns n of one row m).  An FP8 MFMA of 16x16x128 takes a
// whole block, so its sums are scaled and added without a second MFMA in
// between, three tiles behind the one that is issued.
//
// Per step of one block of 128 the two tiles, [TM x 128] and [TN x 128] bytes,
// are copied straight to LDS (16 bytes a lane, no registers in between) into
// one of two buffers while the waves multiply from the other; one barrier a
// step.  An LDS row is 128 bytes, its eight 16-byte pieces stored in the order
// piece ^ ((row >> 1) & 7), so that the lanes of a read, which run over rows,
// spread over all 64 banks (two rows fill them).  Which k a lane's piece holds is free as long as both
// operands agree: lane quarter q takes pieces q and q + 4.
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

// A lane's share (32 bytes) of 16 rows x 128 k, as the MFMAs take it.
template <bool EXACT>
struct Frag {
  i32x8_t v;
  __device__ __forceinline__ void set(const i32x4_t (&p)[2]) {
    v = __builtin_shufflevector(p[0], p[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <>
struct Frag<true> {
  half8_t v[4];
  __device__ __forceinline__ void set(const i32x4_t (&p)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = e4m3_to_f16(p[i][0], p[i][1]);
      v[2 * i + 1] = e4m3_to_f16(p[i][2], p[i][3]);
    }
  }
};

__device__ __forceinline__ f32x4_t mfma_block(const Frag<false>& a, const Frag<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4_t{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma_block(const Frag<true>& a, const Frag<true>& b) {
  f32x4_t d = {0, 0, 0, 0};
#pragma unroll
  for (int h = 0; h < 4; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[h], b.v[h], d, 0, 0, 0);
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
  static constexpr int MT = TM / WM / 16, NT = TN / WN / 16;
  static constexpr int LAG = 3;                     // tiles between an MFMA and the use of its sums
  static constexpr int COLS = DUAL ? TN / 2 : TN;   // output columns of a tile
  static constexpr int ROWS = TM + TN;              // LDS rows of a buffer
  static constexpr int PIECES = ROWS * 8 / THREADS; // 16-byte pieces a thread copies per step
  static constexpr int SB = TN / 128;               // w's scale blocks across the tile
  static_assert(TM % (8 * WAVES) == 0 && COLS % (8 * WAVES) == 0 && THREADS >= TM, "tile shape");
  static_assert(SB >= 1 && TN / WN <= 128 && WAVES % 2 == 0, "a wave's columns share one scale");
  static_assert(!DUAL || (NT == 4 && COLS == 128), "a quantised tile is one block wide");

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
    const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, quad = lane >> 4;
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
    auto copy_piece = [&](int i, int buf, int kb) {
      const int r = i * WAVES * 8;   // the instruction's first row, less the wave's
      const int in = r < TM ? r : (r - TM) % COLS;
      const auto rs = r < TM ? ra : r < TM + COLS ? rw1 : rw2;
      to_lds(rs, v0 + in * K + kb * 128, sm.tile[buf] + (i * WAVES + wave) * 1024);
    };
    auto cut_piece = [&](int i, int buf, int kb) {   // of the last block, cut short: zeros behind K
      const int r = i * WAVES * 8;
      const int in = r < TM ? r : (r - TM) % COLS;
      const auto rs = r < TM ? ra : r < TM + COLS ? rw1 : rw2;
      const bool is_in = kb * 128 + piece * 16 < K;
      const i32x4_t v = load_piece(rs, is_in ? v0 + in * K + kb * 128 : 0);
      *reinterpret_cast<i32x4_t*>(sm.tile[buf] + (i * WAVES + wave) * 1024 + lane * 16) =
          is_in ? v : i32x4_t{0, 0, 0, 0};
    };
    auto stage = [&](int buf, int kb) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if ((kb + 1) * 128 <= K)
          copy_piece(i, buf, kb);
        else
          cut_piece(i, buf, kb);
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

    f32x4_t acc[MT][NT] = {};
    // byte offsets of the lane's two pieces in an LDS row block
    int at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) at[j] = l16 * 128 + (((quad + 4 * j) ^ ((lane >> 1) & 7)) << 4);

    // Fragments in flight: w's of a step, read at the end of the step before; a's
    // one 16-row tile ahead, the last two together.
    i32x4_t wr[NT][2], ar[2][2];
    auto read_w = [&](int j, int buf) {
      const int row = TM + (DUAL ? wn * 32 + (j >> 1) * COLS + (j & 1) * 16 : wn * (TN / WN) + j * 16);
#pragma unroll
      for (int q = 0; q < 2; ++q) wr[j][q] = *reinterpret_cast<const i32x4_t*>(sm.tile[buf] + row * 128 + at[q]);
    };
    auto read_a = [&](int i, int slot, int buf) {
      const int row = wm * (TM / WM) + i * 16;
#pragma unroll
      for (int q = 0; q < 2; ++q) ar[slot][q] = *reinterpret_cast<const i32x4_t*>(sm.tile[buf] + row * 128 + at[q]);
    };
    // Tile t of a step is (i, j): all columns of one row tile after the other, but
    // the last two row tiles column by column, so that w's fragments fall free
    // for the next step's while there is work left.  A tile's block sums lie in
    // d[t % (LAG + 1)] and are scaled and added LAG tiles later, also across steps.
    constexpr int TILES = MT * NT, PAIR = (MT - 2) * NT;
    static_assert(MT >= 4 && TILES % (LAG + 1) == 0 && 2 * NT >= LAG && 2 * NT >= PIECES, "tile shape");
    f32x4_t d[LAG + 1] = {};
    float st[MT][DUAL ? 2 : 1] = {};
    auto row_of = [](int t) { return t < PAIR ? t / NT : MT - 2 + ((t - PAIR) & 1); };
    auto col_of = [](int t) { return t < PAIR ? t % NT : (t - PAIR) >> 1; };
    auto add = [&](int u) {
      const int i = row_of(u), j = col_of(u);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = fmaf(st[i][DUAL ? j >> 1 : 0], d[u % (LAG + 1)][r], acc[i][j][r]);
      asm volatile("" : "+v"(acc[i][j]));   // here, not behind the loop's branches
    };

    load_scales(0);
    put_scales(0);
    stage(0, 0);
    if (KB > 1) stage(1, 1);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < NT; ++j) read_w(j, 0);
    read_a(0, 0, 0);
    for (int kb = 0; kb < KB; ++kb) {
      const int buf = kb & 1;
      if ((kb & 3) == 0 && kb + 4 < KB) load_scales(kb + 4);
      const float* ts = sm.scale[(kb >> 2) & 1][DUAL ? 0 : wn * (TN / WN) / 128][kb & 3] + wm * (TM / WM) + l16;
      float sn[MT][DUAL ? 2 : 1];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < (DUAL ? 2 : 1); ++j) sn[i][j] = ts[j * 4 * TM + i * 16];
      const bool whole = (kb + 3) * 128 <= K;   // the block after the next one is not cut short
      Frag<EXACT> fw[NT], fa[2];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int i = row_of(t), j = col_of(t);
        if (t < PAIR && j == 0) {
          fa[0].set(ar[0]);
          if (i + 1 < MT - 2) {
            read_a(i + 1, 0, buf);
          } else {
            read_a(MT - 2, 0, buf);
            read_a(MT - 1, 1, buf);
          }
        }
        if (t < NT) fw[t].set(wr[t]);
        if (t == PAIR) {
          fa[0].set(ar[0]);
          fa[1].set(ar[1]);
          if ((kb & 3) == 2 && kb + 2 < KB) put_scales(kb + 2);
          // the next block has landed, and every wave has read what it needs of this one
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          if (!whole && kb + 2 < KB) stage(buf, kb + 2);
        }
        d[t % (LAG + 1)] = mfma_block(fw[j], fa[t < PAIR ? 0 : i - (MT - 2)]);
        if (t >= PAIR) {
          const int v = t - PAIR;
          if (v < PIECES && whole) copy_piece(v, buf, kb + 2);
          if (v & 1) read_w(j, buf ^ 1);
          if (t == TILES - 1) read_a(0, 0, buf ^ 1);
        }
        if (t < LAG) {
          add(TILES - LAG + t);
          if (t == LAG - 1) {
#pragma unroll
            for (int r = 0; r < MT; ++r)
#pragma unroll
              for (int b = 0; b < (DUAL ? 2 : 1); ++b) st[r][b] = sn[r][b];
          }
        } else {
          add(t - LAG);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int t = 0; t < LAG; ++t) add(TILES - LAG + t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

    if constexpr (!DUAL) {
      T* c = static_cast<T*>(g.c);
      const bool wide = N % 4 == 0;   // rows' outputs stay aligned to four
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 16 + l16;
        if (m >= rt.rows) continue;
        T* row = c + (size_t)(rt.first + m) * N;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int n = n0 + wn * (TN / WN) + j * 16 + 4 * quad;
          if (wide) {
            typedef T T4 __attribute__((ext_vector_type(4)));
            T4 o;
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = (T)acc[i][j][r];
            if (n < N) *reinterpret_cast<T4*>(row + n) = o;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < N) row[n + r] = (T)acc[i][j][r];
          }
        }
      }
    } else {
      // h = silu(gate) up; a row's maximum over the 128 columns: in the lane, over
      // the four lanes of the row, over the WN waves
      uint32_t* part = reinterpret_cast<uint32_t*>(&sm.tile[0][0]);   // [WN][TM]
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float z = acc[i][j][r];
            acc[i][j][r] = z / (1.0f + expf(-z)) * acc[i][2 + j][r];
            m = max(m, finite_abs_bits(acc[i][j][r]));
          }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (quad == 0) part[wn * TM + wm * (TM / WM) + i * 16 + l16] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 16 + l16;
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < WN; ++v) top = max(top, part[v * TM + m]);
        const uint32_t f = scale_field(top);
        if (m >= rt.rows) continue;
        uint8_t* row = static_cast<uint8_t*>(g.c) + (size_t)(rt.first + m) * N + n0 + wn * 32 + 4 * quad;
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = acc[i][r >> 2][r & 3];
        const uint2 o = to_e4m3(v, inverse_scale_of(f));
        *reinterpret_cast<uint32_t*>(row) = o.x;
        *reinterpret_cast<uint32_t*>(row + 16) = o.y;
        if (wn == 0 && quad == 0) g.cs[(size_t)(rt.first + m) * NB + nt] = scale_of(f);
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
