// The tiled kernel of the block-scaled FP8 products (k_fp8_gemm.hip): one
// workgroup computes TM x TN outputs, its waves a WM x WN grid of them, on
// 16x16 MFMAs with w as the row operand and a as the column operand (a lane
// holds four neighbouring columns n of one row m).  An FP8 MFMA of 16x16x128 takes a
// whole block, so its sums are scaled and added without a second MFMA in
// between, three tiles behind the one that is issued.
//
// Per step of one block of 128 the two tiles, [TM x 128] and [TN x 128] bytes,
// are copied straight to LDS (16 bytes a lane, no registers in between) into
// one of two or three buffers while the waves multiply from another; one barrier
// a step.  An LDS row is 128 bytes, its eight 16-byte pieces stored in the order
// piece ^ ((row >> 1) & 7) (w's: piece ^ w_turn(row)), so that the lanes of a read,
// which run over rows, spread over all 64 banks (two rows fill them).  Which k a
// lane's piece holds is free as long as both operands agree: lane quarter q takes
// pieces q and q + 4.
#pragma once

#include "fp8_device.hpp"
#include "silu.hpp"
#include "tiles.hpp"

namespace zinc {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
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
__device__ __forceinline__ void mfma_blocks(const Frag<true>& a0, const Frag<true>& b0, f32x4_t& d0,
                                            const Frag<true>& a1, const Frag<true>& b1, f32x4_t& d1) {
  d0 = d1 = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    d0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0.v[h], b0.v[h], d0, 0, 0, 0);
    d1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1.v[h], b1.v[h], d1, 0, 0, 0);
  }
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
  int row_tiles, col_tiles;   // an upper bound of the row tiles, where experts are grouped
  int splits;           // parts of K, each with its own output,
  size_t part;          // this many values after the one before
  void* c;
  float* cs;            // scales of a quantised output
};

// The same for the whole workgroup and not written by the kernel: scalar loads.
__device__ __forceinline__ const __attribute__((address_space(4))) float* uniform(const float* p) {
  return (const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

// DUAL: columns [0, TN / 2) of the tile are gate's rows, the others up's, and the
// output is silu(gate) up quantised to e4m3 (one block of 128 columns a tile).
//
// What bounds it, on random data: with FP8 MFMAs the power limit (8192 x 11008 x 4096
// 330 us, 2240 TFLOP/s at about 1.9 GHz, on one weight again and again, 379 us with weights that
// come from HBM; the MFMAs alone reach 3900 with their four FMAs).
// With fp16 MFMAs 1230 TFLOP/s for 8192^2 x 4096 (16-bit stores), the rate of a large bf16 library product
// (1210): they are busy 53 % of the cycles, and with fewer vector instructions, no
// copies' latency or other orders the time stays within 3 % while the clock moves against it.
//
// Workgroups are persistent: each walks its units (a tile, or a part of its K)
// and copies the next unit's first blocks while it finishes the one before, so a
// unit costs its steps and its stores.  Consecutive workgroup ids go to the
// eight XCDs in turn, so an XCD takes a contiguous run of the units; eight row
// tiles are walked per column, which keeps both operands' tiles in its L2.
template <int TM, int TN, int WM, int WN, bool EXACT, bool DUAL, typename T>
struct TileKernel {
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int MT = TM / WM / 16, NT = TN / WN / 16;
  // Tiles whose MFMAs are issued together (the fp16 MFMAs of a tile wait for one
  // another, so those of two take turns), and tiles between an MFMA and the use of
  // its sums, which lie in a ring.
  static constexpr int GROUP = EXACT ? 2 : 1, LAG = EXACT ? 2 : 3, RING = 4;
  static constexpr int COLS = DUAL ? TN / 2 : TN;   // output columns of a tile
  static constexpr int ROWS = TM + TN;              // LDS rows of a buffer
  static constexpr int PIECES = ROWS * 8 / THREADS; // 16-byte pieces a thread copies per step
  // 16-bit outputs are stored past the caches: 8192 x 11008 x 4096 328 us against 368, whose
  // stores push the operands' tiles out of L2.  fp32 ones may be parts of K or an
  // expert layer's rows, read again soon.
  static constexpr bool STREAMED = sizeof(T) == 2;
  // Buffers: with three, the copies of two blocks are in flight; where one workgroup fits a
  // CU either way.  Within 1.5 % of two for the experts, top-8 of 64 (256 tokens 103.8 us against 105,
  // 512 130 both, 4001 414 against 409); 32000 fp32 rows of 2048 x 768 148 - 151 against 148 - 158.
  // 256 x 256 has no room for a third, the small tiles fill LDS with more workgroups.
  static constexpr int NBUF = TN == 256 && TM <= 128 ? 3 : 2;
  static constexpr int BAND = 8;                    // row tiles walked per column
  // workgroups a CU holds by registers: three waves a SIMD where a wave has 32 sums, else two
  static constexpr int HELD = (MT * NT * 4 <= 32 ? 12 : 8) / WAVES;
  static_assert(TM % (8 * WAVES) == 0 && COLS % (8 * WAVES) == 0 && THREADS >= TM && TM % 64 == 0, "tile shape");
  static_assert(TN / WN <= 128 && TN / WN % 32 == 0 && WAVES % 4 == 0, "a wave's columns share one scale");
  static_assert(!DUAL || (NT == 4 && COLS == 128), "a quantised tile is one block wide");

  // How the pieces of w's LDS row are turned: rows are read as 8 q + r, q and r below 4.
  static __device__ __forceinline__ int w_turn(int row) { return ((row >> 1) & 1) + 2 * ((row >> 3) & 3); }

  struct Smem {
    uint8_t tile[NBUF][ROWS * 128];
    float sa[NBUF][TM];                      // a's scales of the buffer's block
    uint32_t part[DUAL ? WN * TM : 1];    // the waves' row maxima
  };
  // behind it, where experts are grouped: starts[E + 1], the experts' first rows,
  // and ends[E], the row tiles up to and with each
  static size_t smem_bytes(int experts) { return sizeof(Smem) + (experts ? 4 * (2 * (size_t)experts + 1) : 0); }

  struct Unit {
    int expert, first, rows;   // the tile's rows of a
    int nt, split, kb0, kbs;   // its column tile and blocks of K
  };

  static __device__ __forceinline__ Unit unit_at(const GemmArgs& g, const int32_t* starts, const int32_t* ends,
                                                 int row_tiles, int KB, long long u) {
    Unit r;
    const int per_row = g.col_tiles * g.splits;
    const int band = (int)(u / ((long long)BAND * per_row));
    const int in = (int)(u - (long long)band * BAND * per_row);
    const int size = min(BAND, row_tiles - band * BAND);
    const int col = in / size, mt = band * BAND + in - col * size;
    r.split = col / g.col_tiles;
    r.nt = col - r.split * g.col_tiles;
    const int each = (KB + g.splits - 1) / g.splits;
    r.kb0 = r.split * each;
    r.kbs = min(each, KB - r.kb0);
    if (!g.offsets) {
      r.expert = 0;
      r.first = mt * TM;
      r.rows = min(TM, g.M - r.first);
      return r;
    }
    tile_rows<TM>(g, starts, ends, mt, r);
    return r;
  }

  static __device__ __forceinline__ void run(const GemmArgs& g, Smem& sm) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, quad = lane >> 4;
    const int K = g.K, N = g.N, KB = (K + 127) / 128, NB = (N + 127) / 128;
    int32_t* starts = reinterpret_cast<int32_t*>(&sm + 1);
    int32_t* ends = starts + g.E + 1;
    int row_tiles = g.row_tiles;
    if (g.offsets) {
      row_tiles = make_tables<TM>(g, starts, ends);
      __syncthreads();
    }
    // this workgroup's units: u, u + stride, ... below last
    const long long total = (long long)row_tiles * g.col_tiles * g.splits, per = (total + 7) / 8;
    const int stride = gridDim.x / 8;
    const long long last = min(total, (long long)((blockIdx.x & 7) + 1) * per);
    long long u = (long long)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (u >= last) return;

    // Copies run ahead of the products: unit `ld`, its block `lk`, by buffer loads whose
    // bounds are the tile's parts of the matrices (rows behind the last are not
    // read; their products go nowhere).  Instruction i of a wave carries LDS rows
    // 8 (i WAVES + wave) .. + 7.
    const int a_piece = (lane & 7) ^ ((lane >> 4) + 4 * (wave & 1));
    const int w_piece = (lane & 7) ^ (((lane >> 4) & 1) + 2 * (wave & 3));
    const int v0 = (8 * wave + (lane >> 3)) * K;
    Unit ld = unit_at(g, starts, ends, row_tiles, KB, u);
    long long lu = u;
    int lk = 0;
    Buffer ra, rw1, rw2, rs;
    auto open = [&] {
      const int n0 = ld.nt * COLS, cols = min(COLS, N - n0);
      const size_t w_at = ((size_t)ld.expert * N + n0) * K;
      ra = tile_buffer(g.a + (size_t)ld.first * K, ld.rows * K);
      rw1 = tile_buffer(g.w + w_at, cols * K);
      rw2 = tile_buffer((DUAL ? g.w2 : g.w) + w_at, cols * K);
      rs = tile_buffer(reinterpret_cast<const uint8_t*>(g.sa + (size_t)ld.first * KB), ld.rows * KB * 4);
    };
    open();
    auto copy_piece = [&](int i, int buf) {
      const int r = i * WAVES * 8;   // the instruction's first row, less the wave's
      const int in = r < TM ? r : (r - TM) % COLS;
      to_lds(r < TM ? ra : r < TM + COLS ? rw1 : rw2,
             v0 + in * K + (ld.kb0 + lk) * 128 + 16 * (r < TM ? a_piece : w_piece),
             sm.tile[buf] + (i * WAVES + wave) * 1024);
    };
    auto copy_scales = [&](int buf) {
      if (wave * 64 < TM)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(sm.sa[buf] + wave * 64),
                                                 4, (tid * KB + ld.kb0 + lk) * 4, 0, 0, 0);
    };
    auto whole = [&] { return lu < last && (ld.kb0 + lk + 1) * 128 <= K; };
    auto copy_cut = [&](int buf) {   // the last block of K, cut short: zeros behind it
      if (DUAL || lu >= last) return;   // (gate's and up's K has whole blocks only)
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int r = i * WAVES * 8, kb = ld.kb0 + lk;
        const int in = r < TM ? r : (r - TM) % COLS, piece = r < TM ? a_piece : w_piece;
        const bool is_in = kb * 128 + piece * 16 < K;
        const i32x4_t v = load_piece(r < TM ? ra : r < TM + COLS ? rw1 : rw2,
                                     is_in ? v0 + in * K + kb * 128 + piece * 16 : 0);
        *reinterpret_cast<i32x4_t*>(sm.tile[buf] + (i * WAVES + wave) * 1024 + lane * 16) =
            is_in ? v : i32x4_t{0, 0, 0, 0};
      }
      copy_scales(buf);
    };
    auto advance = [&] {
      if (lu >= last || ++lk < ld.kbs) return;
      lk = 0;
      lu += stride;
      if (lu < last) {
        ld = unit_at(g, starts, ends, row_tiles, KB, lu);
        open();
      }
    };
    auto copy_all = [&](int buf) {
      if (whole()) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) copy_piece(i, buf);
        copy_scales(buf);
      } else {
        copy_cut(buf);
      }
      advance();
    };

    f32x4_t acc[MT][NT];
    // byte offsets of the lane's two pieces in an LDS row block
    // MFMA row 4 q + r of column tile j is column 32 (j / 2) + 8 q + 4 (j % 2) + r of
    // the wave's, so that a lane's sums of two column tiles are eight neighbours.
    int at[2], wat[2];
    const int wrow = 8 * (l16 >> 2) + (l16 & 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      at[j] = l16 * 128 + (((quad + 4 * j) ^ ((lane >> 1) & 7)) << 4);
      wat[j] = wrow * 128 + (((quad + 4 * j) ^ w_turn(wrow)) << 4);
    }
    // Fragments in flight: w's of a step, read at the end of the step before; a's
    // one 16-row tile ahead, the last two together.
    i32x4_t wr[NT][2], ar[2][2];
    auto read_w = [&](int j, int buf) {
      const int row = TM + (DUAL ? wn * 32 + (j >> 1) * COLS : wn * (TN / WN) + (j >> 1) * 32) + (j & 1) * 4;
#pragma unroll
      for (int q = 0; q < 2; ++q) wr[j][q] = *reinterpret_cast<const i32x4_t*>(sm.tile[buf] + row * 128 + wat[q]);
    };
    auto read_a = [&](int i, int slot, int buf) {
      const int row = wm * (TM / WM) + i * 16;
#pragma unroll
      for (int q = 0; q < 2; ++q) ar[slot][q] = *reinterpret_cast<const i32x4_t*>(sm.tile[buf] + row * 128 + at[q]);
    };
    // Tile t of a step is (i, j): all columns of one row tile after the other, but
    // the last two row tiles column by column, so that w's fragments fall free
    // for the next step's while there is work left.  A tile's block sums lie in
    // d[t % RING] and are scaled and added LAG tiles later, also across steps.
    constexpr int TILES = MT * NT, PAIR = (MT - 2) * NT;
    static_assert(MT >= 4 && TILES % RING == 0 && NT % 2 == 0 && 2 * NT >= LAG, "tile shape");
    constexpr int EACH = (PIECES + 2 * NT - 1) / (2 * NT);   // copies beside a tile of the last quarter
    f32x4_t d[RING];
    float st[MT][DUAL ? 2 : 1];
    auto row_of = [](int t) { return t < PAIR ? t / NT : MT - 2 + ((t - PAIR) & 1); };
    auto col_of = [](int t) { return t < PAIR ? t % NT : (t - PAIR) >> 1; };
    auto add = [&](int v) {
      const int i = row_of(v), j = col_of(v);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[i][j][r] = fmaf(st[i][DUAL ? j >> 1 : 0], d[v % RING][r], acc[i][j][r]);
      asm volatile("" : "+v"(acc[i][j]));   // here, not behind the loop's branches
    };

    copy_all(0);
    bool ahead = whole();   // the later blocks' copies may be in flight behind the first's
    copy_all(1);
    if constexpr (NBUF == 3) {
      ahead = ahead && whole();
      copy_all(2);
    }
    if (ahead)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 1) * PIECES) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < NT; ++j) read_w(j, 0);
    read_a(0, 0, 0);
    int buf = 0;
    auto after = [](int b) { return NBUF == 2 ? b ^ 1 : b == NBUF - 1 ? 0 : b + 1; };
    for (; u < last; u += stride) {
      const Unit cu = unit_at(g, starts, ends, row_tiles, KB, u);
      const int n0 = cu.nt * COLS;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < RING; ++i) d[i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int b = 0; b < (DUAL ? 2 : 1); ++b) st[i][b] = 0.0f;
      // w's scales: one a wave and step (two with gate and up)
      const size_t sw_at =
          ((size_t)cu.expert * NB + (DUAL ? cu.nt : min((n0 + wn * (TN / WN)) >> 7, NB - 1))) * KB + cu.kb0;
      const auto sw1 = uniform(g.sw + sw_at), sw2 = uniform((DUAL ? g.sw2 : g.sw) + sw_at);
      for (int kb = 0; kb < cu.kbs; ++kb, buf = after(buf)) {
        const float t1 = sw1[kb], t2 = DUAL ? sw2[kb] : 0.0f;
        float sn[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) sn[i] = sm.sa[buf][wm * (TM / WM) + i * 16 + l16];
        const bool fast = whole();
        const int next = after(buf);
        Frag<EXACT> fw[NT], fa[2];
#pragma unroll
        for (int t0 = 0; t0 < TILES; t0 += GROUP) {
#pragma unroll
          for (int t = t0; t < t0 + GROUP; ++t) {
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
              // the next block has landed, and every wave has read what it needs of this one
              if (NBUF == 3 && ahead)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PIECES) : "memory");
              else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
              __builtin_amdgcn_s_barrier();
              asm volatile("" ::: "memory");
              if (!fast) copy_cut(buf);
            }
          }
          auto a_of = [&](int t) -> const Frag<EXACT>& { return fa[t < PAIR ? 0 : row_of(t) - (MT - 2)]; };
          if constexpr (EXACT)
            mfma_blocks(fw[col_of(t0)], a_of(t0), d[t0 % RING], fw[col_of(t0 + 1)], a_of(t0 + 1), d[(t0 + 1) % RING]);
          else
            d[t0 % RING] = mfma_block(fw[col_of(t0)], a_of(t0));
#pragma unroll
          for (int t = t0; t < t0 + GROUP; ++t) {
            if (t >= PAIR) {
              const int v = t - PAIR;
              if (fast) {
#pragma unroll
                for (int c = v * EACH; c < (v + 1) * EACH; ++c)
                  if (c < PIECES) copy_piece(c, buf);
                if (t == TILES - 1) copy_scales(buf);
              }
              if (v & 1) read_w(col_of(t), next);
              if (t == TILES - 1) read_a(0, 0, next);
            }
            if (t < LAG) {
              add(TILES - LAG + t);
              if (t == LAG - 1) {
#pragma unroll
                for (int r = 0; r < MT; ++r) {
                  st[r][0] = sn[r] * t1;
                  if (DUAL) st[r][DUAL ? 1 : 0] = sn[r] * t2;
                }
              }
            } else {
              add(t - LAG);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        advance();
        ahead = fast;
      }
#pragma unroll
      for (int t = 0; t < LAG; ++t) add(TILES - LAG + t);
      store(g, sm, cu, n0, N, NB, wm, wn, l16, quad, acc);
    }
  }

  static __device__ __forceinline__ void store(const GemmArgs& g, Smem& sm, const Unit& cu, int n0, int N, int NB,
                                               int wm, int wn, int l16, int quad, f32x4_t (&acc)[MT][NT]) {
    if constexpr (!DUAL) {
      T* c = static_cast<T*>(g.c) + (size_t)cu.split * g.part;
      const bool wide = N % 8 == 0;   // rows' outputs stay aligned to eight
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 16 + l16;
        if (m >= cu.rows) continue;
        T* row = c + (size_t)(cu.first + m) * N;
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          const int n = n0 + wn * (TN / WN) + j * 16 + 8 * quad;
          float v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = acc[i][j + (r >> 2)][r & 3];
          if (wide) {
            if (n < N) store8<STREAMED>(row + n, v);
          } else {
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (n + r < N) row[n + r] = (T)v[r];
          }
        }
      }
    } else {
      // h = silu(gate) up; a row's maximum over the 128 columns: in the lane, over
      // the four lanes of the row, over the WN waves
      uint32_t* part = sm.part;
      float h[MT][8], low = 0.0f;
      bool whole[MT];
      auto z = [&](int i, int r) { return acc[i][r >> 2][r & 3]; };
      auto u = [&](int i, int r) { return acc[i][2 + (r >> 2)][r & 3]; };
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          h[i][r] = silu_times(z(i, r), u(i, r));
          low = fminf(low, z(i, r));
        }
      if (__any(low < kTail)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 8; ++r) h[i][r] = silu_times<true>(z(i, r), u(i, r));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t m = max_finite(h[i], whole[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (quad == 0) part[wn * TM + wm * (TM / WM) + i * 16 + l16] = m;
      }
      // (written again a unit later, behind the barriers of its steps)
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = wm * (TM / WM) + i * 16 + l16;
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < WN; ++v) top = max(top, part[v * TM + m]);
        const uint32_t f = scale_field(top);
        if (m >= cu.rows) continue;
        uint8_t* row = static_cast<uint8_t*>(g.c) + (size_t)(cu.first + m) * N + n0 + wn * 32 + 8 * quad;
        *reinterpret_cast<uint2*>(row) = to_e4m3(h[i], inverse_scale_of(f), whole[i]);
        if (wn == 0 && quad == 0) g.cs[(size_t)(cu.first + m) * NB + cu.nt] = scale_of(f);
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
