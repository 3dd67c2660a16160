// The tiled kernel of the 16-bit products by expert (k_gemm16_*.hip), all three of a training step:
//   forward  c[r][n]      = sum_k a[r][k]  w[e][n][k]      the rows r of expert e
//   input    da[r][k]     = sum_n dc[r][n] w[e][n][k]
//   weight   dw[e][n][k]  = sum_r dc[r][n] a[r][k]
// One workgroup computes TM x TN outputs, its waves a WM x WN grid of them, on 16x16x32 MFMAs.  P is the
// operand of the output's rows, Q that of its columns; Q is the MFMA's row operand, so that a lane holds
// neighbouring columns of one output row.
//
// Per step of 64 along the summed dimension both tiles are copied straight to LDS (16 bytes a lane, no
// registers in between) into one of two or three buffers while the waves multiply from another; one
// barrier a step.  An operand whose summed dimension is contiguous lies in LDS as [rows][64], one whose
// rows are summed over as [64][columns], read by transposing loads (ds_read_b64_tr_b16: lanes 4 i .. 4 i + 3
// of 16 name row i's 16 values, lane 4 c + t gets value t of piece c from each of the four rows).  The 16-byte pieces
// of a row are turned by the row's number, so that the lanes of a read spread over the banks.
#pragma once

#include "fp8_device.hpp"
#include "gemm16_plan.hpp"
#include "tiles.hpp"

namespace zinc {

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4_t mfma16(i16x8_t a, i16x8_t b, f32x4_t c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(i16x8_t a, i16x8_t b, f32x4_t c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8_t, a), __builtin_bit_cast(bhalf8_t, b), c,
                                                 0, 0, 0);
}

__device__ __forceinline__ i16x4_t read_turned(const uint8_t* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)lds);
}

// Rows in whole 128-byte lines.  As an MFMA operand lane l of 16 holds row l's pieces q and q + 4 (16 bytes
// each, q its quarter of the wave); a load of piece q + 4 (l / 8) of row l % 8, and one of row 8 + l % 8, take
// two such quarters of 8 rows each, which is 128 bytes a row.  The lower lanes' second load and the upper
// lanes' first then change places; to store, the same again.  (8192 x 11008 values read and written by 64-byte
// pieces 95 us, by 128 75, by 256 and 1024 74.)
__device__ __forceinline__ void trade_lines(i32x4_t& first, i32x4_t& second) {
  const bool low = (threadIdx.x & 8) == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = first[i], y = second[i], give = low ? y : x;
    const int get = __builtin_amdgcn_update_dpp(give, give, 0x128, 0xF, 0xF, false);   // row_ror:8
    first[i] = low ? x : get;
    second[i] = low ? get : y;
  }
}

struct Gemm16Args {
  const void* p;    // a, or dc
  const void* q;    // w, or a
  const int32_t* offsets;
  int E, M, N, K;   // experts, rows, w's rows and columns
  void* c;
  int splits;       // parts of the summed dimension, each with its own output,
  size_t part;      // this many values after the one before
  int32_t* queue;   // the next unit of each XCD, 32 apart, from blocks / 8 on; or null: dealt out in turn
};

template <Product F, int TM, int TN, int WM, int WN, int BUFFERS, typename T, typename O>
struct Gemm16 {
  static constexpr Product kProduct = F;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int MT = TM / WM / 16, NT = TN / WN / 16;
  static constexpr bool P_T = F == kWeight, Q_T = F != kForward;   // summed over rows of the matrix
  // Columns of two neighbouring 16-wide tiles taken in turns of four, so that a lane's sums are eight
  // neighbours.  The transposing reads would meet two to a bank so; their lanes hold two times four, and trade them
  // where 16-bit outputs are stored.
  static constexpr bool WIDE = !Q_T;
  static constexpr int PI = TM / 8 / WAVES, QI = TN / 8 / WAVES, COPIES = PI + QI;   // copies a wave, a step
  static constexpr int BUFFER = (TM + TN) * 128;
  static constexpr int NBUF = BUFFERS;
  // The smallest tile's waves hold a step's fragments in full, so its buffer is free, and the next step's reads and
  // copies on their way, from the step's start; a CU that holds one workgroup otherwise waits for each read (2331
  // rows of 7 x 520 x 1032: 16.3 us, so 16.1, and 12.6 with the three buffers that the forward product takes).  Over
  // 90 products the best of all cuts takes 4 % less so; three buffers, and two workgroups a CU instead of three, cost
  // dw 2 %, da gains 1 % with two or three.
  static constexpr bool EAGER = NT == 2;
  static constexpr int BAND = 8;   // row tiles walked per column
  // Large tiles' outputs are stored past the caches, in whole lines (in half lines memory writes half as much
  // again): 32768 rows of 64 experts, 768 x 2048, from queues, by trace, on the same operands again and again dw in fp32
  // 146 us, in lines that the caches hold 186, da 122 and 128; on operands from HBM dw 174 and 181, da 140 and 141.
  static constexpr bool STREAMED = NT == 4;
  // workgroups a CU holds by registers
  static constexpr int HELD = (MT * NT * 4 <= 32 ? 12 : 8) / WAVES;
  static_assert(TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0 && WAVES % 4 == 0, "whole copies");
  static_assert(MT >= 4 && (NT == 2 || NT == 4), "tile shape");
  static_assert((!P_T || WAVES * (512 / TM) % 16 == 0) && (!Q_T || WAVES * (512 / TN) % 16 == 0),
                "a lane's turn is the same in all of its copies");

  // LDS: the buffers, the numbers of the units in hand, and tables: starts[E + 1], the experts' first rows,
  // and ends[E], the row tiles up to and with each; kWeight: rows[E] and the experts in the order of their units
  static size_t smem_bytes(int E) { return NBUF * BUFFER + 16 + 4 * (2 * (size_t)E + 1); }

  struct Unit {
    int expert, first, rows;   // rows of the matrix: the tile's, or the expert's (kWeight)
    int p0, q0, steps;        // first output row (kWeight) and column
    int split, k0;            // its part of the summed dimension, from this step (row, kWeight) on
  };

  // How a row's pieces are turned.  [rows][64] of P: two rows fill the banks; of Q, whose rows are read as
  // 8 q + r with q and r below 4, likewise.  [64][columns]: the eight rows of half a wave's read.
  static __device__ __forceinline__ int p_turn(int row) { return (row >> 1) & 7; }
  static __device__ __forceinline__ int q_turn(int row) { return ((row >> 1) & 1) + 2 * ((row >> 3) & 3); }
  template <int W>
  static __device__ __forceinline__ int t_turn(int row) {
    return W >= 128 ? 2 * ((row & 3) + 4 * ((row >> 3) & 1)) : 2 * (((row >> 1) & 1) + 2 * ((row >> 3) & 1));
  }

  static __device__ __forceinline__ Unit unit_at(const Gemm16Args& g, const int32_t* starts, const int32_t* ends,
                                                 int row_tiles, int col_tiles, int u) {
    Unit r;
    if constexpr (F == kWeight) {
      const int row_t = (g.N + TM - 1) / TM, each = row_t * col_tiles, at = u / (each * g.splits);
      const int inside = u - at * each * g.splits, in = inside % each;
      r.split = inside / each;
      r.expert = __builtin_amdgcn_readfirstlane(ends[at]);
      const int band = in / (BAND * col_tiles), k = in - band * BAND * col_tiles;
      const int size = min(BAND, row_t - band * BAND), col = k / size;
      r.p0 = (band * BAND + k - col * size) * TM;
      r.q0 = col * TN;
      const int lo = min(max(g.offsets[r.expert], 0), g.M), hi = min(max(g.offsets[r.expert + 1], lo), g.M);
      const int part = ((hi - lo + g.splits - 1) / g.splits + 63) / 64 * 64;
      r.k0 = min(r.split * part, hi - lo);
      r.first = __builtin_amdgcn_readfirstlane(lo + r.k0);
      r.rows = __builtin_amdgcn_readfirstlane(min(part, hi - lo - r.k0));
      r.steps = max(NBUF + 1, (r.rows + 63) / 64);   // steps behind the last row: zeros
    } else {
      const int per_row = col_tiles * g.splits, band = u / (BAND * per_row), in = u - band * BAND * per_row;
      const int size = min(BAND, row_tiles - band * BAND), column = in / size;
      r.split = column / col_tiles;
      const int col = column - r.split * col_tiles;
      tile_rows<TM>(g, starts, ends, band * BAND + in - column * size, r);
      r.p0 = 0;
      r.q0 = col * TN;
      const int all = ((F == kForward ? g.K : g.N) + 63) / 64, each = (all + g.splits - 1) / g.splits;
      r.k0 = r.split * each;
      r.steps = max(NBUF + 1, min(each, all - r.k0));
    }
    return r;
  }

  // The experts with most rows first, dealt out to the XCDs' queues (each a contiguous run of the order)
  // back and forth: 0 .. 7, 7 .. 0, ...; fewer than eight keep their order.  Those without rows stand behind them.
  // Returns how many have rows.
  static __device__ __forceinline__ int order_experts(const Gemm16Args& g, int32_t* rows, int32_t* order) {
    for (int e = threadIdx.x; e < g.E; e += THREADS) {
      const int lo = min(max(g.offsets[e], 0), g.M);
      rows[e] = max(min(g.offsets[e + 1], g.M) - lo, 0);
    }
    __syncthreads();
    int reached = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
      const int e = e0 + (threadIdx.x & 63);
      reached += __popcll(__ballot(e < g.E && rows[e] > 0));
    }
    const int whole = reached / 8, rest = reached % 8;
    for (int e = threadIdx.x; e < g.E; e += THREADS) {
      const int mine = rows[e];
      int rank = 0;
      for (int o = 0; o < g.E; ++o) rank += rows[o] > mine || (rows[o] == mine && o < e);
      int at = rank;
      if (whole && rank < reached) {
        const int turn = rank / 8;
        auto xcd_of = [](int turn, int in) { return turn & 1 ? 7 - in : in; };
        const int xcd = xcd_of(turn, rank % 8);
        at = xcd * whole + turn;
        for (int i = 0; i < rest; ++i) at += xcd_of(whole, i) < xcd;
      }
      order[at] = e;
    }
    __syncthreads();
    return reached;
  }

  // Zeros in dw, or in its parts, for the experts without rows, order[reached] and on, 64 KB a workgroup in turn
  // (5.3 TB/s; 8 rows of 256 experts, 312 x 4152, both gradients 142 us, by products of no steps 312).
  static __device__ __forceinline__ void clear_absent(const Gemm16Args& g, const int32_t* order, int reached, int block,
                                                      int blocks) {
    constexpr int kChunk = 4096;   // of 16 bytes
    const size_t pieces = (size_t)g.N * g.K * sizeof(O) / 16;
    const int chunks = (int)((pieces + kChunk - 1) / kChunk);
    const long long all = (long long)(g.E - reached) * chunks * g.splits;
    for (long long u = block; u < all; u += blocks) {
      const int at = (int)(u / chunks), split = at / (g.E - reached);
      const size_t first = (size_t)(u - (long long)at * chunks) * kChunk;
      const size_t expert = order[reached + at - split * (g.E - reached)];
      i32x4_t* to = reinterpret_cast<i32x4_t*>(static_cast<O*>(g.c) + split * g.part + expert * g.N * g.K) + first;
      const int n = (int)(pieces - first < kChunk ? pieces - first : kChunk);
      for (int i = threadIdx.x; i < n; i += THREADS) __builtin_nontemporal_store(i32x4_t{0, 0, 0, 0}, to + i);
    }
  }

  // Workgroup `block` of `blocks`, a multiple of eight.
  static __device__ __forceinline__ void run(const Gemm16Args& g, uint8_t* smem, int block, int blocks) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, quad = lane >> 4;
    // the matrices' row lengths, the output's columns
    const int ldp = F == kForward ? g.K : g.N, ldq = g.K, cols = F == kForward ? g.N : g.K;
    const int col_tiles = (cols + TN - 1) / TN;
    int32_t* ring = reinterpret_cast<int32_t*>(smem + NBUF * BUFFER);   // unit n of this workgroup: ring[n & 3]
    int32_t* starts = ring + 4;
    int32_t* ends = starts + g.E + 1;
    int row_tiles = 0, total;
    if constexpr (F == kWeight) {
      const int reached = order_experts(g, starts, ends);
      clear_absent(g, ends, reached, block, blocks);
      total = reached * ((g.N + TM - 1) / TM) * col_tiles * g.splits;
    } else {
      row_tiles = make_tables<TM>(g, starts, ends);
      __syncthreads();
      total = row_tiles * col_tiles * g.splits;
    }
    // An XCD has a contiguous run of the units.  Its workgroups take them in turn, or from its queue and, when
    // that is empty, from the others': then `got` is a number from queue `from`, on its way.
    const int per = (total + 7) / 8, stride = blocks / 8, xcd = block & 7;
    int from = xcd, got = block >> 3;
    auto ask = [&] {   // (one wave)
      if (g.queue && lane == 0) got = atomicAdd(g.queue + 32 * from, 1);
      if (!g.queue) got += stride;
    };
    auto answer = [&] {   // the next unit, or -1; (one wave)
      for (;;) {
        const int at = __builtin_amdgcn_readfirstlane(got);
        if (at < min(per, total - from * per)) return from * per + at;
        if (!g.queue || ((from + 1) & 7) == xcd) return -1;
        from = (from + 1) & 7;
        ask();
      }
    };
    // A unit's number is asked for when the one two before it is done, before the outputs are stored, and told
    // behind that; the copies need it a barrier later at the earliest, since a unit has more steps than buffers.
    auto tell = [&](int n) {
      if (wave == 0) {
        const int unit = answer();
        if (lane == 0) ring[n & 3] = unit;
      }
    };
    tell(0);
    if (wave == 0) ask();
    tell(1);
    __syncthreads();
    auto unit_of = [&](int n) { return __builtin_amdgcn_readfirstlane(ring[n & 3]); };
    if (unit_of(0) < 0) return;

    // Copies run ahead of the products: unit `ld`, its step `lk`.  Copy i of a wave carries the KB of LDS
    // i WAVES + wave of its operand.  Buffer loads are bounded by the tile's part of the matrix; what lies
    // behind it, or behind the summed dimension, arrives as zeros.
    constexpr int kOut = 0x7FFFFFF0;
    constexpr int PR = P_T ? 512 / TM : 8, QR = Q_T ? 512 / TN : 8;   // rows a copy carries
    const int prow = wave * PR + lane / (64 / PR), qrow = wave * QR + lane / (64 / QR);
    const int ppiece = P_T ? (lane % (64 / PR)) ^ t_turn<TM>(prow) : (lane & 7) ^ p_turn(prow);
    const int qpiece = Q_T ? (lane % (64 / QR)) ^ t_turn<TN>(qrow) : (lane & 7) ^ q_turn(qrow);
    const int pv = prow * ldp * 2 + ppiece * 16, qv = qrow * ldq * 2 + qpiece * 16;
    Unit ld = unit_at(g, starts, ends, row_tiles, col_tiles, unit_of(0));
    int ln = 0, lk = 0;   // the unit that is copied and its step
    bool is_more = true;
    i32x4_t rp, rq;
    auto part = [](const void* m, size_t row, int col, int rows, int length) {
      return buffer_words(static_cast<const uint8_t*>(m) + (row * length + col) * 2,
                         rows > 0 ? (rows * length - col) * 2 : 0);
    };
    // the operands' parts for step lk: fixed over a unit where the summed dimension is contiguous, and then cut at
    // the unit's end of it
    int end = 0;
    auto open = [&](bool unit) {
      const int k0 = F == kWeight ? lk * 64 : (ld.k0 + lk) * 64;
      if (unit && F != kWeight) {
        const int length = F == kForward ? g.K : g.N;
        end = g.splits == 1 ? length : min(length, (ld.k0 + (((length + 63) / 64) + g.splits - 1) / g.splits) * 64);
      }
      if constexpr (F == kForward) {
        if (unit) {
          rp = part(g.p, ld.first, 0, ld.rows, ldp);
          rq = part(g.q, (size_t)ld.expert * g.N + ld.q0, 0, min(TN, g.N - ld.q0), ldq);
        }
      } else if constexpr (F == kInput) {
        if (unit) rp = part(g.p, ld.first, 0, ld.rows, ldp);
        rq = part(g.q, (size_t)ld.expert * g.N + min(k0, end), ld.q0, min(64, end - k0), ldq);
      } else {
        const int rows = min(64, ld.rows - k0);
        const size_t at = (size_t)ld.first + min(k0, ld.rows);
        rp = part(g.p, at, ld.p0, rows, ldp);
        rq = part(g.q, at, ld.q0, rows, ldq);
      }
    };
    open(true);
    auto copy_piece = [&](int i, int buf) {
      uint8_t* dst = smem + buf * BUFFER;
      if (i < PI) {
        int off = pv + i * (WAVES * PR) * ldp * 2;
        if constexpr (!P_T) off = (ld.k0 + lk) * 64 + ppiece * 8 < end ? off + (ld.k0 + lk) * 128 : kOut;
        copy_to_lds(rp, off, dst + (i * WAVES + wave) * 1024);
      } else {
        int off = qv + (i - PI) * (WAVES * QR) * ldq * 2;
        if constexpr (!Q_T) off = (ld.k0 + lk) * 64 + qpiece * 8 < end ? off + (ld.k0 + lk) * 128 : kOut;
        copy_to_lds(rq, off, dst + TM * 128 + ((i - PI) * WAVES + wave) * 1024);
      }
    };
    // Behind a step's barrier: the next step, which may be the next unit's.
    auto advance = [&] {
      if (!is_more) return;
      if (++lk < ld.steps) {
        open(false);
        return;
      }
      lk = 0;
      const int next = unit_of(++ln);
      if (next < 0) {
        is_more = false;
        return;
      }
      ld = unit_at(g, starts, ends, row_tiles, col_tiles, next);
      open(true);
    };

    // A lane's fragment of 16 rows (columns) x 64: two of eight values, h = 0 and 1.
    f32x4_t acc[MT][NT];
    const int p_at = wm * (TM / WM), q_at = wn * (TN / WN);   // the wave's first
    int pa[2], qa[2];
    if constexpr (!P_T) {
#pragma unroll
      for (int h = 0; h < 2; ++h) pa[h] = (p_at + l16) * 128 + (((quad + 4 * h) ^ p_turn(l16)) << 4);
    } else {
      const int row = 8 * quad + (l16 >> 2);
      pa[0] = row * TM * 2 + (((p_at / 8 + ((l16 & 3) >> 1)) ^ t_turn<TM>(row)) << 4) + (l16 & 1) * 8;
      pa[1] = 0;
    }
    if constexpr (!Q_T) {
      const int row = 8 * (l16 >> 2) + (l16 & 3);
#pragma unroll
      for (int h = 0; h < 2; ++h) qa[h] = TM * 128 + (q_at + row) * 128 + (((quad + 4 * h) ^ q_turn(row)) << 4);
    } else {
      const int row = 8 * quad + (l16 >> 2);
      qa[0] = TM * 128 + row * TN * 2 + (((q_at / 8 + ((l16 & 3) >> 1)) ^ t_turn<TN>(row)) << 4) + (l16 & 1) * 8;
      qa[1] = 0;
    }
    auto read_t = [](const uint8_t* at, int width, int h) {
      const i16x4_t lo = read_turned(at + (32 * h) * width * 2), hi = read_turned(at + (32 * h + 4) * width * 2);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    constexpr int SLOTS = EAGER ? MT : 2;
    i16x8_t pf[SLOTS][2], qf[NT][2];
    auto read_p = [&](int i, int slot, int buf) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (!P_T)
          pf[slot][h] = *reinterpret_cast<const i16x8_t*>(smem + buf * BUFFER + pa[h] + i * 2048);
        else
          pf[slot][h] = read_t(smem + buf * BUFFER + (pa[0] ^ (i << 5)), TM, h);
      }
    };
    auto read_q = [&](int j, int buf) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (!Q_T)
          qf[j][h] = *reinterpret_cast<const i16x8_t*>(smem + buf * BUFFER + qa[h] + (j >> 1) * 4096 + (j & 1) * 512);
        else
          qf[j][h] = read_t(smem + buf * BUFFER + TM * 128 + ((qa[0] - TM * 128) ^ (j << 5)), TN, h);
      }
    };

#pragma unroll
    for (int b = 0; b < NBUF; ++b) {
#pragma unroll
      for (int i = 0; i < COPIES; ++i) copy_piece(i, b);
      advance();
    }
    int ahead = NBUF - 1;   // copies of whole steps that may be in flight behind those of the step that is waited for
    // waits for all copies but those of the last `ahead` steps
    auto landed = [&](int ahead) {
      if (ahead == NBUF - 1)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 1) * COPIES) : "memory");
      else if (ahead == NBUF - 2)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * COPIES) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    };
    landed(ahead);
    ahead = NBUF - 2;
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < NT; ++j) read_q(j, 0);
#pragma unroll
    for (int i = 0; i < (EAGER ? MT : 1); ++i) read_p(i, i, 0);
    int buf = 0;
    auto after = [](int b) { return NBUF == 2 ? b ^ 1 : b == NBUF - 1 ? 0 : b + 1; };
    constexpr int EACH = (COPIES + NT - 1) / NT;   // copies beside a column of the last two row tiles
    for (int n = 0;; ++n) {
      const int unit = unit_of(n);
      if (unit < 0) return;
      const Unit cu = unit_at(g, starts, ends, row_tiles, col_tiles, unit);
      // A wave whose rows all lie behind the tile's last only copies and keeps step; its SIMD's other wave has the
      // matrix unit to itself (8192 rows of 8 uneven experts x 11008 x 4096, by trace, 709 us, without 734; the gradients
      // of 32768 of 64 x 768 x 2048 299 and 304).
      const bool idle = WM > 1 && (F == kWeight ? g.N - cu.p0 : cu.rows) <= wm * (TM / WM);
      if (idle) {
        for (int k = 0; k < cu.steps; ++k, buf = after(buf)) {
          landed(ahead);
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          const bool more = is_more;
          if (more) {
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy_piece(i, buf);
          }
          advance();
          if (!more) ahead = 0;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) read_q(j, buf);
        read_p(0, 0, buf);
        continue;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
      for (int k = 0; k < cu.steps; ++k, buf = after(buf)) {
        const int next = after(buf);
        if constexpr (EAGER) {
          landed(ahead);
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          const bool more = is_more;
          if (more) {
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy_piece(i, buf);
          }
#pragma unroll
          for (int i = 0; i < MT - 2; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < NT; ++j) acc[i][j] = mfma16(qf[j][h], pf[i][h], acc[i][j], T{});
            read_p(i, i, next);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              acc[MT - 2][j] = mfma16(qf[j][h], pf[SLOTS - 2][h], acc[MT - 2][j], T{});
              acc[MT - 1][j] = mfma16(qf[j][h], pf[SLOTS - 1][h], acc[MT - 1][j], T{});
            }
            read_q(j, next);
            __builtin_amdgcn_sched_barrier(0);
          }
          read_p(MT - 2, SLOTS - 2, next);
          read_p(MT - 1, SLOTS - 1, next);
          advance();
          if (!more) ahead = 0;
          continue;
        }
        // all columns of one row tile after the other, the next tile's fragment on its way
#pragma unroll
        for (int i = 0; i < MT - 2; ++i) {
          read_p(i + 1, (i + 1) & 1, buf);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = mfma16(qf[j][h], pf[i & 1][h], acc[i][j], T{});
          if (i == MT - 3) read_p(MT - 1, (MT - 1) & 1, buf);
          __builtin_amdgcn_sched_barrier(0);
        }
        // the next step's tiles have landed, and every wave has read what it needs of this one's
        landed(ahead);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // the last two row tiles column by column, so that Q's fragments fall free for the next step's
        const bool more = is_more;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[MT - 2][j] = mfma16(qf[j][h], pf[MT & 1][h], acc[MT - 2][j], T{});
            acc[MT - 1][j] = mfma16(qf[j][h], pf[(MT - 1) & 1][h], acc[MT - 1][j], T{});
          }
          if (more) {
#pragma unroll
            for (int i = j * EACH; i < (j + 1) * EACH; ++i)
              if (i < COPIES) copy_piece(i, buf);
          }
          read_q(j, next);
          if (j == NT - 1) read_p(0, 0, next);
          __builtin_amdgcn_sched_barrier(0);
        }
        advance();
        if (!more) ahead = 0;
      }
      const bool asks = is_more && wave == 0;
      if (asks) ask();
      store(g, cu, cols, wm, wn, l16, quad, acc);
      if (asks) tell(n + 2);
    }
  }

  static __device__ __forceinline__ void store(const Gemm16Args& g, const Unit& cu, int cols, int wm, int wn, int l16,
                                               int quad, f32x4_t (&acc)[MT][NT]) {
    // bounded by the tile's rows
    const int rows = F == kWeight ? min(TM, g.N - cu.p0) : cu.rows;
    const size_t first = F == kWeight ? (size_t)cu.expert * g.N + cu.p0 : (size_t)cu.first;
    const Buffer c = tile_buffer(static_cast<const uint8_t*>(g.c) + (cu.split * g.part + first * cols) * sizeof(O),
                                 rows * cols * (int)sizeof(O));
    constexpr int AUX = STREAMED ? 2 : 0;
    const int n0 = cu.q0 + wn * (TN / WN), m0 = wm * (TM / WM), h8 = l16 >> 3, l8 = l16 & 7;
    auto put = [&](i32x4_t v, int row, int n) {
      __builtin_amdgcn_raw_buffer_store_b128(v, c, n < cols ? (row * cols + n) * (int)sizeof(O) : 0x7FFFFFF0, 0, AUX);
    };
    // Two 16-byte pieces of a row, from columns n and m on, as whole lines of two rows.
    auto put_two = [&](i32x4_t first, i32x4_t second, int i, int n, int m) {
      trade_lines(first, second);
      put(first, m0 + i * 16 + l8, n0 + (h8 ? m : n));
      put(second, m0 + i * 16 + 8 + l8, n0 + (h8 ? m : n));
    };
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if constexpr (sizeof(O) == 4) {
#pragma unroll
        for (int j = 0; j < NT; j += 2)
          put_two(__builtin_bit_cast(i32x4_t, acc[i][j]), __builtin_bit_cast(i32x4_t, acc[i][j + 1]), i,
                  16 * j + (WIDE ? 8 : 4) * quad, WIDE ? 16 * j + 8 * quad + 4 : 16 * j + 16 + 4 * quad);
      } else {
        i32x4_t v[NT / 2];
        const int at = WIDE ? 8 * quad : 16 * (quad & 1) + 8 * (quad >> 1);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          typedef O O8 __attribute__((ext_vector_type(8)));
          O8 o;
#pragma unroll
          for (int r = 0; r < 8; ++r) o[r] = (O)acc[i][j + (r >> 2)][r & 3];
          v[j / 2] = __builtin_bit_cast(i32x4_t, o);
          if constexpr (!WIDE) {
            // columns 4 q .. + 3 of the tiles j and j + 1 to 8 (q / 2) .. + 7 of tile j + q % 2: quarters 1 and 3 of
            // the one change places with 0 and 2 of the other
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const auto both =
                  __builtin_amdgcn_permlane16_swap((uint32_t)v[j / 2][d], (uint32_t)v[j / 2][2 + d], false, false);
              v[j / 2][d] = (int)both[0];
              v[j / 2][2 + d] = (int)both[1];
            }
          }
        }
        if constexpr (NT == 4)
          put_two(v[0], v[1], i, at, 32 + at);
        else
          put(v[0], m0 + i * 16 + l16, n0 + at);
      }
    }
  }
};

template <typename KERNEL>
__global__ __launch_bounds__(KERNEL::THREADS) void k_gemm16(Gemm16Args g) {
  extern __shared__ __align__(16) uint8_t smem[];
  KERNEL::run(g, smem, blockIdx.x, gridDim.x);
}

}  // namespace zinc
