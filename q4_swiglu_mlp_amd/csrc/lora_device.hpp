// Device code of the low-rank adapters (k_lora_*.hip):
//   forward   h = A_e x,  y = base + s_e B_e h
//   backward  dh = B_e^T dy,  dx = base + s_e A_e^T dh,  dA_e = s_e dh^T x,  dB_e = s_e dy^T h
// over the rows of adapter e, which the plan (zinc_moe_sort of the rows' adapter ids) lists.  "Position" is
// a row's place in the plan, by adapter.
//
// h and dh are kept in fp32 as parts of their sums ([splits][rows][rank], added in order where they are
// read).  As operands of the second products they are sums of 16-bit terms: three in bf16, which are all of fp32's
// 24 bits (two, 16 bits, take 14 % less in the gradients of rank 128, 8 % of rank 64, 1 % in the rest of up to 64, but
// sums that cancel show the rest); two in fp16, 22 bits: off by 2^-22 of a value at most, as four of the 2^-24 that
// each addition of the sum before may be off by, of which there are eight at least.  fp16's range is not fp32's: its
// terms are taken of h times a power of two, of the row (expand) or of all rows so far (gradients of A and B).
#pragma once

#include "gemm16_tile.hpp"

namespace zinc {

struct LoraPlan {
  const int32_t *offsets, *slot_row, *row_slot;
  int E, M;
};

// A row of the matrices by its position; -1 where the plan names none.
__device__ __forceinline__ int row_at(const LoraPlan& p, int position) {
  const int row = p.row_slot[position];
  return row >= 0 && row < p.M ? row : -1;
}

// The positions of adapter e: lo up to hi.
__device__ __forceinline__ void positions_of(const LoraPlan& p, int e, int& lo, int& hi) {
  lo = min(max(p.offsets[e], 0), p.M);
  hi = min(max(p.offsets[e + 1], lo), p.M);
}

// What a gradient of adapter e is multiplied by.  One without rows is zeros, whatever its scale: that of a slot that
// nobody uses may never have been written.
__device__ __forceinline__ float grad_scale(const float* scales, int e, bool has_rows) {
  return scales && has_rows ? scales[e] : 1.0f;
}

__device__ __forceinline__ i16x8_t load16(const void* p) { return *static_cast<const i16x8_t*>(p); }

// v as the sum of its 16-bit terms, the largest first; what each leaves is exact.  set(term, value).
template <typename T>
constexpr int kTerms = __is_same(T, __bf16) ? 3 : 2;
template <typename T, typename SET>
__device__ __forceinline__ void split_terms(float v, SET set) {
#pragma unroll
  for (int t = 0; t < kTerms<T>; ++t) {
    const T term = (T)v;
    set(t, term);
    v -= (float)term;
    if (t == 0) v = __builtin_isfinite(v) ? v : 0.0f;   // an infinity stays one
  }
}

// The power of two that brings values of at most `top` (the bits of a largest finite magnitude) to 2^13 and above,
// below 2^14, as the exponent to multiply by; bf16 has fp32's range and needs none.
__device__ __forceinline__ int lift(uint32_t top, _Float16) {
  if (top == 0) return 0;
  const int e = 13 + 127 - (int)(top >> 23);
  return e > 100 ? 100 : e;
}
__device__ __forceinline__ int lift(uint32_t, __bf16) { return 0; }
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| <= 126

__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = abs_bits(v);
  return b < 0x7F800000u ? b : 0u;
}

// trade_lines of operands as the MFMAs take them.
__device__ __forceinline__ void trade_lines(i16x8_t& first, i16x8_t& second) {
  i32x4_t x = __builtin_bit_cast(i32x4_t, first), y = __builtin_bit_cast(i32x4_t, second);
  trade_lines(x, y);
  first = __builtin_bit_cast(i16x8_t, x);
  second = __builtin_bit_cast(i16x8_t, y);
}

// F pieces of f a thread: the sums of their parts in order; load(part, piece).  The first part and up to four more of
// every piece are in flight at a time (1626 rows of 16 adapters of rank 128, 2048 to 2048, gradients: the second
// launch 38 us, piece by piece 45).
template <int F, typename LOAD>
__device__ __forceinline__ void sum_parts(f32x4_t (&v)[F], int splits, LOAD load) {
  constexpr int G = F <= 2 ? 4 : F <= 4 ? 2 : 1;
#pragma unroll
  for (int i = 0; i < F; ++i) v[i] = load(0, i);
  for (int q = 1; q < splits; q += G) {
    f32x4_t t[G][F];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < F; ++i) t[g][i] = load(q + g < splits ? q + g : 0, i);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < F; ++i)
        if (q + g < splits) v[i] += t[g][i];
  }
}

// ---------------------------------------------------------------- the first products
// parts[split][position][j] = sum over the split's columns c of z[row][c] w[j][c], or w[c][j] (W_T), j < rank.
// A workgroup takes 16 RT rows of one adapter and a part of the columns, its four waves 32 or 64 columns in turn;
// their sums are joined in LDS.  w is the MFMA's row operand: a lane holds four neighbouring j of one row.
struct ShrinkArgs {
  LoraPlan plan;
  const void* z;     // [M][C]
  const void* w;     // [E][rank][C], or [E][C][rank]
  int C, rank, splits, each;   // columns a split, a multiple of 32
  float* parts;
};

template <typename T, int JT, int RT, bool W_T>
struct Shrink {
  static constexpr int kTiles = JT, TM = 16 * RT;
  static constexpr int KS = JT <= 4 ? 2 : 1, COLS = 32 * KS;   // columns of a wave's step
  static constexpr int STAGE = COLS * JT * 16 * 2 + 64;        // bytes
  // LDS: the waves' sums; W_T: before that each wave's COLS x rank of w
  static size_t smem_bytes() {
    const size_t sums = 3 * (size_t)RT * JT * 1024, stage = W_T ? 4 * (size_t)STAGE : 0;
    return sums > stage ? sums : stage;
  }

  static __device__ __forceinline__ void run(const ShrinkArgs& s, int block, uint8_t* smem) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int tile = block / s.splits, split = block - tile * s.splits;
    const RowTile rt = find_tile<TM>(s.plan.offsets, s.plan.E, s.plan.M, tile);
    if (rt.rows <= 0) return;
    const int C = s.C, rank = s.rank;
    const int c1 = min(C, (split + 1) * s.each);
    const int h8 = l16 >> 3, l8 = l16 & 7;
    // the rows that the lane loads: its own, or (KS 2, in whole lines) l8 and 8 + l8 of each tile
    const T* z[RT][KS];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int at = i * 16 + (KS == 2 ? 8 * k + l8 : l16);
        const int row = at < rt.rows ? row_at(s.plan, rt.first + at) : -1;
        z[i][k] = row < 0 ? nullptr : static_cast<const T*>(s.z) + (size_t)row * C;
      }
    const T* w = static_cast<const T*>(s.w) + (size_t)rt.expert * rank * C;
    uint8_t* stage = smem + wave * STAGE;

    // a step's operands, on their way while the step before is multiplied
    struct Step {
      i16x8_t z[RT][KS], w[JT][KS];
    };
    auto load = [&](int c, Step& d) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int at = c + 8 * quad + (KS == 2 ? 32 * h8 : 0);
#pragma unroll
        for (int i = 0; i < RT; ++i) d.z[i][k] = at < c1 && z[i][k] ? load16(z[i][k] + at) : i16x8_t{};
        if constexpr (!W_T) {
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const int n = j * 16 + (KS == 2 ? 8 * k + l8 : l16);
            d.w[j][k] = at < c1 && n < rank ? load16(w + (size_t)n * C + at) : i16x8_t{};
          }
        } else {   // COLS rows of w, one after the other
          const int bytes = (min(c1, c + COLS) - c) * rank * 2;
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const int b = ((k * JT + j) * 64 + lane) * 16;
            d.w[j][k] = b < bytes ? load16(reinterpret_cast<const uint8_t*>(w + (size_t)c * rank) + b) : i16x8_t{};
          }
        }
      }
    };
    f32x4_t acc[RT][JT] = {};
    auto multiply = [&](Step& d) {
      if constexpr (KS == 2) {
#pragma unroll
        for (int i = 0; i < RT; ++i) trade_lines(d.z[i][0], d.z[i][1]);
        if constexpr (!W_T) {
#pragma unroll
          for (int j = 0; j < JT; ++j) trade_lines(d.w[j][0], d.w[j][1]);
        }
      }
      if constexpr (W_T) {   // by way of LDS; zeros behind the last row
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const int b = ((k * JT + j) * 64 + lane) * 16;
            if (b < COLS * rank * 2) *reinterpret_cast<i16x8_t*>(stage + b) = d.w[j][k];
          }
        __builtin_amdgcn_wave_barrier();
        const uint8_t* from = stage + (8 * quad + (l16 >> 2)) * rank * 2 + (l16 & 3) * 8;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            // (columns from the rank on are the next row's, or what lies behind: their sums are not stored)
            const uint8_t* at = from + k * 64 * rank + j * 32;
            const i16x4_t lo = read_turned(at), hi = read_turned(at + 8 * rank);
            d.w[j][k] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < JT; ++j) acc[i][j] = mfma16(d.w[j][k], d.z[i][k], acc[i][j], T{});
    };
    Step d[2];
    int c = split * s.each + wave * COLS;
    if (c < c1) load(c, d[0]);
    for (; c < c1; c += 8 * COLS) {
      if (c + 4 * COLS < c1) load(c + 4 * COLS, d[1]);
      multiply(d[0]);
      if (c + 4 * COLS >= c1) break;
      if (c + 8 * COLS < c1) load(c + 8 * COLS, d[0]);
      multiply(d[1]);
    }

    f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem);
    if constexpr (W_T) __syncthreads();
    if (wave) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j) sums[(((wave - 1) * RT + i) * JT + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int at = i * 16 + l16;
      float* out = s.parts + ((size_t)split * s.plan.M + rt.first + at) * rank;
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        f32x4_t v = acc[i][j];
#pragma unroll
        for (int o = 0; o < 3; ++o) v += sums[((o * RT + i) * JT + j) * 64 + lane];
        const int n = j * 16 + 4 * quad;
        if (at < rt.rows && n < rank) *reinterpret_cast<f32x4_t*>(out + n) = v;
      }
    }
  }
};

// ---------------------------------------------------------------- the second products
// y[row][n] = base[row][n] + s_e sum_j f[position][j] w[n][j], or w[j][n] (W_T); y's rows without an adapter
// are base's.  A workgroup takes 16 RT rows of one adapter and `span` columns, a wave 32 or 64 columns in turn; the
// operands of the next are on their way while one is multiplied (before y is stored, which may be base).
struct ExpandArgs {
  LoraPlan plan;
  const float* parts;
  int splits, rank, N;
  const void* w;     // [E][N][rank], or [E][rank][N]
  const float* scales;   // may be null: ones
  const void* base;      // may be null: zeros
  void* y;
  int span;            // columns a workgroup, a multiple of 256
  int row_tiles;       // of the rows with adapters
  int spans;           // of a row
  int copies;          // before them: groups of kCopied rows, of which those without an adapter are copied
};

constexpr int kCopied = 64;

template <typename T, int JT, int RT, bool W_T, int CP = JT <= 4 ? 2 : 1>
struct Expand {
  static constexpr int kTiles = JT, TM = 16 * RT, KT = (JT + 1) / 2;
  static constexpr int COLS = 32 * CP;   // columns of a wave's step
  static constexpr int STRIDE = JT * 16 + 4;   // floats a row of f, in LDS
  static constexpr int STAGE = KT * 32 * COLS * 2;   // bytes
  // Many rows of base and y pass the caches by, where they move in whole lines: 8192 x 11008, bf16, rank 64
  // 93 us through the caches, 93 with y past them, 90 with both; rank 16 82, 77 and 71.
  static constexpr bool STREAMED = CP == 2 && RT > 1;
  static __device__ __forceinline__ i16x8_t load_base(const T* p) {
    if constexpr (STREAMED)
      return __builtin_nontemporal_load(reinterpret_cast<const i16x8_t*>(p));
    else
      return load16(p);
  }
  // f's terms, of which the four waves hold the same fragments; the last one lies in LDS where registers would spill
  // (rank 64, four row tiles) or a SIMD would hold one wave instead of two (rank 256, 8192 rows, 4096 to 11008: the
  // forward call 507 us, 591).
  static constexpr int TERMS = kTerms<T>, HELD = TERMS == 3 && (RT == 4 || (JT == 16 && !W_T)) ? 2 : TERMS;
  // LDS: f's rows, their exponents; the last term; W_T: each wave's COLS columns of w, [rank][COLS]
  static constexpr int LAST = TM * STRIDE * 4 + TM * 4, STAGES = LAST + (HELD < TERMS ? RT * KT * 1024 : 0);
  static size_t smem_bytes() { return STAGES + (W_T ? 4 * (size_t)STAGE : 0); }

  // Of kCopied rows those without an adapter; a wave takes a quarter of them, four at a time.
  static __device__ __forceinline__ void copy_rows(const ExpandArgs& s, int first, int span) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = first + lane < s.plan.M ? s.plan.slot_row[first + lane] : 0;
    uint32_t left = (uint32_t)(__ballot(at < 0 || at >= s.plan.M) >> (16 * wave)) & 0xFFFFu;
    const int end = min(s.N, (span + 1) * s.span);
    while (left) {
      int rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rows[i] = left ? first + 16 * wave + (int)__builtin_ctz(left) : -1;
        left &= left - 1;   // (0 stays 0)
      }
      for (int c = span * s.span + lane * 8; c < end; c += 512) {
        i16x8_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = rows[i] >= 0 && s.base ? load16(static_cast<const T*>(s.base) + (size_t)rows[i] * s.N + c) : i16x8_t{};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (rows[i] >= 0) *reinterpret_cast<i16x8_t*>(static_cast<T*>(s.y) + (size_t)rows[i] * s.N + c) = v[i];
      }
    }
  }

  static __device__ __forceinline__ void run(const ExpandArgs& s, int block, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int tile = block / s.spans, span = block - tile * s.spans;
    if (tile < s.copies) {
      copy_rows(s, tile * kCopied, span);
      return;
    }
    const RowTile rt = find_tile<TM>(s.plan.offsets, s.plan.E, s.plan.M, tile - s.copies);
    if (rt.rows <= 0) return;
    const int N = s.N, rank = s.rank, end = min(N, (span + 1) * s.span);
    const T* w = static_cast<const T*>(s.w) + (size_t)rt.expert * N * rank;
    const T* base = static_cast<const T*>(s.base);
    T* y = static_cast<T*>(s.y);
    uint8_t *stage = smem + STAGES + wave * STAGE, *last = smem + LAST + lane * 16;
    int rows[RT][CP];   // that the lane loads and stores: its own, or (CP 2, in whole lines) l8 and 8 + l8 of a tile
    const int h8 = l16 >> 3, l8 = l16 & 7;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const int at = i * 16 + (CP == 2 ? 8 * c + l8 : l16);
        rows[i][c] = at < rt.rows ? row_at(s.plan, rt.first + at) : -1;
      }
    struct Step {
      i16x8_t w[CP * 2][KT], base[RT][CP];
    };
    auto load = [&](int n0, Step& d) {
      // MFMA row 4 q + r of tile j is column 32 (j / 2) + 8 q + 4 (j % 2) + r, so that a lane holds eight neighbours
#pragma unroll
      for (int j = 0; j < CP * 2; ++j)
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          if constexpr (!W_T) {
            const int n = n0 + 32 * (j >> 1) + 8 * (l16 >> 2) + 4 * (j & 1) + (l16 & 3), at = k * 32 + 8 * quad;
            d.w[j][k] = n < N && at < rank ? load16(w + (size_t)n * rank + at) : i16x8_t{};
          } else {   // COLS columns of w's rows
            constexpr int EACH = COLS / 8;
            const int at = (j * KT + k) * (64 / EACH) + lane / EACH, n = n0 + (lane % EACH) * 8;
            d.w[j][k] = at < rank && n < N ? load16(w + (size_t)at * N + n) : i16x8_t{};
          }
        }
      const int n = n0 + 8 * quad + (CP == 2 ? 32 * h8 : 0);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < CP; ++c)
          d.base[i][c] =
              base && rows[i][c] >= 0 && n < N ? load_base(base + (size_t)rows[i][c] * N + n) : i16x8_t{};
    };
    Step d[2];
    int n0 = span * s.span + wave * COLS;
    if (n0 < end) load(n0, d[0]);   // (on its way while f is taken)

    float* f = reinterpret_cast<float*>(smem);
    int* lifts = reinterpret_cast<int*>(f + TM * STRIDE);
    constexpr int F = (TM * JT * 16 + 1023) / 1024;
    f32x4_t v[F];
    sum_parts(v, s.splits, [&](int q, int i) {
      const int m = (i * 1024 + tid * 4) / (JT * 16), j = (i * 1024 + tid * 4) - m * (JT * 16);
      if (m >= rt.rows || j >= rank) return f32x4_t{};
      return *reinterpret_cast<const f32x4_t*>(s.parts + (q * (size_t)s.plan.M + rt.first + m) * rank + j);
    });
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int m = (i * 1024 + tid * 4) / (JT * 16), j = (i * 1024 + tid * 4) - m * (JT * 16);
      if (m < TM) *reinterpret_cast<f32x4_t*>(f + m * STRIDE + j) = v[i];
    }
    __syncthreads();
    if constexpr (!__is_same(T, __bf16)) {   // four threads a row
      if (tid < TM * 4) {
        uint32_t top = 0;
        for (int j = tid & 3; j < JT * 16; j += 4) top = max(top, finite_bits(f[(tid >> 2) * STRIDE + j]));
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
        if ((tid & 3) == 0) lifts[tid >> 2] = lift(top, T{});
      }
      __syncthreads();
    }
    const float scale = s.scales ? s.scales[rt.expert] : 1.0f;
    i16x8_t ft[HELD][RT][KT];
    float back[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = i * 16 + l16, e = __is_same(T, __bf16) ? 0 : lifts[m];
      const float up = power(e);
      back[i] = power(-e);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        T terms[TERMS][8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int j = k * 32 + 8 * quad + r;
          split_terms<T>(j < JT * 16 ? f[m * STRIDE + j] * up : 0.0f, [&](int t, T v) { terms[t][r] = v; });
        }
#pragma unroll
        for (int t = 0; t < HELD; ++t) ft[t][i][k] = *reinterpret_cast<i16x8_t*>(terms[t]);
        if constexpr (HELD < TERMS)
          if (i % 4 == wave)
            *reinterpret_cast<i16x8_t*>(last + (i * KT + k) * 1024) = *reinterpret_cast<i16x8_t*>(terms[HELD]);
      }
    }
    if constexpr (HELD < TERMS) __syncthreads();

    auto multiply = [&](int n0, Step& d) {
      if constexpr (W_T) {
#pragma unroll
        for (int i = 0; i < KT * CP * 2; ++i)
          *reinterpret_cast<i16x8_t*>(stage + (i * 64 + lane) * 16) = d.w[i / KT][i % KT];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < CP * 2; ++j)
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const uint8_t* from =
                stage + (k * 32 + 8 * quad + (l16 >> 2)) * COLS * 2 + (j >> 1) * 64 + (l16 & 3) * 16 + (j & 1) * 8;
            const i16x4_t lo = read_turned(from), hi = read_turned(from + 4 * COLS * 2);
            d.w[j][k] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        __builtin_amdgcn_wave_barrier();
      }
      const int n = n0 + 8 * quad + (CP == 2 ? 32 * h8 : 0);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if constexpr (CP == 2) trade_lines(d.base[i][0], d.base[i][1]);
        i16x8_t out[CP], fl[KT];
        if constexpr (HELD < TERMS) {
          asm volatile("" ::: "memory");   // (read here each time, not held from before the loop)
#pragma unroll
          for (int k = 0; k < KT; ++k) fl[k] = *reinterpret_cast<const i16x8_t*>(last + (i * KT + k) * 1024);
        }
#pragma unroll
        for (int c = 0; c < CP; ++c) {
          typedef T T8 __attribute__((ext_vector_type(8)));
          const T8 b = __builtin_bit_cast(T8, d.base[i][c]);
          T8 o;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x4_t acc = {};
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int t = TERMS - 1; t >= 0; --t)
                acc = mfma16(d.w[2 * c + j][k], t < HELD ? ft[t < HELD ? t : 0][i][k] : fl[k], acc, T{});
#pragma unroll
            for (int r = 0; r < 4; ++r) o[4 * j + r] = (T)fmaf(scale, acc[r] * back[i], (float)b[4 * j + r]);
          }
          out[c] = __builtin_bit_cast(i16x8_t, o);
        }
        if constexpr (CP == 2) trade_lines(out[0], out[1]);
#pragma unroll
        for (int c = 0; c < CP; ++c)
          if (rows[i][c] >= 0 && n < N)
            store_vector<STREAMED>(reinterpret_cast<i16x8_t*>(y + (size_t)rows[i][c] * N + n), out[c]);
      }
    };
    for (; n0 < end; n0 += 8 * COLS) {
      if (n0 + 4 * COLS < end) load(n0 + 4 * COLS, d[1]);
      multiply(n0, d[0]);
      if (n0 + 4 * COLS >= end) break;
      if (n0 + 8 * COLS < end) load(n0 + 8 * COLS, d[0]);
      multiply(n0 + 4 * COLS, d[1]);
    }
  }
};

// ---------------------------------------------------------------- the adapters' gradients
// out[c][j] (or out[j][c], J_FIRST) = s_e sum over the adapter's positions p of z[row(p)][c] f[p][j].
// A workgroup takes 128 columns of one adapter and a part of its rows, 64 at a time: z's rows and f's
// terms go to LDS and both operands are read transposed; the next 64 rows are on their way meanwhile.  Each
// wave has 32 columns.
struct LoraGradArgs {
  LoraPlan plan;
  const void* z;      // [M][C]
  const float* f;     // parts
  int f_splits, rank, C;
  const float* scales;
  int splits;         // of the rows; more than one: fp32 sums, one after the other, unscaled
  void* out;
};

template <typename T, int JT, bool J_FIRST>
struct LoraGrad {
  static constexpr int COLS = 128, FROW = JT * 32;   // bytes a row of f's terms
  static constexpr int TERMS = kTerms<T>;
  // LDS: z's rows, f's terms one after the other, the waves' largest values
  static size_t smem_bytes() { return 64 * COLS * 2 + TERMS * 64 * FROW + 64; }

  static __device__ __forceinline__ void run(const LoraGradArgs& s, int block, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int col_tiles = (s.C + COLS - 1) / COLS;
    const int e = block / (col_tiles * s.splits), in = block - e * col_tiles * s.splits;
    const int split = in / col_tiles, c0 = (in - split * col_tiles) * COLS;
    int lo, hi;
    positions_of(s.plan, e, lo, hi);
    const int each = ((hi - lo + s.splits - 1) / s.splits + 63) / 64 * 64;
    const int p0 = min(hi, lo + split * each), p1 = min(hi, p0 + each);
    const int rank = s.rank;
    uint8_t *zt = smem, *ft = smem + 64 * COLS * 2;
    uint32_t* tops = reinterpret_cast<uint32_t*>(ft + TERMS * 64 * FROW);
    auto turn = [](int row) { return 2 * ((row & 3) + 4 * ((row >> 3) & 1)); };   // of a row's 16 pieces

    i16x8_t zv[4];
    f32x4_t fv[JT];
    const int zrow = tid >> 4, zc = c0 + (tid & 15) * 8;   // rows zrow, + 16, + 32, + 48
    int rows[4];   // of the step that is loaded next
    auto load_rows = [&](int p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = p + i * 16 + zrow;
        rows[i] = at < p1 ? row_at(s.plan, at) : -1;
      }
    };
    auto load = [&](int p) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        zv[i] = rows[i] >= 0 && zc < s.C ? load16(static_cast<const T*>(s.z) + (size_t)rows[i] * s.C + zc) : i16x8_t{};
      load_rows(p + 64);
      sum_parts(fv, s.f_splits, [&](int q, int i) {   // (f of a position without a row is zero)
        const int at = p + (i * 256 + tid) / (JT * 4), j = ((i * 256 + tid) % (JT * 4)) * 4;
        if (at >= p1 || j >= rank) return f32x4_t{};
        return *reinterpret_cast<const f32x4_t*>(s.f + (q * (size_t)s.plan.M + at) * rank + j);
      });
    };
    f32x4_t acc[2][JT] = {};
    int lifted = 100;   // the sums are of f times 2^lifted
    load_rows(p0);
    if (p0 < p1) load(p0);
    for (int p = p0; p < p1; p += 64) {
      if constexpr (!__is_same(T, __bf16)) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < JT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = max(top, finite_bits(fv[i][r]));
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        const int up = top ? min(lifted, lift(top, T{})) : lifted;
        if (up != lifted) {
          // (sums so far are zero while lifted is 100, or were of values that this leaves in range)
          const float by = up - lifted < -126 ? 0.0f : power(up - lifted);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[c][j][r] *= by;
          lifted = up;
        }
      } else {
        lifted = 0;
      }
      const float up = power(lifted);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = i * 16 + zrow;
        *reinterpret_cast<i16x8_t*>(zt + at * COLS * 2 + (((tid & 15) ^ turn(at)) << 4)) = zv[i];
      }
#pragma unroll
      for (int i = 0; i < JT; ++i) {
        const int at = (i * 256 + tid) / (JT * 4), j = ((i * 256 + tid) % (JT * 4)) * 4;
        T terms[TERMS][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) split_terms<T>(fv[i][r] * up, [&](int t, T v) { terms[t][r] = v; });
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
          *reinterpret_cast<i16x4_t*>(ft + (t * 64 + at) * FROW + j * 2) = *reinterpret_cast<i16x4_t*>(terms[t]);
      }
      if (p + 64 < p1) load(p + 64);
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 32 * h + 8 * quad + (l16 >> 2);
        auto two = [](const uint8_t* a, int stride) {
          const i16x4_t x = read_turned(a), y = read_turned(a + 4 * stride);
          return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        i16x8_t zf[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
          zf[c] = two(zt + row * COLS * 2 + (((4 * wave + 2 * c + ((l16 & 3) >> 1)) ^ turn(row)) << 4) + (l16 & 1) * 8,
                      COLS * 2);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int at = row * FROW + j * 32 + (l16 & 3) * 8;
          i16x8_t ff[TERMS];
#pragma unroll
          for (int t = 0; t < TERMS; ++t) ff[t] = two(ft + t * 64 * FROW + at, FROW);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
              acc[c][j] = J_FIRST ? mfma16(zf[c], ff[t], acc[c][j], T{}) : mfma16(ff[t], zf[c], acc[c][j], T{});
        }
      }
      __syncthreads();
    }
    const float back = power(-lifted);
    const float scale = grad_scale(s.scales, e, hi > lo);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        // a lane's four sums: J_FIRST four neighbouring c of one j, else four j of one c
        const int c = c0 + wave * 32 + k * 16 + (J_FIRST ? 4 * quad : l16), at = j * 16 + (J_FIRST ? l16 : 4 * quad);
        if (c >= s.C || at >= rank) continue;
        const size_t to = J_FIRST ? ((size_t)e * rank + at) * s.C + c : ((size_t)e * s.C + c) * rank + at;
        const f32x4_t v = acc[k][j] * back;
        if (s.splits > 1) {
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(s.out) + (size_t)split * s.plan.E * rank * s.C + to) = v;
        } else {
          typedef T T4 __attribute__((ext_vector_type(4)));
          T4 o;
#pragma unroll
          for (int r = 0; r < 4; ++r) o[r] = (T)(scale * v[r]);
          *reinterpret_cast<T4*>(static_cast<T*>(s.out) + to) = o;
        }
      }
  }
};

}  // namespace zinc
