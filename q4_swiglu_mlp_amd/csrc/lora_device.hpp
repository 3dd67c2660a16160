// Device code of the low-rank adapters (k_lora.hip):
//   forward   h = A_e x,  y = base + s_e B_e h
//   backward  dh = B_e^T dy,  dx = base + s_e A_e^T dh,  dA_e = s_e dh^T x,  dB_e = s_e dy^T h
// over the rows of adapter e, which the plan (zinc_moe_sort of the rows' adapter ids) lists.  "Position" is
// a row's place in the plan, by adapter.
//
// h and dh are kept in fp32 as parts of their sums ([splits][rows][rank], added in order where they are
// read).  As operands of the second products they are two 16-bit terms, high and low: 16 bits of a value in
// bf16, 21 in fp16, so that they cost the 16-bit results nothing.  fp16's range is not fp32's: its terms
// are taken of h times a power of two, of the row (expand) or of all rows so far (gradients of A and B).
#pragma once

#include "gemm16_tile.hpp"

namespace zinc {

constexpr int kMaxRank = 256;

struct LoraPlan {
  const int32_t *offsets, *slot_row, *row_slot;
  int E, M;
};

// A row of the matrices by its position; -1 where the plan names none.
__device__ __forceinline__ int row_at(const LoraPlan& p, int position) {
  const int row = p.row_slot[position];
  return row >= 0 && row < p.M ? row : -1;
}

__device__ __forceinline__ i16x8_t load16(const void* p) { return *static_cast<const i16x8_t*>(p); }

// v as two 16-bit terms.
template <typename T>
__device__ __forceinline__ void two_terms(float v, T& hi, T& lo) {
  hi = (T)v;
  const float rest = v - (float)hi;
  lo = (T)(__builtin_isfinite(rest) ? rest : 0.0f);   // an infinity stays one
}

// The power of two that brings values of at most `top` (the bits of a largest finite magnitude) to 2^13 and above, below
// 2^14, as the exponent to multiply by; bf16 has fp32's range and needs none.
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

// ---------------------------------------------------------------- the first products
// parts[split][position][j] = sum over the split's columns c of z[row][c] w[j][c], or w[c][j] (W_T), j < rank.
// A workgroup takes 16 RT rows of one adapter and a part of the columns, its four waves 32 columns in turn;
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
  static constexpr int TM = 16 * RT;
  // LDS: the waves' sums; W_T: before that each wave's 32 x rank of w
  static size_t smem_bytes() {
    const size_t sums = 3 * (size_t)RT * JT * 1024, stage = W_T ? 4 * (size_t)(32 * JT * 16 * 2 + 64) : 0;
    return sums > stage ? sums : stage;
  }

  static __device__ __forceinline__ void run(const ShrinkArgs& s, uint8_t* smem) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int tile = blockIdx.x / s.splits, split = blockIdx.x - tile * s.splits;
    const RowTile rt = find_tile<TM>(s.plan.offsets, s.plan.E, s.plan.M, tile);
    if (rt.rows <= 0) return;
    const int C = s.C, rank = s.rank;
    const int c0 = split * s.each, c1 = min(C, c0 + s.each);
    const T* z[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int at = i * 16 + l16;
      const int row = at < rt.rows ? row_at(s.plan, rt.first + at) : -1;
      z[i] = row < 0 ? nullptr : static_cast<const T*>(s.z) + (size_t)row * C;
    }
    const T* w = static_cast<const T*>(s.w) + (size_t)rt.expert * rank * C;
    uint8_t* stage = smem + wave * (32 * JT * 16 * 2 + 64);
    f32x4_t acc[RT][JT] = {};
    for (int c = c0 + wave * 32; c < c1; c += 128) {
      const int at = c + 8 * quad;
      const bool in = at < C;
      i16x8_t zf[RT], wf[JT];
#pragma unroll
      for (int i = 0; i < RT; ++i) zf[i] = in && z[i] ? load16(z[i] + at) : i16x8_t{};
      if constexpr (!W_T) {
#pragma unroll
        for (int j = 0; j < JT; ++j)
          wf[j] = in && j * 16 + l16 < rank ? load16(w + (size_t)(j * 16 + l16) * C + at) : i16x8_t{};
      } else {
        // 32 rows of w, one after the other, to LDS; zeros behind the last
        const int bytes = (min(C, c + 32) - c) * rank * 2, all = 32 * rank * 2;
        i16x8_t v[JT];
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int b = (j * 64 + lane) * 16;
          v[j] = b < bytes ? load16(reinterpret_cast<const uint8_t*>(w + (size_t)c * rank) + b) : i16x8_t{};
        }
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int b = (j * 64 + lane) * 16;
          if (b < all) *reinterpret_cast<i16x8_t*>(stage + b) = v[j];
        }
        __builtin_amdgcn_wave_barrier();
        const uint8_t* from = stage + (8 * quad + (l16 >> 2)) * rank * 2 + (l16 & 3) * 8;
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          // (columns from the rank on are the next row's, or what lies behind: their sums are not stored)
          const i16x4_t lo = read_turned(from + j * 32), hi = read_turned(from + 4 * rank * 2 + j * 32);
          wf[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j) acc[i][j] = mfma16(wf[j], zf[i], acc[i][j], T{});
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
// are base's.  A workgroup takes 16 RT rows of one adapter and kSpan columns, a wave 32 columns in turn.
struct ExpandArgs {
  LoraPlan plan;
  const float* parts;
  int splits, rank, N;
  const void* w;     // [E][N][rank], or [E][rank][N]
  const float* scales;   // may be null: ones
  const void* base;      // may be null: zeros
  void* y;
  int row_tiles;   // of the rows with adapters; behind them workgroups for those without
};

constexpr int kSpan = 512, kCopied = 64;   // columns and, of rows without an adapter, rows a workgroup

template <typename T, int JT, int RT, bool W_T>
struct Expand {
  static constexpr int TM = 16 * RT, KT = (JT + 1) / 2;
  static constexpr int STRIDE = JT * 16 + 4;   // floats a row of f, in LDS
  // LDS: f's rows, their exponents; W_T: each wave's 32 columns of w, [rank][32]
  static size_t smem_bytes() { return (size_t)TM * STRIDE * 4 + TM * 4 + (W_T ? 4 * (size_t)KT * 32 * 64 : 0); }

  static __device__ __forceinline__ void copy_rows(const ExpandArgs& s, int first) {
    const int n = blockIdx.y * kSpan + (threadIdx.x & 63) * 8;
    if (n >= s.N) return;
    for (int row = first + (threadIdx.x >> 6); row < min(s.plan.M, first + kCopied); row += 4) {
      const int at = s.plan.slot_row[row];
      if (at >= 0 && at < s.plan.M) continue;
      const size_t to = (size_t)row * s.N + n;
      *reinterpret_cast<i16x8_t*>(static_cast<T*>(s.y) + to) =
          s.base ? load16(static_cast<const T*>(s.base) + to) : i16x8_t{};
    }
  }

  static __device__ __forceinline__ void run(const ExpandArgs& s, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int tile = blockIdx.x, span = blockIdx.y;
    if (tile >= s.row_tiles) {
      copy_rows(s, (tile - s.row_tiles) * kCopied);
      return;
    }
    const RowTile rt = find_tile<TM>(s.plan.offsets, s.plan.E, s.plan.M, tile);
    if (rt.rows <= 0) return;
    const int N = s.N, rank = s.rank;
    float* f = reinterpret_cast<float*>(smem);
    int* lifts = reinterpret_cast<int*>(f + TM * STRIDE);
    for (int i = tid * 4; i < TM * JT * 16; i += 1024) {
      const int m = i / (JT * 16), j = i - m * (JT * 16);
      f32x4_t v = {};
      if (m < rt.rows && j < rank) {
        const float* at = s.parts + (size_t)(rt.first + m) * rank + j;
        v = *reinterpret_cast<const f32x4_t*>(at);
        for (int p = 1; p < s.splits; ++p)
          v += *reinterpret_cast<const f32x4_t*>(at + (size_t)p * s.plan.M * rank);
      }
      *reinterpret_cast<f32x4_t*>(f + m * STRIDE + j) = v;
    }
    __syncthreads();
    if (tid < TM) {
      uint32_t top = 0;
      for (int j = 0; j < JT * 16; ++j) top = max(top, finite_bits(f[tid * STRIDE + j]));
      lifts[tid] = lift(top, T{});
    }
    __syncthreads();
    const float scale = s.scales ? s.scales[rt.expert] : 1.0f;
    i16x8_t fh[RT][KT], fl[RT][KT];
    float back[RT];
    T* y[RT];
    const T* base[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = i * 16 + l16, e = lifts[m];
      const float up = power(e);
      back[i] = power(-e);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        T hi[8], lo[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int j = k * 32 + 8 * quad + r;
          two_terms(j < JT * 16 ? f[m * STRIDE + j] * up : 0.0f, hi[r], lo[r]);
        }
        fh[i][k] = *reinterpret_cast<i16x8_t*>(hi);
        fl[i][k] = *reinterpret_cast<i16x8_t*>(lo);
      }
      const int row = m < rt.rows ? row_at(s.plan, rt.first + m) : -1;
      y[i] = row < 0 ? nullptr : static_cast<T*>(s.y) + (size_t)row * N;
      base[i] = row < 0 || !s.base ? nullptr : static_cast<const T*>(s.base) + (size_t)row * N;
    }
    const T* w = static_cast<const T*>(s.w) + (size_t)rt.expert * N * rank;
    uint8_t* stage = smem + TM * STRIDE * 4 + TM * 4 + wave * KT * 32 * 64;
    const int end = min(N, (span + 1) * kSpan);
    for (int n0 = span * kSpan + wave * 32; n0 < end; n0 += 128) {
      // MFMA row 4 q + r of tile j is column 8 q + 4 j + r, so that a lane holds eight neighbours
      i16x8_t wf[2][KT];
      if constexpr (!W_T) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = n0 + 8 * (l16 >> 2) + 4 * j + (l16 & 3);
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const int at = k * 32 + 8 * quad;
            wf[j][k] = n < N && at < rank ? load16(w + (size_t)n * rank + at) : i16x8_t{};
          }
        }
      } else {
        i16x8_t v[KT * 2];
#pragma unroll
        for (int i = 0; i < KT * 2; ++i) {
          const int j = i * 16 + (lane >> 2), n = n0 + (lane & 3) * 8;
          v[i] = j < rank && n < N ? load16(w + (size_t)j * N + n) : i16x8_t{};
        }
#pragma unroll
        for (int i = 0; i < KT * 2; ++i) *reinterpret_cast<i16x8_t*>(stage + (i * 64 + lane) * 16) = v[i];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const uint8_t* from = stage + (k * 32 + 8 * quad + (l16 >> 2)) * 64 + (l16 & 3) * 16 + j * 8;
            const i16x4_t lo = read_turned(from), hi = read_turned(from + 256);
            wf[j][k] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        __builtin_amdgcn_wave_barrier();
      }
      const int n = n0 + 8 * quad;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float v[8] = {};
        const bool in = y[i] && n < N;
        if (in && base[i]) load8(base[i] + n, v);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x4_t acc = {};
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            acc = mfma16(wf[j][k], fl[i][k], acc, T{});
            acc = mfma16(wf[j][k], fh[i][k], acc, T{});
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) v[4 * j + r] = fmaf(scale, acc[r] * back[i], v[4 * j + r]);
        }
        if (in) store8(y[i] + n, v);
      }
    }
  }
};

// ---------------------------------------------------------------- the adapters' gradients
// out[c][j] (or out[j][c], J_FIRST) = s_e sum over the adapter's positions p of z[row(p)][c] f[p][j].
// A workgroup takes 64 columns of one adapter and a part of its rows, 64 at a time: z's rows and f's two
// terms go to LDS and both operands are read transposed.  Each wave has 16 columns.
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
  static constexpr int FROW = JT * 32;   // bytes
  static size_t smem_bytes() { return 64 * 128 + 2 * 64 * FROW + 64; }

  static __device__ __forceinline__ void run(const LoraGradArgs& s, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int col_tiles = (s.C + 63) / 64;
    const int e = blockIdx.x / (col_tiles * s.splits), in = blockIdx.x - e * col_tiles * s.splits;
    const int split = in / col_tiles, c0 = (in - split * col_tiles) * 64;
    const int lo = min(max(s.plan.offsets[e], 0), s.plan.M), hi = min(max(s.plan.offsets[e + 1], lo), s.plan.M);
    const int each = ((hi - lo + s.splits - 1) / s.splits + 63) / 64 * 64;
    const int p0 = min(hi, lo + split * each), p1 = min(hi, p0 + each);
    const int rank = s.rank;
    uint8_t *zt = smem, *fh = smem + 64 * 128, *fl = fh + 64 * FROW;
    uint32_t* tops = reinterpret_cast<uint32_t*>(fl + 64 * FROW);
    f32x4_t acc[JT] = {};
    int lifted = 100;   // the sums are of f times 2^lifted
    for (int p = p0; p < p1; p += 64) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = i * 32 + (tid >> 3), c = c0 + (tid & 7) * 8;
        const int row = p + at < p1 ? row_at(s.plan, p + at) : -1;
        const i16x8_t v =
            row >= 0 && c < s.C ? load16(static_cast<const T*>(s.z) + (size_t)row * s.C + c) : i16x8_t{};
        *reinterpret_cast<i16x8_t*>(zt + at * 128 + (((tid & 7) ^ (2 * (((at >> 1) & 1) + 2 * ((at >> 3) & 1)))) << 4)) = v;
      }
      float v[JT * 4];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < JT; ++i) {
        const int at = (i * 256 + tid) / (JT * 4), j = ((i * 256 + tid) % (JT * 4)) * 4;
        f32x4_t t = {};
        if (p + at < p1 && j < rank && row_at(s.plan, p + at) >= 0) {
          const float* from = s.f + (size_t)(p + at) * rank + j;
          t = *reinterpret_cast<const f32x4_t*>(from);
          for (int q = 1; q < s.f_splits; ++q)
            t += *reinterpret_cast<const f32x4_t*>(from + (size_t)q * s.plan.M * rank);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[i * 4 + r] = t[r];
          top = max(top, finite_bits(t[r]));
        }
      }
      if constexpr (sizeof(T) == 2 && !__is_same(T, __bf16)) {
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
          for (int j = 0; j < JT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][r] *= by;
          lifted = up;
        }
      } else {
        lifted = 0;
      }
      const float up = power(lifted);
#pragma unroll
      for (int i = 0; i < JT; ++i) {
        const int at = (i * 256 + tid) / (JT * 4), j = ((i * 256 + tid) % (JT * 4)) * 4;
        T h4[4], l4[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) two_terms(v[i * 4 + r] * up, h4[r], l4[r]);
        *reinterpret_cast<i16x4_t*>(fh + at * FROW + j * 2) = *reinterpret_cast<i16x4_t*>(h4);
        *reinterpret_cast<i16x4_t*>(fl + at * FROW + j * 2) = *reinterpret_cast<i16x4_t*>(l4);
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 32 * h + 8 * quad + (l16 >> 2);
        auto two = [](const uint8_t* a, int stride) {
          const i16x4_t x = read_turned(a), y = read_turned(a + 4 * stride);
          return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        const int turn = 2 * (((row >> 1) & 1) + 2 * ((row >> 3) & 1));
        const i16x8_t zf =
            two(zt + row * 128 + (((2 * wave + ((l16 & 3) >> 1)) ^ turn) << 4) + (l16 & 1) * 8, 128);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int at = row * FROW + j * 32 + (l16 & 3) * 8;
          const i16x8_t a = two(fl + at, FROW), b = two(fh + at, FROW);
          if constexpr (J_FIRST) {
            acc[j] = mfma16(zf, a, acc[j], T{});
            acc[j] = mfma16(zf, b, acc[j], T{});
          } else {
            acc[j] = mfma16(a, zf, acc[j], T{});
            acc[j] = mfma16(b, zf, acc[j], T{});
          }
        }
      }
      __syncthreads();
    }
    const float back = power(-lifted);
    const float scale = s.scales ? s.scales[e] : 1.0f;
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      // a lane's four sums: J_FIRST four neighbouring c of one j, else four j of one c
      const int c = c0 + wave * 16 + (J_FIRST ? 4 * quad : l16), at = j * 16 + (J_FIRST ? l16 : 4 * quad);
      if (c >= s.C || at >= rank) continue;
      const size_t to = J_FIRST ? ((size_t)e * rank + at) * s.C + c : ((size_t)e * s.C + c) * rank + at;
      f32x4_t v = acc[j] * back;
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
