// An MoE layer's token permutation: the sort of routed slots by expert, the
// gather of token rows into that order, the weighted way back, and gradients.
//
// The sort is a stable counting sort: slot i = t * top_k + s goes behind every
// slot of a smaller expert and behind the earlier slots of its own, so the
// order, and with it every later sum, is a function of the ids alone (no
// atomic decides a place).  It is bound by its launches and the latency of its few steps:
// 64 experts, 512 slots 3.3 us, 32768 slots 7.7 us in two launches (floor 0.1 us by bytes).
#include "fp8_device.hpp"
#include "launch.hpp"

namespace zinc {
namespace {

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int kMaxE = 1024;
// Sorted by one workgroup in one launch: 2048 slots of 64 experts 4.6 us against 6.0 in two
// launches, 4096 slots 6.6 and 6.2 (replayed; a second launch costs the host 4 us more).
constexpr int kOneBlockSlots = 4096;
constexpr int kSortMaxBlocks = 256;

// Slots per workgroup, a multiple of 512 (whole steps of 64 a wave): up to 4096
// slots one workgroup; else 1024, which spreads 65536 slots over 64 workgroups, or
// what 256 workgroups need.
int sort_tile(int S) {
  if (S <= kOneBlockSlots) return (S + kSortThreads - 1) / kSortThreads * kSortThreads;
  const int t = (S + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return ((t < 1024 ? 1024 : t) + kSortThreads - 1) / kSortThreads * kSortThreads;
}
int sort_blocks(int S) { return S > 0 ? (S + sort_tile(S) - 1) / sort_tile(S) : 0; }

// One step of a wave: 64 slots, one a lane, in order.  Returns the slot's rank among the
// wave's slots of its expert and counts them in cnt; the lanes with the same
// expert are found by ballots over the bits of the id.
__device__ __forceinline__ int rank_step(int e, bool ok, int E, int lane, int* cnt) {
  uint64_t same = __ballot(ok);
  for (int bit = 1; bit < E; bit <<= 1) {
    const uint64_t m = __ballot((e & bit) != 0);
    same &= (e & bit) ? m : ~m;
  }
  const int below = __popcll(same & ((1ull << lane) - 1));
  int rank = 0;
  if (ok) rank = cnt[e] + below;
  __builtin_amdgcn_wave_barrier();
  if (ok && below == 0) cnt[e] = rank + __popcll(same);
  __builtin_amdgcn_wave_barrier();
  return rank;
}

// Exclusive scan over the experts of count(e), two a thread; first(e, value) receives
// each.  Returns the sum.
template <typename COUNT, typename FIRST>
__device__ __forceinline__ int scan_experts(int E, int* wsum, COUNT count, FIRST first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e0 = 2 * tid, c0 = e0 < E ? count(e0) : 0, c1 = e0 + 1 < E ? count(e0 + 1) : 0;
  int scan = c0 + c1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(scan, d, 64);
    if (lane >= d) scan += o;
  }
  if (lane == 63) wsum[wave] = scan;
  __syncthreads();
  int base = scan - c0 - c1, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) base += wsum[w];
    all += wsum[w];
  }
  if (e0 < E) first(e0, base);
  if (e0 + 1 < E) first(e0 + 1, base + c0);
  return all;
}

// Up to 4096 slots: ranks stay in registers while the counts become first rows.
__global__ __launch_bounds__(kSortThreads) void k_sort_one(const int32_t* __restrict__ ids, int S, int E, int tile,
                                                           int32_t* __restrict__ offsets,
                                                           int32_t* __restrict__ slot_row,
                                                           int32_t* __restrict__ row_slot,
                                                           int32_t* __restrict__ dev_error) {
  constexpr int STEPS = kOneBlockSlots / kSortThreads;
  __shared__ int cnt[kSortWaves][kMaxE];
  __shared__ int wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int share = tile / kSortWaves, lo = wave * share, steps = share / 64;
  int e[STEPS], rank[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int i = lo + 64 * k + lane;
    e[k] = k < steps && i < S ? ids[i] : -1;
  }
  for (int j = tid; j < E; j += kSortThreads)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) cnt[w][j] = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    if (k >= steps) continue;
    const bool ok = e[k] >= 0 && e[k] < E;
    bad |= !ok && lo + 64 * k + lane < S;
    rank[k] = rank_step(e[k], ok, E, lane, cnt[wave]);
  }
  if (bad && dev_error) atomicOr(dev_error, 1);
  __syncthreads();
  const int valid = scan_experts(
      E, wsum,
      [&](int j) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c += cnt[w][j];
        return c;
      },
      [&](int j, int first) {
        offsets[j] = first;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
          const int c = cnt[w][j];
          cnt[w][j] = first;
          first += c;
        }
      });
  if (tid == 0) offsets[E] = valid;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int i = lo + 64 * k + lane;
    if (k >= steps || i >= S) continue;
    const bool ok = e[k] >= 0 && e[k] < E;
    const int row = ok ? cnt[wave][e[k]] + rank[k] : -1;
    slot_row[i] = row;
    if (ok) row_slot[row] = i;
  }
  for (int r = valid + tid; r < S; r += kSortThreads) row_slot[r] = -1;
}

// More slots, first launch: each slot's rank among its wave's, kept in slot_row,
// and the counts of the workgroup, hist[block][E], and of its waves.
__global__ __launch_bounds__(kSortThreads) void k_sort_rank(const int32_t* __restrict__ ids, int S, int E, int tile,
                                                            int32_t* __restrict__ hist, int32_t* __restrict__ whist,
                                                            int32_t* __restrict__ slot_row,
                                                            int32_t* __restrict__ dev_error) {
  __shared__ int cnt[kSortWaves][kMaxE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int j = tid; j < E; j += kSortThreads)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) cnt[w][j] = 0;
  const int share = tile / kSortWaves;
  const int lo = blockIdx.x * tile + wave * share, hi = min(S, lo + share);
  __syncthreads();
  bool bad = false;
  for (int i0 = lo; i0 < hi; i0 += 64) {
    const int i = i0 + lane;
    const int e = i < hi ? ids[i] : -1;
    const bool ok = e >= 0 && e < E;
    bad |= !ok && i < hi;
    const int rank = rank_step(e, ok, E, lane, cnt[wave]);
    if (i < hi) slot_row[i] = rank;
  }
  if (bad && dev_error) atomicOr(dev_error, 1);
  __syncthreads();
  for (int j = tid; j < E; j += kSortThreads) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      whist[((size_t)blockIdx.x * kSortWaves + w) * E + j] = c;   // of the waves before
      c += cnt[w][j];
    }
    hist[blockIdx.x * E + j] = c;
  }
}

// Second launch: first rows from all workgroups' counts, then each slot's row.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const int32_t* __restrict__ ids, int S, int E, int tile,
                                                             const int32_t* __restrict__ hist,
                                                             const int32_t* __restrict__ whist,
                                                             int32_t* __restrict__ offsets,
                                                             int32_t* __restrict__ slot_row,
                                                             int32_t* __restrict__ row_slot) {
  __shared__ int total[kMaxE], before[kMaxE], wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int j = tid; j < E; j += kSortThreads) total[j] = before[j] = 0;
  __syncthreads();
  // threads side by side take neighbouring experts, groups of them every few workgroups
  int width = 1;
  while (width < E && width < kSortThreads) width <<= 1;
  const int part = tid / width, parts = kSortThreads / width, blocks = gridDim.x;
  for (int j = tid & (width - 1); j < E; j += width) {
    int all = 0, mine = 0;
    for (int b = part; b < blocks; b += parts) {
      const int c = hist[(size_t)b * E + j];
      all += c;
      mine += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&total[j], all);
    atomicAdd(&before[j], mine);
  }
  __syncthreads();
  const int valid = scan_experts(E, wsum, [&](int j) { return total[j]; },
                                 [&](int j, int first) {
                                   if (blockIdx.x == 0) offsets[j] = first;
                                   before[j] += first;
                                 });
  if (blockIdx.x == 0 && tid == 0) offsets[E] = valid;
  __syncthreads();
  const int share = tile / kSortWaves;
  const int lo = blockIdx.x * tile + wave * share, hi = min(S, lo + share);
  const int32_t* wh = whist + ((size_t)blockIdx.x * kSortWaves + wave) * E;
  for (int i = lo + lane; i < hi; i += 64) {
    const int e = ids[i];
    const bool ok = e >= 0 && e < E;
    const int row = ok ? before[e] + wh[e] + slot_row[i] : -1;
    slot_row[i] = row;
    if (ok) row_slot[row] = i;
  }
  for (int r = valid + blockIdx.x * kSortThreads + tid; r < S; r += gridDim.x * kSortThreads) row_slot[r] = -1;
}

__global__ void k_sort_empty(int E, int32_t* __restrict__ offsets) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// xs[slot_row[t, s]] = x[t]: a thread carries 16 bytes of one token's row to
// its top_k places, so x is read once.  Bound by HBM, the stores: 4096 x 2048 bf16 to eight
// places each 29 us, 5.2 TB/s, a large copy's rate (23.5 us into a tensor that the last-level cache
// still holds).
__global__ __launch_bounds__(256) void k_gather(const uint4* __restrict__ x, int pieces, int M, int top_k,
                                                const int32_t* __restrict__ slot_row, uint4* __restrict__ xs) {
  const int c = (int)blockIdx.y * 256 + (int)threadIdx.x, n_rows = M * top_k;
  if (c >= pieces) return;
  for (long long t = blockIdx.x; t < M; t += gridDim.x) {
    const uint4 v = x[t * pieces + c];
    for (int s0 = 0; s0 < top_k; s0 += 8) {
      int row[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) row[s] = s0 + s < top_k ? slot_row[t * top_k + s0 + s] : -1;
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if ((unsigned)row[s] < (unsigned)n_rows) xs[(long long)row[s] * pieces + c] = v;
    }
  }
}

// y[t] = sum_s p[t, s] ys[slot_row[t, s]] in fp32, in the order of s; eight slots' rows
// are in flight at a time.  Bound by the rows' reads from HBM: 4096 x 2048 bf16, eight slots, 30 us,
// 5.1 TB/s (23 us where the last-level cache holds the rows; an expert call's fp32 rows, just written,
// 46 us, 6.1 TB/s).
template <typename T_IN, typename T, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const T_IN* __restrict__ ys, int H, int M, int top_k,
                                                 const int32_t* __restrict__ slot_row, const float* __restrict__ p,
                                                 T* __restrict__ y) {
  constexpr int AHEAD = 8;
  const int c = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 8, n_rows = M * top_k;
  if (c >= H) return;
  for (long long t = blockIdx.x; t < M; t += gridDim.x) {
    float a[8] = {};
    for (int s0 = 0; s0 < top_k; s0 += AHEAD) {
      int row[AHEAD];
      float w[AHEAD], v[AHEAD][8];
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const bool in = s0 + s < top_k;
        row[s] = in ? slot_row[t * top_k + s0 + s] : -1;
        w[s] = WEIGHTED && in ? p[t * top_k + s0 + s] : 1.0f;
        if ((unsigned)row[s] >= (unsigned)n_rows) row[s] = -1;
      }
#pragma unroll
      for (int s = 0; s < AHEAD; ++s)
        if (row[s] >= 0) load8(ys + (long long)row[s] * H + c, v[s]);
#pragma unroll
      for (int s = 0; s < AHEAD; ++s)
        if (row[s] >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = WEIGHTED ? fmaf(w[s], v[s][i], a[i]) : a[i] + v[s][i];
        }
    }
    store8(y + t * H + c, a);
  }
}

// One wave per slot: dys[row] = p dy[t], dp = <dy[t], ys[row]>, so a token's dy is
// read once a slot, from the caches after the first.  Bound by HBM: 4096 x 2048 bf16,
// eight slots, 57 us, 5.0 TB/s (50 us on the same rows again).
template <typename T>
__global__ __launch_bounds__(256) void k_combine_backward(const T* __restrict__ dy, const T* __restrict__ ys, int H,
                                                          int S, int top_k, const int32_t* __restrict__ slot_row,
                                                          const float* __restrict__ p, T* __restrict__ dys,
                                                          float* __restrict__ dp) {
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  if (i >= S) return;
  const int r = slot_row[i];
  float dot = 0.0f;
  if (r >= 0 && r < S) {
    const float w = p[i];
    const T* d = dy + (long long)(i / top_k) * H;
    const T* v = ys + (long long)r * H;
    T* o = dys + (long long)r * H;
    for (int c = lane * 8; c < H; c += 512) {
      float a[8], b[8];
      load8(d + c, a);
      load8(v + c, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dot = fmaf(a[j], b[j], dot);
        a[j] *= w;
      }
      store8(o + c, a);
    }
  }
  dot = wave_sum_f32(dot);
  if (lane == 0) dp[i] = dot;
}

// Workgroups of 256 threads over (token, 256 pieces of its row).  A grid holds
// fewer than 2^32 threads, so tokens past 2^18 are taken in turn.
dim3 token_grid(int M, int pieces) {
  return dim3((unsigned)(M < (1 << 18) ? M : (1 << 18)), (unsigned)((pieces + 255) / 256));
}

template <typename T_IN, typename T, bool WEIGHTED>
void combine(const void* ys, int M, int top_k, int H, const int32_t* slot_row, const float* p, void* y,
             hipStream_t stream) {
  hipLaunchKernelGGL((k_combine<T_IN, T, WEIGHTED>), token_grid(M, H / 8), dim3(256), 0, stream,
                     static_cast<const T_IN*>(ys), H, M, top_k, slot_row, p, static_cast<T*>(y));
}

template <bool WEIGHTED>
void combine_type(const void* ys, int type, int M, int top_k, int H, const int32_t* slot_row, const float* p, void* y,
                  hipStream_t stream) {
  if (type == 0) combine<_Float16, _Float16, WEIGHTED>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 1) combine<__bf16, __bf16, WEIGHTED>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 2) combine<float, float, WEIGHTED>(ys, M, top_k, H, slot_row, p, y, stream);
}

template <typename T>
void combine_backward(const void* dy, const void* ys, int M, int top_k, int H, const int32_t* slot_row, const float* p,
                      void* dys, float* dp, hipStream_t stream) {
  const int S = M * top_k;
  hipLaunchKernelGGL(k_combine_backward<T>, dim3((unsigned)((S + 3) / 4)), dim3(256), 0, stream,
                     static_cast<const T*>(dy), static_cast<const T*>(ys), H, S, top_k, slot_row, p,
                     static_cast<T*>(dys), dp);
}

}  // namespace

// The workgroups' histograms, by a bound on their number that does not fall as slots are added:
// past 262144 slots a workgroup takes more of them, and then there are fewer than 256.
size_t moe_sort_workspace_bytes(int S, int E) {
  if (S <= kOneBlockSlots) return 0;
  const int b = (S + 1023) / 1024;
  return (size_t)(b < kSortMaxBlocks ? b : kSortMaxBlocks) * (1 + kSortWaves) * E * sizeof(int32_t);
}

hipError_t launch_moe_sort(const int32_t* ids, int S, int E, int32_t* offsets, int32_t* slot_row, int32_t* row_slot,
                           void* ws, int32_t* dev_error, hipStream_t stream) {
  const int b = sort_blocks(S), tile = sort_tile(S);
  if (b == 0) {
    hipLaunchKernelGGL(k_sort_empty, dim3(1), dim3(256), 0, stream, E, offsets);
  } else if (b == 1) {
    hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kSortThreads), 0, stream, ids, S, E, tile, offsets, slot_row,
                       row_slot, dev_error);
  } else {
    int32_t* hist = static_cast<int32_t*>(ws);
    int32_t* whist = hist + (size_t)b * E;
    hipLaunchKernelGGL(k_sort_rank, dim3(b), dim3(kSortThreads), 0, stream, ids, S, E, tile, hist, whist, slot_row,
                       dev_error);
    hipLaunchKernelGGL(k_sort_place, dim3(b), dim3(kSortThreads), 0, stream, ids, S, E, tile, hist, whist, offsets,
                       slot_row, row_slot);
  }
  return hipGetLastError();
}

hipError_t launch_moe_gather(const void* x, int row_bytes, int M, int top_k, const int32_t* slot_row, void* xs,
                             hipStream_t stream) {
  const int pieces = row_bytes / 16;
  hipLaunchKernelGGL(k_gather, token_grid(M, pieces), dim3(256), 0, stream, static_cast<const uint4*>(x), pieces, M,
                     top_k, slot_row, static_cast<uint4*>(xs));
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* ys, int type, int M, int top_k, int H, const int32_t* slot_row,
                              const float* p, void* y, hipStream_t stream) {
  if (p)
    combine_type<true>(ys, type, M, top_k, H, slot_row, p, y, stream);
  else
    combine_type<false>(ys, type, M, top_k, H, slot_row, p, y, stream);
  return hipGetLastError();
}

hipError_t launch_moe_combine_rows(const float* ys, int type, int M, int top_k, int H, const int32_t* slot_row,
                                   const float* p, void* y, hipStream_t stream) {
  if (type == 0) combine<float, _Float16, true>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 1) combine<float, __bf16, true>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 2) combine<float, float, true>(ys, M, top_k, H, slot_row, p, y, stream);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* dy, const void* ys, int type, int M, int top_k, int H,
                                       const int32_t* slot_row, const float* p, void* dys, float* dp,
                                       hipStream_t stream) {
  if (type == 0) combine_backward<_Float16>(dy, ys, M, top_k, H, slot_row, p, dys, dp, stream);
  if (type == 1) combine_backward<__bf16>(dy, ys, M, top_k, H, slot_row, p, dys, dp, stream);
  if (type == 2) combine_backward<float>(dy, ys, M, top_k, H, slot_row, p, dys, dp, stream);
  return hipGetLastError();
}

}  // namespace zinc
