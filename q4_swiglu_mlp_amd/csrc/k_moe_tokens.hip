// An MoE layer's token permutation: the sort of routed slots by expert, the
// gather of token rows into that order, the weighted way back, and gradients.
//
// The sort is a stable counting sort: slot i = t * top_k + s goes behind every
// slot of a smaller expert and behind the earlier slots of its own, so the
// order, and with it every later sum, is a function of the ids alone (no
// atomic decides a place).
#include "fp8_device.hpp"
#include "launch.hpp"

namespace zinc {
namespace {

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int kMaxE = 1024;
constexpr int kSortMaxBlocks = 256;

// Slots per workgroup: at least 4096 (a smaller sort is one workgroup and one
// launch), and at most 256 workgroups.  A multiple of 512, so that every
// wave's share is whole steps of 64.
int sort_tile(int S) {
  const int t = (S + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return ((t < 4096 ? 4096 : t) + kSortThreads - 1) / kSortThreads * kSortThreads;
}
int sort_blocks(int S) { return S > 0 ? (S + sort_tile(S) - 1) / sort_tile(S) : 0; }

// Per-workgroup counts of each expert's slots.
__global__ __launch_bounds__(kSortThreads) void k_sort_hist(const int32_t* __restrict__ ids, int S, int E, int tile,
                                                            int32_t* __restrict__ hist) {
  __shared__ int cnt[kMaxE];
  for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * tile, hi = min(S, lo + tile);
  for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[blockIdx.x * E + e] = cnt[e];
}

// Each wave counts its contiguous share of the workgroup's slots; the counts
// become the first row of every (wave, expert); then the wave walks its share
// 64 slots at a time, a lane's place being its expert's next row plus the
// number of lower lanes with the same expert (ballots over the bits of the id).
__global__ __launch_bounds__(kSortThreads) void k_sort(const int32_t* __restrict__ ids, int S, int E, int tile,
                                                       const int32_t* __restrict__ hist, int32_t* __restrict__ offsets,
                                                       int32_t* __restrict__ slot_row, int32_t* __restrict__ row_slot,
                                                       int32_t* __restrict__ dev_error) {
  __shared__ int next[kSortWaves][kMaxE];
  __shared__ int total[kMaxE], before[kMaxE], wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < E; e += kSortThreads) {
    total[e] = 0;
    before[e] = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) next[w][e] = 0;
  }
  __syncthreads();
  const int share = tile / kSortWaves;
  const int lo = blockIdx.x * tile + wave * share, hi = min(S, lo + share);
  bool bad = false;
  for (int i = lo + lane; i < hi; i += 64) {
    const int e = ids[i];
    if (e >= 0 && e < E)
      atomicAdd(&next[wave][e], 1);
    else
      bad = true;
  }
  if (bad && dev_error) atomicOr(dev_error, 1);
  // all workgroups' counts, and those of the workgroups before this one
  if (hist) {
    for (int j = tid; j < E * (int)gridDim.x; j += kSortThreads) {
      const int b = j / E, e = j - b * E, c = hist[j];
      if (c) {
        atomicAdd(&total[e], c);
        if (b < (int)blockIdx.x) atomicAdd(&before[e], c);
      }
    }
  }
  __syncthreads();
  // exclusive scan over the experts, two a thread
  int t0 = 0, t1 = 0;
  const int e0 = 2 * tid, e1 = e0 + 1;
  auto count = [&](int e) {
    if (e >= E) return 0;
    if (hist) return total[e];
    int c = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c += next[w][e];
    return c;
  };
  t0 = count(e0);
  t1 = count(e1);
  int scan = t0 + t1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(scan, d, 64);
    if (lane >= d) scan += o;
  }
  if (lane == 63) wsum[wave] = scan;
  __syncthreads();
  int base = scan - t0 - t1, valid = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) base += wsum[w];
    valid += wsum[w];
  }
  auto place = [&](int e, int first) {
    if (e >= E) return;
    if (blockIdx.x == 0) offsets[e] = first;
    int at = first + before[e];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = next[w][e];
      next[w][e] = at;
      at += c;
    }
  };
  place(e0, base);
  place(e1, base + t0);
  if (blockIdx.x == 0 && tid == 0) offsets[E] = valid;
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 64) {
    const int i = i0 + lane;
    const int e = i < hi ? ids[i] : -1;
    const bool ok = e >= 0 && e < E;
    uint64_t same = __ballot(ok);
    for (int bit = 1; bit < E; bit <<= 1) {
      const uint64_t m = __ballot((e & bit) != 0);
      same &= (e & bit) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (ok) row = next[wave][e] + rank;
    __builtin_amdgcn_wave_barrier();
    if (ok && rank == 0) next[wave][e] = row + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < hi) slot_row[i] = row;
    if (ok) row_slot[row] = i;
  }
  for (int r = valid + blockIdx.x * kSortThreads + tid; r < S; r += gridDim.x * kSortThreads) row_slot[r] = -1;
}

__global__ void k_sort_empty(int E, int32_t* __restrict__ offsets) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// xs[slot_row[t, s]] = x[t]: a thread carries 16 bytes of one token's row to
// its top_k places, so x is read once.
__global__ __launch_bounds__(256) void k_gather(const uint4* __restrict__ x, int pieces, int M, int top_k,
                                                const int32_t* __restrict__ slot_row, uint4* __restrict__ xs) {
  const int c = (int)blockIdx.y * 256 + (int)threadIdx.x, n_rows = M * top_k;
  if (c >= pieces) return;
  for (long long t = blockIdx.x; t < M; t += gridDim.x) {
    const uint4 v = x[t * pieces + c];
    for (int s = 0; s < top_k; ++s) {
      const int r = slot_row[t * top_k + s];
      if (r >= 0 && r < n_rows) xs[(long long)r * pieces + c] = v;
    }
  }
}

// y[t] = sum_s p[t, s] ys[slot_row[t, s]] in fp32, in the order of s.
template <typename T, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const T* __restrict__ ys, int H, int M, int top_k,
                                                 const int32_t* __restrict__ slot_row, const float* __restrict__ p,
                                                 T* __restrict__ y) {
  const int c = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 8, n_rows = M * top_k;
  if (c >= H) return;
  for (long long t = blockIdx.x; t < M; t += gridDim.x) {
    float a[8] = {};
    for (int s = 0; s < top_k; ++s) {
      const int r = slot_row[t * top_k + s];
      if (r < 0 || r >= n_rows) continue;
      float v[8];
      load8(ys + (long long)r * H + c, v);
      const float w = WEIGHTED ? p[t * top_k + s] : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = WEIGHTED ? fmaf(w, v[i], a[i]) : a[i] + v[i];
    }
    store8(y + t * H + c, a);
  }
}

// One wave per slot: dys[row] = p dy[t], dp = <dy[t], ys[row]>.
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

template <typename T>
void combine(const void* ys, int M, int top_k, int H, const int32_t* slot_row, const float* p, void* y,
             hipStream_t stream) {
  const dim3 grid = token_grid(M, H / 8);
  if (p)
    hipLaunchKernelGGL((k_combine<T, true>), grid, dim3(256), 0, stream, static_cast<const T*>(ys), H, M, top_k,
                       slot_row, p, static_cast<T*>(y));
  else
    hipLaunchKernelGGL((k_combine<T, false>), grid, dim3(256), 0, stream, static_cast<const T*>(ys), H, M, top_k,
                       slot_row, p, static_cast<T*>(y));
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

size_t moe_sort_workspace_bytes(int S, int E) {
  const int b = sort_blocks(S);
  return b > 1 ? (size_t)b * E * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int S, int E, int32_t* offsets, int32_t* slot_row, int32_t* row_slot,
                           void* ws, int32_t* dev_error, hipStream_t stream) {
  const int b = sort_blocks(S), tile = sort_tile(S);
  int32_t* hist = b > 1 ? static_cast<int32_t*>(ws) : nullptr;
  if (b == 0)
    hipLaunchKernelGGL(k_sort_empty, dim3(1), dim3(256), 0, stream, E, offsets);
  if (b > 1) hipLaunchKernelGGL(k_sort_hist, dim3(b), dim3(kSortThreads), 0, stream, ids, S, E, tile, hist);
  if (b > 0)
    hipLaunchKernelGGL(k_sort, dim3(b), dim3(kSortThreads), 0, stream, ids, S, E, tile, hist, offsets, slot_row,
                       row_slot, dev_error);
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
  if (type == 0) combine<_Float16>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 1) combine<__bf16>(ys, M, top_k, H, slot_row, p, y, stream);
  if (type == 2) combine<float>(ys, M, top_k, H, slot_row, p, y, stream);
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
