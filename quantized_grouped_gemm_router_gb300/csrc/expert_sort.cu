// moe_sort_tokens: assignments sorted by expert, stably, without atomics on global memory.
//
// A counting sort with E + 1 bins (the last one for assignments without an expert): the place of
// assignment a is (all of lower bins) + (those of its bin in earlier chunks, in earlier warps of its
// chunk, in lower lanes of its warp's step, or in earlier steps). Up to kSortSingle assignments are one
// CTA's chunk. Above, one launch counts every chunk's bins and a second one places them: each of its CTAs
// counts its own chunk per warp while the first launch still runs, then adds up all chunks' counts itself
// (chunks * (E + 1) integers out of L2), so that nothing waits for a scan by a single CTA. Bound by launches and dependent
// round trips: 64 assignments of 256 experts take 3.1 us, 4096 7.2, 131064 10.3 (16.9 with per-warp histograms in the first
// launch and eight loads in flight in the second).
#include "expert_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBatch = 4;            // steps whose ids are loaded together
constexpr int kSortSingle = 1024;    // assignments that one CTA sorts alone: 4096 take 10.3 us so, 7 by two launches

__device__ __forceinline__ int bin_of(const SortParams& p, int a, bool valid, bool* bad) {
  const int id = valid ? __ldg(p.ids + a) : -1;
  *bad |= id >= p.n_experts;
  return id < 0 || id >= p.n_experts ? p.n_experts : id;
}

// The warp's run of the chunk: [begin, end).
struct Run {
  int begin, end;
};
__device__ __forceinline__ Run warp_run(const SortParams& p, int c, int warp, int warps) {
  const int begin = c * p.chunk, end = min(p.n, begin + p.chunk);
  const int per = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
  const int b = min(end, begin + warp * per);
  return {b, min(end, b + per)};
}

// Adds the bins of a warp's run to run[0 .. n_experts]: the lowest lane of each bin's peers adds their number.
__device__ __forceinline__ void count_run(const SortParams& p, Run r, int* run, bool* bad) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  for (int b = r.begin; b < r.end; b += 32 * kBatch) {
    int e[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) e[i] = bin_of(p, b + 32 * i + lane, b + 32 * i + lane < r.end, bad);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b + 32 * i >= r.end) break;
      const bool valid = b + 32 * i + lane < r.end;
      const unsigned peers = __match_any_sync(~0u, valid ? e[i] : -1 - lane);
      if (valid && (peers & below) == 0u) run[e[i]] += __popc(peers);
      __syncwarp();
    }
  }
}

// A chunk's bins, in any order: one histogram by atomics in shared memory.
__global__ void __launch_bounds__(kThreads) sort_count_kernel(const SortParams p) {
  __shared__ int s_bins[kMaxExperts + 1];
  const int bins = p.n_experts + 1;
  for (int i = threadIdx.x; i < bins; i += kThreads) s_bins[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();  // the ids are complete: the placing kernel may read them at once
  const int begin = blockIdx.x * p.chunk, end = min(p.n, begin + p.chunk);
  bool bad = false;
  for (int a = begin + threadIdx.x; a < end; a += kThreads) atomicAdd(&s_bins[bin_of(p, a, true, &bad)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kThreads) p.counts[(size_t)blockIdx.x * bins + e] = s_bins[e];
}

// SINGLE: one chunk, no counts of others.
template <bool SINGLE>
__global__ void __launch_bounds__(kThreads) sort_place_kernel(const SortParams p, int warps) {
  extern __shared__ int smem[];  // base[bins], total[bins], run[warps][bins]
  __shared__ int s_scan[kWarps];
  const int bins = p.n_experts + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  int *base = smem, *total = smem + bins, *runs = smem + 2 * bins, *run = runs + warp * bins;
  for (int i = tid; i < (2 + warps) * bins; i += kThreads) smem[i] = 0;
  __syncthreads();
  if (SINGLE) {
    pdl_wait();
    pdl_launch_dependents();
  }
  bool bad = false;
  const Run r = warp < warps ? warp_run(p, blockIdx.x, warp, warps) : Run{0, 0};
  if (warp < warps) count_run(p, r, run, &bad);
  if (__any_sync(~0u, bad) && lane == 0) raise_index(p.hdr);
  if (!SINGLE) {
    pdl_wait();
    pdl_launch_dependents();
    // groups of threads add up every groups-th chunk for a bin each: base the earlier chunks, total all
    const int groups = bins < kThreads ? kThreads / bins : 1;
    for (int i = tid; i < groups * bins; i += kThreads) {
      const int g = i / bins, e = i - g * bins;
      int before = 0, all = 0;
      for (int c0 = g; c0 < p.chunks; c0 += 16 * groups) {
        int v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          v[u] = c0 + u * groups < p.chunks ? __ldcg(p.counts + (size_t)(c0 + u * groups) * bins + e) : 0;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          all += v[u];
          if (c0 + u * groups < (int)blockIdx.x) before += v[u];
        }
      }
      if (all) atomicAdd(&total[e], all);  // integers in shared memory: any order gives the same
      if (before) atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  if (SINGLE) {
    for (int e = tid; e < bins; e += kThreads) {
      int n = 0;
#pragma unroll 8
      for (int w = 0; w < warps; ++w) n += runs[w * bins + e];
      total[e] = n;
    }
    __syncthreads();
  }
  // exclusive scan of the experts' totals, one expert to a thread
  const int mine = tid < p.n_experts ? total[tid] : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int sums = s_scan[lane];  // the warps' totals: every warp scans them for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, sums, o);
    if (lane >= o) sums += v;
  }
  const int before = warp ? __shfl_sync(~0u, sums, warp - 1) : 0;
  const int offset = before + incl - mine;
  if (tid < p.n_experts) base[tid] += offset;
  if (blockIdx.x == 0 && tid < p.n_experts) p.offsets[tid] = offset;
  if (tid == p.n_experts - 1) {
    base[p.n_experts] += offset + mine;
    if (blockIdx.x == 0) p.offsets[p.n_experts] = offset + mine;
  }
  __syncthreads();
  for (int e = tid; e < bins; e += kThreads) {
    int at = base[e];
    for (int w0 = 0; w0 < warps; w0 += 8) {
      int n[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) n[w] = w0 + w < warps ? runs[(w0 + w) * bins + e] : 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w0 + w < warps) runs[(w0 + w) * bins + e] = at;
        at += n[w];
      }
    }
  }
  __syncthreads();
  const unsigned below = (1u << lane) - 1u;
  for (int b = r.begin; b < r.end; b += 32 * kBatch) {
    int e[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) e[i] = bin_of(p, b + 32 * i + lane, b + 32 * i + lane < r.end, &bad);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int a = b + 32 * i + lane;
      if (a - lane >= r.end) break;
      const bool valid = a < r.end;
      const unsigned peers = __match_any_sync(~0u, valid ? e[i] : -1 - lane);
      if (valid) {
        const int at = run[e[i]] + __popc(peers & below);
        const bool placed = e[i] < p.n_experts;
        p.perm[at] = placed ? a : -1;
        p.inv[a] = placed ? at : -1;
      }
      __syncwarp();
      if (valid && (peers & below) == 0u) run[e[i]] += __popc(peers);
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_sort_tokens(SortParams p, cudaStream_t s) {
  constexpr int kMostBins = kMaxExperts + 1;
  static const cudaError_t attr = [] {
    const int all = (int)((2 + kWarps) * kMostBins * sizeof(int));
    cudaError_t e = cudaFuncSetAttribute(sort_place_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, all);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_place_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, all);
    return e;
  }();
  if (attr != cudaSuccess) return attr;
  const int bins = p.n_experts + 1;
  if (p.n <= kSortSingle) {
    p.chunk = kSortSingle;
    p.chunks = 1;
    const int warps = p.n < 32 ? 1 : (p.n + 31) / 32 < kWarps ? (p.n + 31) / 32 : kWarps;
    return launch_pdl(sort_place_kernel<true>, 1, kThreads, (2 + warps) * bins * sizeof(int), 1, s, p, warps);
  }
  const int most = sm_count() < kSortMaxChunks ? sm_count() : kSortMaxChunks;
  const int per = (p.n + most - 1) / most;
  p.chunk = per < kThreads ? kThreads : (per + 31) / 32 * 32;
  p.chunks = (p.n + p.chunk - 1) / p.chunk;
  cudaError_t e = launch_pdl(sort_count_kernel, p.chunks, kThreads, 0, 1, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(sort_place_kernel<false>, p.chunks, kThreads, (2 + kWarps) * bins * sizeof(int), 1, s, p, kWarps);
}

}  // namespace moe
