// ex_sort.cu -- the place of each slot in the order by expert (a stable counting sort).
//
// position[s] = #{s' : key(s') < key(s)} + #{s' < s : key(s') = key(s)}, with key(s) the slot's
// expert, or `experts` for a slot without one.  One CTA: each warp counts the keys of its own
// contiguous run of slots, a scan over (key, warp) turns the counts into starts, and each warp
// walks its run again, 32 slots at a time, giving a slot its key's start plus the number of
// equal keys before it in the warp.
#include "ex_common.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kSortWarps = 16;
constexpr int kSortThreads = 32 * kSortWarps;

template <typename Id>
__device__ __forceinline__ int key_of(const Id* ids, size_t s, int experts) {
  const Id v = ids[s];
  return v >= 0 && v < experts ? static_cast<int>(v) : experts;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const Id* __restrict__ ids, int slots, int experts,
                                                            int* __restrict__ position, int* __restrict__ offsets) {
  extern __shared__ int counts[];  // [kSortWarps][experts + 1]
  __shared__ int warp_sums[kSortWarps];
  __shared__ int carry;
  const int keys = experts + 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int run = (slots + kSortWarps - 1) / kSortWarps;
  const int begin = min(slots, warp * run), end = min(slots, begin + run);
  int* mine = counts + warp * keys;
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) counts[i] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int s = begin + lane; s < end; s += 32) atomicAdd(&mine[key_of(ids, s, experts)], 1);
  __syncthreads();
  // exclusive scan over the keys, and over the warps within a key
  for (int base = 0; base < keys; base += kSortThreads) {
    const int e = base + threadIdx.x;
    int total = 0;
    if (e < keys)
      for (int w = 0; w < kSortWarps; ++w) total += counts[w * keys + e];
    int incl = total;
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int start = carry + incl - total;
    for (int w = 0; w < warp; ++w) start += warp_sums[w];
    __syncthreads();
    if (threadIdx.x == kSortThreads - 1) carry = start + total;
    if (e < keys) {
      offsets[e] = start;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = counts[w * keys + e];
        counts[w * keys + e] = start;
        start += c;
      }
    }
    __syncthreads();
  }
  for (int s0 = begin; s0 < end; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < end;
    const unsigned live = __ballot_sync(~0u, in);
    if (in) {
      const int key = key_of(ids, s, experts);
      const unsigned same = __match_any_sync(live, key);
      const int before = __popc(same & ((1u << lane) - 1));
      const int start = mine[key];
      __syncwarp(live);
      if (before == 0) mine[key] = start + __popc(same);
      position[s] = start + before;
    }
    __syncwarp();
  }
}

}  // namespace

size_t sort_workspace(size_t, int) { return 16; }

cudaError_t launch_sort(const void* ids, int id_bytes, size_t slots, int experts, int* position, int* offsets, void*,
                        cudaStream_t stream) {
  const size_t smem = sizeof(int) * kSortWarps * (experts + 1);
  const auto run = [&](auto kernel, auto* p) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 sizeof(int) * kSortWarps * (ZC_MOE_MAX_EXPERTS + 1));
    if (err != cudaSuccess) return err;
    return launch(kernel, 1, kSortThreads, smem, stream, false, p, static_cast<int>(slots), experts, position, offsets);
  };
  return id_bytes == 8 ? run(sort_kernel<long long>, static_cast<const long long*>(ids))
                       : run(sort_kernel<int>, static_cast<const int*>(ids));
}

}  // namespace ex
}  // namespace zc
