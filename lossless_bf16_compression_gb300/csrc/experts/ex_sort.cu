// ex_sort.cu -- the place of each slot in the order by expert (a stable counting sort).
//
// position[s] = #{s' : key(s') < key(s)} + #{s' < s : key(s') = key(s)}, with key(s) the slot's
// expert, or `experts` for a slot without one.  Each CTA takes a contiguous run of slots: a first
// kernel counts the keys of every run, a second turns the counts into starts (a run's key starts
// after all smaller keys and after the same key in the runs before it) and walks the run again,
// 32 slots of a warp at a time, giving a slot its key's start plus the number of equal keys before it
// in the warp.  A call of one run needs only the second kernel.  Bound by latency: two launches
// and a few dependent loads: 16384 x 8 slots of 64 experts 9.6 us, 64 x 8 4.2 us.
#include "ex_common.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kSortWarps = 16;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr size_t kRunSlots = 1024;  // slots of a run, while there are at most kMaxRuns
constexpr size_t kMaxRuns = 128;    // every CTA of the second kernel reads every run's counts

// Dynamic shared memory that needs no asking: 48 KB less what the kernel has itself.
constexpr size_t kPlainShared = 48 * 1024 - 1024;

size_t runs_of(size_t slots) {
  const size_t r = (slots + kRunSlots - 1) / kRunSlots;
  return r < 1 ? 1 : r > kMaxRuns ? kMaxRuns : r;
}

template <typename Id>
__device__ __forceinline__ int key_of(const Id* ids, size_t s, int experts) {
  const Id v = ids[s];
  return v >= 0 && v < experts ? static_cast<int>(v) : experts;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) count_kernel(const Id* ids, int slots, int run, int experts,
                                                             int* counts) {
  extern __shared__ int bins[];
  wait_for_previous();
  let_next_start();
  const int keys = experts + 1;
  const int begin = min(slots, static_cast<int>(blockIdx.x) * run), end = min(slots, begin + run);
  for (int i = threadIdx.x; i < keys; i += kSortThreads) bins[i] = 0;
  __syncthreads();
  for (int s = begin + threadIdx.x; s < end; s += kSortThreads) atomicAdd(&bins[key_of(ids, s, experts)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < keys; i += kSortThreads) counts[static_cast<size_t>(blockIdx.x) * keys + i] = bins[i];
}

// counts: [runs][experts + 1] from count_kernel; not read when there is one run.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads) place_kernel(const Id* ids, int slots, int run, int runs,
                                                             int experts, const int* counts, int* position,
                                                             int* offsets) {
  extern __shared__ int bins[];  // [kSortWarps][experts + 1]
  __shared__ int warp_sums[kSortWarps];
  __shared__ int carry;
  if (runs == 1) wait_for_previous();  // else the ids are there: count_kernel started after them
  const int keys = experts + 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int first = min(slots, static_cast<int>(blockIdx.x) * run), last = min(slots, first + run);
  const int part = (last - first + kSortWarps - 1) / kSortWarps;
  const int begin = min(last, first + warp * part), end = min(last, begin + part);
  int* mine = bins + warp * keys;
  for (int i = threadIdx.x; i < kSortWarps * keys; i += kSortThreads) bins[i] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int s = begin + lane; s < end; s += 32) atomicAdd(&mine[key_of(ids, s, experts)], 1);
  if (runs > 1) wait_for_previous();
  let_next_start();  // not before the wait: what starts after this kernel reads x without one
  __syncthreads();
  for (int base = 0; base < keys; base += kSortThreads) {
    const int e = base + threadIdx.x;
    int total = 0, before = 0;  // of this key: in all the runs, and in the runs before this one
    if (e < keys) {
      if (runs > 1) {
        for (int r = 0; r < runs; ++r) {
          const int c = counts[static_cast<size_t>(r) * keys + e];
          total += c;
          if (r < static_cast<int>(blockIdx.x)) before += c;
        }
      } else {
        for (int w = 0; w < kSortWarps; ++w) total += bins[w * keys + e];
      }
    }
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
      if (blockIdx.x == 0) offsets[e] = start;
      start += before;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = bins[w * keys + e];
        bins[w * keys + e] = start;
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
      const int ahead = __popc(same & ((1u << lane) - 1));
      const int start = mine[key];
      __syncwarp(live);
      if (ahead == 0) mine[key] = start + __popc(same);
      position[s] = start + ahead;
    }
    __syncwarp();
  }
}

}  // namespace

size_t sort_workspace(size_t slots, int experts) {
  const size_t r = runs_of(slots);
  return r > 1 ? 4 * r * (static_cast<size_t>(experts) + 1) : 0;
}

cudaError_t launch_sort(const void* ids, int id_bytes, size_t slots, int experts, int* position, int* offsets,
                        void* workspace, cudaStream_t stream) {
  const int runs = static_cast<int>(runs_of(slots)), run = static_cast<int>((slots + runs - 1) / runs);
  const int n = static_cast<int>(slots);
  int* counts = static_cast<int*>(workspace);
  const size_t row = sizeof(int) * (experts + 1);
  const auto go = [&](auto* p) {
    using Id = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
    cudaError_t err = cudaSuccess;
    if (kSortWarps * row > kPlainShared)
      err = allow_shared_memory<place_kernel<Id>>(kSortWarps * sizeof(int) * (ZC_MOE_MAX_EXPERTS + 1));
    if (err == cudaSuccess && runs > 1)
      err = launch(ZC_KERNEL_MOE_SORT, count_kernel<Id>, runs, kSortThreads, row, stream, p, n, run, experts, counts);
    if (err == cudaSuccess)
      err = launch(ZC_KERNEL_MOE_SORT, place_kernel<Id>, runs, kSortThreads, kSortWarps * row, stream, p, n, run, runs,
                   experts, counts, position, offsets);
    return err;
  };
  return id_bytes == 8 ? go(static_cast<const long long*>(ids)) : go(static_cast<const int*>(ids));
}

}  // namespace ex
}  // namespace zc
