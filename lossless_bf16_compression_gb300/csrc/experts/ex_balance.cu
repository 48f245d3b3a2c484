// ex_balance.cu -- the balance loss of a router, its counts and slopes.
//
// Each lane keeps the sums of its columns' probabilities in registers over all of its tokens; the warps' are added in
// shared memory in their order, the CTAs' by the first of a cluster or by a second kernel, in theirs, so nothing depends on
// timing.  The counts are whole numbers, for which order does not matter.  Bound by latency and by the exponentials: 64 x 64
// 4.3 us, 777 x 40 5.1 (a cluster; by two kernels 7.5 and by this one 6.9 while divisions and one id at a time stood in
// the way), 32768 x 64 in fp32 7.0, 16384 x 256 in bfloat16 8.6, of which the second kernel takes about 1.5 (2.5 while a
// thread asked for one part after the other).
#include "ex_router.cuh"

namespace zc {
namespace ex {
namespace {

// Rows that a warp takes at a time, so that their loads are in flight together, and warps of a CTA: what registers allow.
template <typename R>
constexpr int rows_at_once() { return R::N <= 8 ? 4 : 1; }
template <typename R>
constexpr int balance_warps() { return R::N <= 8 ? 32 : 16; }
template <typename R>
constexpr int sum_rows() { return R::N <= 8 ? balance_warps<R>() : 8; }  // in shared memory, up to 32 KB
constexpr int kIds = 4;  // of a thread, asked for together
// CTAs: at most as many as a GB300 has SMs (written down: how long the workspace is is said without a device), a cluster's.
constexpr size_t kMaxParts = 152, kCluster = 8;

struct Parts {  // of each CTA: sums, counts, tokens
  float* sums;
  int *counts, *tokens;
};
__host__ __device__ inline Parts parts_of(void* workspace, size_t ctas, size_t experts) {
  float* s = static_cast<float*>(workspace);
  int* c = reinterpret_cast<int*>(s + ctas * experts);
  return {s, c, c + ctas * experts};
}

// experts / (k n^2) as the sum of two fp32 numbers, to 2^-44 of it, and a count's multiple of it, rounded once.  (k n^2 is two
// fp32 numbers too.  A 64-bit division took the kernels 1500 cycles, and whole numbers of 64 bits, made two, up to 3000 where
// a CTA's 32 warps all did it.)
struct Unit {
  float hi, lo;
};
__device__ __forceinline__ Unit unit_of(int experts, int k, int n) {
  if (n == 0) return {0, 0};
  if (n >= 1 << 24) {  // n is no fp32 number
    const double u = experts / (static_cast<double>(k) * n * n);
    return {static_cast<float>(u), static_cast<float>(u - static_cast<float>(u))};
  }
  const float m = n, kf = k, square = m * m, h = kf * square, l = fmaf(kf, square, -h) + kf * fmaf(m, m, -square);
  const float dh = h + l, dl = l - (dh - h), hi = __fdiv_rn(experts, dh);
  return {hi, __fdiv_rn(fmaf(-hi, dl, fmaf(-hi, dh, experts)), dh)};
}
__device__ __forceinline__ float times(int c, const Unit& u) {
  const float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<int>(ch)), p = ch * u.hi;
  return p + (fmaf(ch, u.hi, -p) + fmaf(ch, u.lo, cl * u.hi));
}

// What another CTA of the cluster has in the place of `p`.
__device__ __forceinline__ uint32_t peek(const void* p, int rank) {
  uint32_t v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Few CTAs are one cluster, whose first adds their sums; more leave them to a second kernel.
template <typename R>
__global__ void __launch_bounds__(32 * balance_warps<R>())
    balance_kernel(const typename R::T* logits, size_t pitch, const int* ids, size_t tokens, size_t each, int experts, int k, int score,
                   float* loss, int* counts, float* slope, void* workspace) {
  constexpr int N = R::N, W = R::W;
  constexpr int kRows = rows_at_once<R>(), kBalanceWarps = balance_warps<R>(), kBalanceThreads = 32 * kBalanceWarps;
  constexpr int kTokens = kBalanceThreads / W;  // side by side
  constexpr int kSums = sum_rows<R>(), kColumns = N * W;
  __shared__ float sums[kSums * kColumns], losses[32];
  __shared__ int found[kColumns], live_of[32], tokens_here;
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) found[e] = 0;
  if (threadIdx.x < 32) live_of[lane] = 0;
  const size_t begin = min(tokens, blockIdx.x * each), end = min(tokens, begin + each);
  float sum[N];
  int live = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0;
  for (size_t first = begin; first < end; first += kTokens * kRows) {
    const int* chosen = ids + first * k;
    const int slots = static_cast<int>(min(end - first, static_cast<size_t>(kTokens * kRows))) * k;
    int id[kIds];
    const auto ask = [&](int s) {
#pragma unroll
      for (int i = 0; i < kIds; ++i) id[i] = s + i * kBalanceThreads < slots ? chosen[s + i * kBalanceThreads] : -1;
    };
    ask(threadIdx.x);
    R r[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const size_t t = first + threadIdx.x / W + u * kTokens;
      r[u].load(logits + t * pitch, t < end ? experts : 0);  // (behind the last: a row of nothing)
    }
    if (first == begin) __syncthreads();  // (the counts are cleared; the rows are on their way)
    for (int s = threadIdx.x;;) {
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (id[i] >= 0 && id[i] < experts) atomicAdd(&found[id[i]], 1);
      if ((s += kIds * kBalanceThreads) >= slots) break;
      ask(s);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (first + u * kTokens + warp * (32 / W) >= end) break;  // none of the warp's is left
      float p[N], top = -kInf;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = to_float(r[u].v[i]);
        top = larger(top, p[i]);
      }
      top = row_max<W>(top);
      if (W == 32 && top == -kInf) continue;
      live += top != -kInf;
      const float m = top == -kInf ? 0.0f : score == ZC_SCORE_SOFTMAX ? top : fminf(top, 0.0f);
      float total = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = score == ZC_SCORE_SOFTMAX ? expf(p[i] - m) : scaled_sigmoid(p[i], m).s;
        total += p[i];
      }
      total = row_sum<W>(total);
      const float f = total == 0 ? 0.0f : __fdividef(1.0f, total);  // (0: a row of padding)
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += p[i] * f;
    }
  }
  // The tokens of a warp.
#pragma unroll
  for (int d = W; d < 32; d *= 2) {
    live += __shfl_xor_sync(~0u, live, d);
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += __shfl_xor_sync(~0u, sum[i], d);
  }
  if (begin >= end) __syncthreads();
  if (lane == 0) live_of[warp] = live;
#pragma unroll
  for (int round = 0; round < kBalanceWarps / kSums; ++round) {
    if (warp / kSums == round) {
      float* to = sums + warp % kSums * kColumns;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = R::column(i);
        if (lane < W) to[c] = round == 0 ? sum[i] : to[c] + sum[i];
      }
    }
    __syncthreads();
  }
  // The rows of sums, by several threads for each column (row r becomes the sum of rows r, r + readers, ...).
  constexpr int kReaders = kBalanceThreads / kColumns < 8 ? kBalanceThreads / kColumns : 8, kLeft = kReaders > 1 ? kReaders : kSums;
  if constexpr (kReaders > 1) {
    if (threadIdx.x < kReaders * kColumns) {
      float s = 0;
#pragma unroll
      for (int r = 0; r < kSums; r += kReaders) s += sums[r * kColumns + threadIdx.x];
      sums[threadIdx.x] = s;
    }
    __syncthreads();
  }
  const int rows = __reduce_add_sync(~0u, live_of[lane]);
  const int ctas = gridDim.x;
  const bool together = ctas <= static_cast<int>(kCluster);
  const Parts parts = parts_of(workspace, ctas, experts);
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) {
    float s = 0;
#pragma unroll
    for (int r = 0; r < kLeft; ++r) s += sums[r * kColumns + e];
    if (together) {
      sums[e] = s;
    } else {
      parts.sums[blockIdx.x * static_cast<size_t>(experts) + e] = s;
      parts.counts[blockIdx.x * static_cast<size_t>(experts) + e] = found[e];
    }
  }
  if (!together) {
    if (threadIdx.x == 0) parts.tokens[blockIdx.x] = rows;
    return;
  }
  if (ctas > 1) {
    if (threadIdx.x == 0) tokens_here = rows;
    cluster_sync();
  }
  if (blockIdx.x == 0) {
    float mine = 0;  // of the loss
    if (warp * 32 < experts) {
      const int all = ctas == 1 ? rows : __reduce_add_sync(~0u, lane < ctas ? static_cast<int>(peek(&tokens_here, lane)) : 0);
      const Unit unit = unit_of(experts, k, all);
      for (int e = threadIdx.x; e < experts; e += kBalanceThreads) {
        float s = sums[e];
        int c = found[e];
#pragma unroll
        for (int b = 1; b < static_cast<int>(kCluster); ++b) {
          if (b < ctas) {
            s += __uint_as_float(peek(sums + e, b));
            c += static_cast<int>(peek(found + e, b));
          }
        }
        const float u = times(c, unit);
        counts[e] = c;
        slope[e] = u;
        mine += u * s;
      }
    }
    mine = row_sum<32>(mine);
    if (lane == 0) losses[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const float all = row_sum<32>(lane < kBalanceWarps ? losses[lane] : 0.0f);
      if (lane == 0) *loss = all;
    }
  }
  if (ctas > 1) cluster_sync();  // (their memory has been read)
}

// The CTAs' parts added: one cluster, each of its CTAs a share of the experts, for every expert several threads that
// read at the same time.
constexpr int kSettleThreads = 1024, kSettleCtas = 8, kAtOnce = 5;  // (parts that a thread asks for together: all, of 256 experts)
__global__ void __launch_bounds__(kSettleThreads) __cluster_dims__(kSettleCtas, 1, 1)
    settle_kernel(void* workspace, int ctas, int experts, int k, int each, float inverse, float* loss, int* counts, float* slope) {
  __shared__ float sums[kSettleThreads];
  __shared__ int totals[kSettleThreads], live[kSettleThreads / 32];
  __shared__ float losses[32];  // in the first CTA: of each CTA's first four warps
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (warp == 0) losses[lane] = 0;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // (waited for before the first CTA's memory is used)
  wait_for_previous();
  let_next_start();
  const Parts parts = parts_of(workspace, ctas, experts);
  const int rank = blockIdx.x;
  const int begin = min(experts, rank * each), end = min(experts, begin + each);
  // (Divisions by a factor: the distance of (a + 1/2) / b from a whole number is at least 1 / 2b, and a is at most 1024.)
  const auto over_each = [&](int a) { return static_cast<int>((a + 0.5f) * inverse); };
  const int readers = min(32, over_each(kSettleThreads)), reader = over_each(threadIdx.x), e = begin + threadIdx.x - reader * each;
  int n = threadIdx.x < ctas ? parts.tokens[threadIdx.x] : 0;
  float s = 0;
  int c = 0;
  if (reader < readers && e < end) {
    for (int first = reader; first < ctas; first += kAtOnce * readers) {
      float sum[kAtOnce];
      int count[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int b = first + i * readers;
        sum[i] = b < ctas ? parts.sums[static_cast<size_t>(b) * experts + e] : 0.0f;
        count[i] = b < ctas ? parts.counts[static_cast<size_t>(b) * experts + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) s += sum[i], c += count[i];
    }
  }
  n = __reduce_add_sync(~0u, n);
  sums[threadIdx.x] = s;
  totals[threadIdx.x] = c;
  if (lane == 0) live[warp] = n;
  __syncthreads();
  // The readers' sums (up to 32), to eight and then to one.
  if (threadIdx.x < 8 * each && readers > 8) {
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      const int at = threadIdx.x + i * 8 * each;
      if (at < readers * each) s += sums[at], c += totals[at];
    }
    sums[threadIdx.x] = s;
    totals[threadIdx.x] = c;
  }
  __syncthreads();
  if (threadIdx.x < (each + 31) / 32 * 32) {  // whole warps
    const Unit unit = unit_of(experts, k, __reduce_add_sync(~0u, live[lane]));
    float mine = 0;
    if (threadIdx.x < end - begin) {
#pragma unroll
      for (int r = 1; r < 8; ++r)
        if (r < readers) s += sums[r * each + threadIdx.x], c += totals[r * each + threadIdx.x];
      const float u = times(c, unit);
      counts[e] = c;
      slope[e] = u;
      mine = u * s;
    }
    mine = row_sum<32>(mine);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lane == 0) {  // into the first CTA
      const auto at = static_cast<uint32_t>(__cvta_generic_to_shared(&losses[rank * 4 + warp]));
      asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.f32 [a], %1;\n\t}" ::"r"(at),
                   "f"(mine)
                   : "memory");
    }
  } else {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && warp == 0) {
    const float all = row_sum<32>(losses[lane]);
    if (lane == 0) *loss = all;
  }
}
static_assert((ZC_MOE_MAX_EXPERTS / kSettleCtas + 31) / 32 * kSettleCtas == 32, "a place for each warp's part of the loss");

// CTAs for a call: one while its warps have two rows each at most; a cluster of eight, which needs neither a second kernel
// nor a workspace, while they have sixteen (the same on the device: 2048 x 64 7.9 and 8.1 us, but 6.9 instead of 8.5 a
// call, which the host bounds); else as many as SMs, while each warp has a row.
size_t balance_ctas(size_t tokens, int experts) {
  const size_t side = 32 * (experts <= 256 ? 32 : 16) / lanes_of(experts);  // tokens side by side in a CTA
  const size_t n = tokens <= 2 * side ? 1 : (tokens + side - 1) / side;
  if (n <= 2 * kCluster) return n < kCluster ? n : kCluster;
  return n < kMaxParts ? n : kMaxParts;
}

}  // namespace

size_t balance_workspace(size_t tokens, int experts) {
  const size_t n = balance_ctas(tokens, experts);
  return n > kCluster ? n * (2 * static_cast<size_t>(experts) + 1) * 4 : 0;
}

cudaError_t launch_balance(const RouterShape& s, const void* logits, size_t pitch, const int* ids, float* loss, int* counts,
                           float* slope, void* workspace, cudaStream_t stream) {
  const size_t ctas = balance_ctas(s.tokens, s.experts), each = (s.tokens + ctas - 1) / ctas;
  const bool together = ctas <= kCluster;
  const cudaError_t err = by_row(s.type, s.experts, true, {logits}, {pitch}, [&](auto row) {
    using R = decltype(row);
    return launch_clusters(ZC_KERNEL_MOE_BALANCE, together ? static_cast<int>(ctas) : 1, balance_kernel<R>, static_cast<unsigned>(ctas),
                           32 * balance_warps<R>(), 0, stream, static_cast<const typename R::T*>(logits), pitch, ids, s.tokens, each,
                           s.experts, s.k, s.score, loss, counts, slope, workspace);
  });
  if (err != cudaSuccess || together) return err;
  const int share = (s.experts + kSettleCtas - 1) / kSettleCtas;
  return launch(ZC_KERNEL_MOE_BALANCE, settle_kernel, kSettleCtas, kSettleThreads, 0, stream, workspace, static_cast<int>(ctas),
                s.experts, s.k, share, 1.0f / share, loss, counts, slope);
}

}  // namespace ex
}  // namespace zc
