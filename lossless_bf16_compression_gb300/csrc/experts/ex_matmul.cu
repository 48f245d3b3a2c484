// ex_matmul.cu -- the experts' products on 8-bit blocks, the weights' gradient among them.
//
// out[q, p] = sum over blocks b of 2^(sp[p, b] + sq[q, b]) sum over the block's 128 columns of
// P[p, .] Q[q, .], with P and Q rows of 8-bit values.  For matmul P is the weights of a group and
// Q the group's rows; for the weights' gradient P is x and Q is dy, both transposed, and the sum
// runs over the blocks of one group.  out is contiguous along p.
//
// GB300 design.  The tensor cores take 8-bit operands with power-of-two scales as they are
// (block-scaled products: a scale for each row and 32 columns; a block of 128 uses one scale four
// times), so nothing is ever rescaled and a tile's sum stays in tensor memory in fp32 from the
// first block to the last.  One persistent CTA an SM walks tiles of 128 rows of P by TQ rows of
// Q.  P lies along the 128 tensor-memory lanes, so a column of the accumulator is a run of 128
// consecutive outputs: the epilogue stores whole 64-byte (bf16) or 128-byte (fp32) segments
// straight from registers, with no transposition, and a ragged group's last tile only skips
// columns.  Roles: warp 0 issues the TMA loads (128 columns a stage), warp 1 the products, warp 2
// brings the scales, warps 4-7 write the results while the next tile's products run.
//
// Scales are kept four blocks to a word, [word][row]: a warp reads 128 rows' words as four
// coalesced loads and stores one 16-byte vector a lane, which is the shape the copy to tensor
// memory takes (row r at byte 16 (r % 32) + 4 (r / 32)); byte b % 4 is picked by the instruction.
#include <mutex>

#include "ex_fp8.cuh"
#include "ex_tcgen05.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kThreads = 256;
constexpr int kTileP = 128;
constexpr int kMaxTileQ = 256;
constexpr int kMaxStages = 12;
constexpr int kScaleSlots = 2;
constexpr int kSlotBytes = 512 * 3;  // P's scales, and up to two chunks of 128 rows of Q
constexpr int kColumns = 512;        // tensor memory: all of it (one CTA an SM)
constexpr int kChunk = 32;           // accumulator columns a warp reads at once
// Two accumulators of 256 columns and the scales do not fit in 512 columns: with tiles of 256 the
// second accumulator starts at column 224, and the epilogue reads the 32 columns they share first.
constexpr int kSecond = 224;

struct TileParams {
  const uint32_t *p_scales, *q_scales;  // words
  int p_fmt, q_fmt, groups, out_fp32;
  int p_rows, q_rows;         // rows of P (of one group), and of Q in all
  int blocks;                 // by_blocks: the capacity; else the blocks of a row
  int words;                  // scale words of a row
  bool by_blocks;             // the groups are runs of blocks, and out has a matrix for each
  int tile_q, stages;
  const int* offsets;         // rows (or blocks) of each group; null: one group
  void* out;
  size_t out_pitch;
  int* status;
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t scales_full[kScaleSlots], scales_empty[kScaleSlots];
  uint64_t sum_full[2], sum_empty[2], drained;
  uint32_t tmem;
  unsigned failed;
  int start[ZC_MOE_MAX_EXPERTS + 2];         // first row (or block) of each group
  long long tiles[ZC_MOE_MAX_EXPERTS + 2];   // tiles before each group
};

struct Tile {
  int group, p0, q0, q1;  // rows p0 .. of P, rows q0 .. q1 - 1 of Q
  int b0, b1;             // blocks
};

// Walks this CTA's tiles; every role walks them alike.
struct Walk {
  const TileParams& p;
  const Shared& s;
  long long t;
  int g = 0;
  __device__ Walk(const TileParams& p_, const Shared& s_) : p(p_), s(s_), t(blockIdx.x) {}
  __device__ bool next(Tile* out) {
    const int last = p.by_blocks ? p.groups : p.groups + 1;
    if (t >= s.tiles[last]) return false;
    while (s.tiles[g + 1] <= t) ++g;
    const int p_tiles = (p.p_rows + kTileP - 1) / kTileP;
    const long long local = t - s.tiles[g];
    const int q = static_cast<int>(local / p_tiles);
    out->group = g;
    out->p0 = static_cast<int>(local % p_tiles) * kTileP;
    if (p.by_blocks) {
      out->q0 = q * p.tile_q;
      out->q1 = min(p.q_rows, out->q0 + p.tile_q);
      out->b0 = s.start[g];
      out->b1 = s.start[g + 1];
    } else {
      out->q0 = s.start[g] + q * p.tile_q;
      out->q1 = min(s.start[g + 1], out->q0 + p.tile_q);
      out->b0 = 0;
      out->b1 = g == p.groups ? 0 : p.blocks;  // rows without a group: zeros
    }
    t += gridDim.x;
    return true;
  }
};

// The groups' starts (checked) and the tiles before each group, by one warp.
__device__ void plan_tiles(const TileParams& p, Shared& s) {
  const int lane = threadIdx.x % 32;
  const int limit = p.by_blocks ? p.blocks : p.q_rows;
  const int n = p.by_blocks ? p.groups : p.groups + 1;  // row groups: one more, the rows behind them
  const auto start_of = [&](int g) {
    if (g > p.groups) return limit;
    if (p.offsets == nullptr) return g == 0 ? 0 : limit;
    return p.offsets[g];
  };
  const long long p_tiles = (p.p_rows + kTileP - 1) / kTileP;
  long long before = 0;
  int floor = 0;  // starts never go back below this
  bool bad = false;
  for (int base = 0; base <= n; base += 32) {
    const int g = base + lane;
    const int raw = g <= n ? start_of(g) : limit;
    int v = min(max(raw, 0), limit);
    if (g == 0) v = 0;
    bad |= g <= n && raw != v;
    const int clamped = v;
    v = max(v, floor);
    for (int d = 1; d < 32; d *= 2) v = max(v, __shfl_up_sync(~0u, v, d));
    bad |= v != clamped;
    // this group's end is the next lane's start
    int next = __shfl_down_sync(~0u, v, 1);
    if (lane == 31) {
      const int r = g + 1 <= n ? start_of(g + 1) : limit;
      next = max(v, min(max(r, 0), limit));
    }
    const long long q = p.by_blocks ? (p.q_rows + p.tile_q - 1) / p.tile_q : (next - v + p.tile_q - 1) / p.tile_q;
    long long incl = g < n ? q * p_tiles : 0;
    const long long mine = incl;
    for (int d = 1; d < 32; d *= 2) {
      const long long u = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += u;
    }
    if (g <= n) {
      s.start[g] = v;
      s.tiles[g] = before + incl - mine;
    }
    before += __shfl_sync(~0u, incl, 31);
    floor = __shfl_sync(~0u, v, 31);
  }
  if (bad) set_error(p.status, ZC_ERR_CORRUPT);
}

// 128 rows' scale words as the copy to tensor memory takes them.
__device__ __forceinline__ uint4 scale_words(const uint32_t* words, int row0, int rows) {
  const int lane = threadIdx.x % 32;
  uint4 v;
  uint32_t* o = &v.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 32 * i + lane;
    o[i] = r < rows ? __ldg(words + r) : 0x7F7F7F7Fu;
  }
  return v;
}

__device__ __forceinline__ void put(float* to, uint32_t v) { *to = __uint_as_float(v); }
__device__ __forceinline__ void put(__nv_bfloat16* to, uint32_t v) { *to = __float2bfloat16_rn(__uint_as_float(v)); }

// The epilogue: warps 4-7, each its 32 lanes (rows of P) of every finished tile.
template <typename Out>
__device__ __forceinline__ void write_sums(const TileParams& p, Shared& s, uint32_t tmem, uint32_t accumulator) {
  const int quarter = threadIdx.x / 32 % 4, lane = threadIdx.x % 32;
  volatile unsigned* failed = &s.failed;
  const bool shared_columns = p.tile_q > kSecond;
  Walk walk(p, s);
  Tile tile;
  unsigned sums = 0;
  while (walk.next(&tile)) {
    const int pr = tile.p0 + 32 * quarter + lane, columns = tile.q1 - tile.q0;
    const size_t base = (p.by_blocks ? static_cast<size_t>(tile.group) * p.q_rows : 0) + tile.q0;
    Out* out = static_cast<Out*>(p.out) + base * p.out_pitch + pr;
    const int chunks = (columns + kChunk - 1) / kChunk;
    if (tile.b0 == tile.b1) {
      if (pr < p.p_rows)
        for (int c = 0; c < columns; ++c) put(out + c * p.out_pitch, 0u);
      continue;
    }
    if (!__all_sync(~0u, wait_phase(&s.sum_full[sums % 2], sums / 2 % 2, failed))) break;
    tcgen05_fence_after();
    const uint32_t from = tmem + (static_cast<uint32_t>(quarter) << 21) + sums % 2 * accumulator;
    // the first accumulator's shared columns are its last ones, the second's its first
    const int all = p.tile_q / kChunk, turn = shared_columns && sums % 2 == 0 ? all - 1 : 0;
    const auto chunk_at = [&](int i) { return i + turn < all ? i + turn : i + turn - all; };
    const auto store = [&](const uint32_t(&v)[kChunk], int chunk) {
      Out* to = out + static_cast<size_t>(chunk) * kChunk * p.out_pitch;
      const int n = columns - chunk * kChunk;
      if (pr >= p.p_rows) return;
      if (n >= kChunk) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) put(to + i * p.out_pitch, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          if (i < n) put(to + i * p.out_pitch, v[i]);
      }
    };
    const auto release = [&] {
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sum_empty[sums % 2]);
    };
    if (p.tile_q < kChunk) {  // 16 columns
      uint32_t v[16];
      tmem_load(from, v);
      tmem_load_wait(v);
      release();
      if (pr < p.p_rows)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < columns) put(out + i * p.out_pitch, v[i]);
    } else {
      // one chunk is stored while the next one is read
      uint32_t v[2][kChunk];
      tmem_load(from + chunk_at(0) * kChunk, v[0]);
#pragma unroll 2
      for (int i = 0; i < all; ++i) {
        tmem_load_wait(v[i % 2]);
        if (i == (shared_columns ? 0 : all - 1)) release();
        if (i + 1 < all) tmem_load(from + chunk_at(i + 1) * kChunk, v[(i + 1) % 2]);
        if (chunk_at(i) < chunks) store(v[i % 2], chunk_at(i));
        __syncwarp();
      }
    }
    ++sums;
  }
}

__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ TileParams p,
                                                             const __grid_constant__ CUtensorMap p_map,
                                                             const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ uint8_t raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stage_bytes = (kTileP + p.tile_q) * kBlock;
  uint8_t* slots = tiles + p.stages * stage_bytes;
  Shared& s = *reinterpret_cast<Shared*>(slots + kScaleSlots * kSlotBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(&s.full[i], 1);
        mbar_init(&s.empty[i], 1);
      }
      for (int i = 0; i < kScaleSlots; ++i) {
        mbar_init(&s.scales_full[i], 2);
        mbar_init(&s.scales_empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s.sum_full[i], 1);
        mbar_init(&s.sum_empty[i], 4);
      }
      mbar_init(&s.drained, 1);
      s.failed = 0;
      fence_mbar_init();
    }
  } else if (warp == 1) {
    tmem_alloc(&s.tmem, kColumns);
  } else if (warp == 2) {
    plan_tiles(p, s);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = s.tmem;
  const uint32_t scale_columns = tmem + kColumns - 16 * kScaleSlots;
  const uint32_t accumulator = min(p.tile_q, kSecond);  // columns from one accumulator to the next
  volatile unsigned* failed = &s.failed;

  Walk walk(p, s);
  Tile tile;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      unsigned phase = 0, loads = 0;
      bool ok = true;
      while (ok && walk.next(&tile)) {
        for (int b = tile.b0; b < tile.b1; ++b) {
          if (!(ok = wait_phase(&s.empty[stage], phase ^ 1, failed))) break;
          mbar_arrive_expect_tx(&s.full[stage], stage_bytes);
          const uint32_t at = smem_u32(tiles + stage * stage_bytes);
          tma_load_3d(at, &p_map, b * kBlock, tile.p0, p.by_blocks ? 0 : tile.group, &s.full[stage]);
          tma_load_2d(at + kTileP * kBlock, &q_map, b * kBlock, tile.q0, &s.full[stage]);
          ++loads;
          if (++stage == p.stages) stage = 0, phase ^= 1;
        }
      }
      // given up: the loads in flight still write this CTA's memory, so wait for them
      if (!ok)
        for (unsigned i = 0; i < loads && i < static_cast<unsigned>(p.stages); ++i) {
          if (--stage < 0) stage = p.stages - 1, phase ^= 1;
          const unsigned long long start = now_ns();
          while (!mbar_try_wait(&s.full[stage], phase) && now_ns() - start < kWaitLimitNs) {}
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t desc = product_desc(p.p_fmt, p.q_fmt, p.tile_q);
      int stage = 0, slot = 0;
      unsigned phase = 0, slot_phase = 0, sums = 0;
      // Tile j needs its accumulator read out: that of tile j - 2, and, where the accumulators
      // share columns, those of tile j - 1 (the epilogue reads in order, so that implies the rest).
      const unsigned lag = p.tile_q > kSecond ? 1 : 2;
      bool ok = true;
      while (ok && walk.next(&tile)) {
        if (tile.b0 == tile.b1) continue;
        if (sums >= lag) {
          const unsigned j = sums - lag;
          if (!(ok = wait_phase(&s.sum_empty[j % 2], j / 2 % 2, failed))) break;
          tcgen05_fence_after();
        }
        const uint32_t d = tmem + sums % 2 * accumulator;
        for (int b = tile.b0; b < tile.b1; ++b) {
          const uint32_t sp = scale_columns + slot * 16, sq = sp + 4;
          if (b == tile.b0 || b % 4 == 0) {
            if (!(ok = wait_phase(&s.scales_full[slot], slot_phase, failed))) break;
            tcgen05_fence_after();
            const uint32_t at = smem_u32(slots + slot * kSlotBytes);
            copy_scales(sp, scales_desc(at));
            copy_scales(sq, scales_desc(at + 512));
            if (p.tile_q > 128) copy_scales(sq + 4, scales_desc(at + 1024));
          }
          if (!(ok = wait_phase(&s.full[stage], phase, failed))) break;
          tcgen05_fence_after();
          const uint32_t at = smem_u32(tiles + stage * stage_bytes);
          const uint64_t pd = operand_desc(at), qd = operand_desc(at + kTileP * kBlock);
          const uint32_t desc_b = with_scale_byte(desc, b % 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // 32 columns each
            product(d, pd + 2 * i, qd + 2 * i, desc_b, sp, sq, b != tile.b0 || i != 0);
          commit_to(&s.empty[stage]);
          if (b % 4 == 3 || b == tile.b1 - 1) {
            commit_to(&s.scales_empty[slot]);
            if (++slot == kScaleSlots) slot = 0, slot_phase ^= 1;
          }
          if (++stage == p.stages) stage = 0, phase ^= 1;
        }
        if (!ok) break;
        commit_to(&s.sum_full[sums % 2]);
        ++sums;
      }
      if (!ok) {  // given up: the products in flight end before tensor memory is freed
        commit_to(&s.drained);
        const unsigned long long start = now_ns();
        while (!mbar_try_wait(&s.drained, 0) && now_ns() - start < kWaitLimitNs) {}
      }
    }
  } else if (warp < 4) {
    // warp 2 brings P's scales, warp 3 Q's; each has its next words' loads in flight while it
    // waits for a slot
    const bool is_p = warp == 2;
    const int chunks = is_p || p.tile_q <= 128 ? 1 : 2;
    uint4 next[2];
    int b = 0;
    bool more = walk.next(&tile);
    const auto fetch = [&] {  // the words of the blocks from b on
      while (more && b >= tile.b1) {
        more = walk.next(&tile);
        b = tile.b0;
      }
      if (!more) return;
      const size_t w = b / 4;
      if (is_p) {
        const uint32_t* at = p.p_scales + (p.by_blocks ? 0 : static_cast<size_t>(tile.group) * p.words * p.p_rows);
        next[0] = scale_words(at + w * p.p_rows, tile.p0, p.p_rows);
      } else {
        const uint32_t* at = p.q_scales + w * p.q_rows;
        next[0] = scale_words(at, tile.q0, tile.q1);
        if (chunks > 1) next[1] = scale_words(at, tile.q0 + 128, tile.q1);
      }
      b = (b / 4 + 1) * 4;
    };
    b = more ? tile.b0 : 0;
    fetch();
    int slot = 0;
    unsigned phase = 0;
    for (bool one = more; one; ) {
      const uint4 now[2] = {next[0], next[1]};
      fetch();
      one = more;
      if (!__all_sync(~0u, wait_phase(&s.scales_empty[slot], phase ^ 1, failed))) break;
      uint4* to = reinterpret_cast<uint4*>(slots + slot * kSlotBytes) + lane + (is_p ? 0 : 32);
      to[0] = now[0];
      if (chunks > 1) to[32] = now[1];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.scales_full[slot]);
      if (++slot == kScaleSlots) slot = 0, phase ^= 1;
    }
  } else {
    if (p.out_fp32) write_sums<float>(p, s, tmem, accumulator);
    else write_sums<__nv_bfloat16>(p, s, tmem, accumulator);
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tcgen05_fence_after();
    tmem_free(tmem, kColumns);
  }
  if (threadIdx.x == 0 && s.failed) set_error(p.status, ZC_ERR_TIMEOUT);
}

size_t smem_bytes(int tile_q, int stages) {
  return 1024 + static_cast<size_t>(stages) * (kTileP + tile_q) * kBlock + kScaleSlots * kSlotBytes + sizeof(Shared);
}
constexpr size_t kSmemLimit = 227 * 1024;

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    else
      cudaGetLastError();
  });
  return fn;
}

// Tiles of box_rows rows x 128 bytes of `matrices` matrices of rows x pitch bytes, 128-byte swizzle; what lies
// outside reads as zero.  Loads start at columns that are multiples of 128.
cudaError_t tile_map(const uint8_t* base, size_t pitch, size_t rows, size_t matrices, int dims, int box_rows,
                     CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t size[3] = {pitch, rows, matrices};
  const cuuint64_t strides[2] = {pitch, pitch * rows};
  const cuuint32_t box[3] = {kBlock, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<uint8_t*>(base), size, strides, box,
                            unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_tiles(TileParams& t, const uint8_t* pv, size_t p_pitch, size_t p_matrices, const uint8_t* qv,
                         size_t q_pitch, const DeviceInfo& dev, cudaStream_t stream) {
  t.stages = 2;
  while (t.stages < kMaxStages && smem_bytes(t.tile_q, t.stages + 1) <= kSmemLimit) ++t.stages;
  t.status = dev.status;
  CUtensorMap p_map, q_map;
  cudaError_t err = tile_map(pv, p_pitch, t.p_rows, p_matrices, 3, kTileP, &p_map);
  if (err == cudaSuccess) err = tile_map(qv, q_pitch, t.q_rows, 1, 2, t.tile_q, &q_map);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemLimit));
  if (err != cudaSuccess) return err;
  const size_t most = ceil_div(t.p_rows, kTileP) *
                      (t.by_blocks ? ceil_div(t.q_rows, t.tile_q) * t.groups : t.q_rows / t.tile_q + t.groups + 1);
  const unsigned grid = static_cast<unsigned>(most < static_cast<size_t>(dev.sm_count) ? most : dev.sm_count);
  return launch(matmul_kernel, grid, kThreads, smem_bytes(t.tile_q, t.stages), stream, false, t, p_map, q_map);
}

// Rows of Q a tile takes: the smallest that holds an average group.
int tile_rows(size_t average) {
  int t = 16;
  while (t < kMaxTileQ && static_cast<size_t>(t) < average) t *= 2;
  return t;
}

}  // namespace

cudaError_t launch_matmul(const Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  const size_t blocks = ceil_div(p.k, kBlock), active = p.rows < static_cast<size_t>(p.groups) ? p.rows : p.groups;
  TileParams t{};
  t.p_scales = reinterpret_cast<const uint32_t*>(p.b_scales);
  t.q_scales = reinterpret_cast<const uint32_t*>(p.a_scales);
  t.p_fmt = p.b_fmt;
  t.q_fmt = p.a_fmt;
  t.groups = p.groups;
  t.out_fp32 = p.out_type == ZC_TYPE_FP32;
  t.p_rows = static_cast<int>(p.n);
  t.q_rows = static_cast<int>(p.rows);
  t.blocks = static_cast<int>(blocks);
  t.words = static_cast<int>(ceil_div(blocks, 4));
  t.by_blocks = false;
  t.tile_q = tile_rows(ceil_div(p.rows, active));
  t.offsets = p.offsets;
  t.out = p.out;
  t.out_pitch = p.out_pitch;
  return launch_tiles(t, p.b, blocks * kBlock, p.groups, p.a, blocks * kBlock, dev, stream);
}

cudaError_t launch_weight_grad(const Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  const size_t capacity = p.rows;
  if (capacity == 0)  // no rows at all: zeros
    return cudaMemsetAsync(p.out, 0, p.groups * p.n * p.k * type_bytes(p.out_type), stream);
  TileParams t{};
  t.p_scales = reinterpret_cast<const uint32_t*>(p.b_scales);
  t.q_scales = reinterpret_cast<const uint32_t*>(p.a_scales);
  t.p_fmt = p.b_fmt;
  t.q_fmt = p.a_fmt;
  t.groups = p.groups;
  t.out_fp32 = p.out_type == ZC_TYPE_FP32;
  t.p_rows = static_cast<int>(p.k);
  t.q_rows = static_cast<int>(p.n);
  t.blocks = static_cast<int>(capacity);
  t.words = static_cast<int>(ceil_div(capacity, 4));
  t.by_blocks = true;
  t.tile_q = tile_rows(p.n);
  t.offsets = p.offsets;
  t.out = p.out;
  t.out_pitch = p.k;
  return launch_tiles(t, p.b, capacity * kBlock, 1, p.a, capacity * kBlock, dev, stream);
}

}  // namespace ex
}  // namespace zc
