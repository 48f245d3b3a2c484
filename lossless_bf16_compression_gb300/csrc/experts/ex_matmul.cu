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
// columns.  Tiles of 256 rows of Q are shared by a pair of CTAs, 256 rows of P by 256 of Q with
// each CTA loading half of both, which takes a third off what the SMs read from the L2.  Roles: warp 0 issues the TMA loads (128 columns a stage), warp 1 the products,
// warps 2, 3, 8 and 9 bring the scales, warps 4-7 write the results while the next tile's products
// run.
//
// Scales are kept four blocks to a word, [word][row].  A product's scales lie in tensor memory, row
// r at lane r % 32 (in each quarter of the lanes) and column r / 32, so a warp reads 32 rows' words
// as one coalesced load and stores them as one column; byte b % 4 is picked by the instruction.
#include <mutex>

#include "ex_fp8.cuh"
#include "ex_tcgen05.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kThreads = 320;
constexpr int kBand = 2048;  // rows of P: 152 SMs hold 16 x 9.5 tiles of 128 x 256
constexpr int kTileP = 128;
constexpr int kMaxTileQ = 256;
constexpr int kMaxStages = 12;
constexpr int kMaxTurns = 4;   // words of scales in tensor memory; two where accumulators leave no more room
constexpr int kWordsAhead = 4;
constexpr int kTurnColumns = 16;  // 4 of P's scales, and 4 for every 128 rows of Q
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
  uint64_t scales_full[kMaxTurns], scales_empty[kMaxTurns];
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

// Walks the tiles of this CTA (or pair); every role walks them alike.
template <int G>
struct Walk {
  const TileParams& p;
  const Shared& s;
  long long t;
  int g = 0;
  __device__ Walk(const TileParams& p_, const Shared& s_) : p(p_), s(s_), t(blockIdx.x / G) {}
  __device__ bool next(Tile* out) {
    const int last = p.by_blocks ? p.groups : p.groups + 1;
    if (t >= s.tiles[last]) return false;
    while (s.tiles[g + 1] <= t) ++g;
    const int p_tiles = (p.p_rows + kTileP * G - 1) / (kTileP * G);
    // Within a group: bands of kBand rows of P, and in a band all of P's tiles for each of Q's, so
    // that the tiles in flight at a time cover about as many rows of P as of Q.
    const long long local = t - s.tiles[g], q_tiles = (s.tiles[g + 1] - s.tiles[g]) / p_tiles;
    constexpr int width = kBand / (kTileP * G);
    const int band = static_cast<int>(local / (width * q_tiles));
    const int inside = static_cast<int>(local - band * width * q_tiles);
    const int here = min(width, p_tiles - band * width);
    const int q = inside / here;
    out->group = g;
    out->p0 = (band * width + inside % here) * kTileP * G;
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
    t += gridDim.x / G;
    return true;
  }
};

// The groups' starts (checked) and the tiles before each group, by one warp.
template <int G>
__device__ void plan_tiles(const TileParams& p, Shared& s) {
  const int lane = threadIdx.x % 32;
  const int limit = p.by_blocks ? p.blocks : p.q_rows;
  const int n = p.by_blocks ? p.groups : p.groups + 1;  // row groups: one more, the rows behind them
  const auto start_of = [&](int g) {
    if (g > p.groups) return limit;
    if (p.offsets == nullptr) return g == 0 ? 0 : limit;
    return p.offsets[g];
  };
  const long long p_tiles = (p.p_rows + kTileP * G - 1) / (kTileP * G);
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

// The scale words of rows row0 + lane, + 32, + 64, + 96 (1 past the last row).
__device__ __forceinline__ uint4 scale_words(const uint32_t* words, int row0, int rows) {
  const int r = row0 + static_cast<int>(threadIdx.x % 32);
  const auto word = [&](int i) { return r + 32 * i < rows ? __ldg(words + r + 32 * i) : 0x7F7F7F7Fu; };
  return make_uint4(word(0), word(1), word(2), word(3));
}

__device__ __forceinline__ void put(float* to, uint32_t v) { *to = __uint_as_float(v); }
__device__ __forceinline__ void put(__nv_bfloat16* to, uint32_t v) { *to = __float2bfloat16_rn(__uint_as_float(v)); }

// The epilogue: warps 4-7, each its 32 lanes (rows of P) of every finished tile.
template <int G, typename Out>
__device__ __forceinline__ void write_sums(const TileParams& p, Shared& s, uint32_t tmem, uint32_t accumulator,
                                           int first_row) {
  const int quarter = threadIdx.x / 32 % 4, lane = threadIdx.x % 32;
  volatile unsigned* failed = &s.failed;
  const bool shared_columns = p.tile_q > kSecond;
  Walk<G> walk(p, s);
  Tile tile;
  unsigned sums = 0;
  while (walk.next(&tile)) {
    const int pr = tile.p0 + first_row + 32 * quarter + lane, columns = tile.q1 - tile.q0;
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
      if (lane == 0) arrive_at_leader<G>(&s.sum_empty[sums % 2]);
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

template <int G>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ TileParams p,
                                                             const __grid_constant__ CUtensorMap p_map,
                                                             const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ uint8_t raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int load_q = p.tile_q / G;  // rows of Q that this CTA loads
  const uint32_t stage_bytes = (kTileP + load_q) * kBlock;
  Shared& s = *reinterpret_cast<Shared*>(tiles + p.stages * stage_bytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = G == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int first_row = rank * kTileP;  // of a tile's rows of P

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(&s.full[i], 1);
        mbar_init(&s.empty[i], 1);
      }
      for (int i = 0; i < kMaxTurns; ++i) {
        mbar_init(&s.scales_full[i], 4 * G);
        mbar_init(&s.scales_empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s.sum_full[i], 1);
        mbar_init(&s.sum_empty[i], 4 * G);
      }
      mbar_init(&s.drained, 1);
      s.failed = 0;
      fence_mbar_init();
    }
  } else if (warp == 1) {
    tmem_alloc<G>(&s.tmem, kColumns);
  } else if (warp == 2) {
    plan_tiles<G>(p, s);
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (G == 2) cluster_sync();  // the pair's barriers are set up
  tcgen05_fence_after();
  const uint32_t tmem = s.tmem;
  const unsigned turns = p.tile_q > 128 ? 2 : kMaxTurns;
  const uint32_t scale_columns = tmem + kColumns - kTurnColumns * turns;
  const uint32_t accumulator = min(p.tile_q, kSecond);  // columns from one accumulator to the next
  volatile unsigned* failed = &s.failed;

  Walk<G> walk(p, s);
  Tile tile;
  if (warp == 0) {
    int stage = 0;
    unsigned phase = 0, loads = 0;
    bool ok = true;
    while (ok && walk.next(&tile)) {
      const int z = p.by_blocks ? 0 : tile.group;
      for (int b = tile.b0; b < tile.b1; ++b) {
        if (!(ok = __all_sync(~0u, wait_phase(&s.empty[stage], phase ^ 1, failed)))) break;
        const uint32_t at = smem_u32(tiles) + stage * stage_bytes, bar = leaders<G>(&s.full[stage]);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], G * stage_bytes);
          tma_load_3d<G>(at, &p_map, b * kBlock, tile.p0 + first_row, z, bar);
          tma_load_2d<G>(at + kTileP * kBlock, &q_map, b * kBlock, tile.q0 + rank * load_q, bar);
        }
        ++loads;
        if (++stage == p.stages) stage = 0, phase ^= 1;
      }
    }
    // given up: the loads in flight still write the CTA's (or pair's) memory, so wait for them
    if (!ok && rank == 0)
      for (unsigned i = 0; i < loads && i < static_cast<unsigned>(p.stages); ++i) {
        if (--stage < 0) stage = p.stages - 1, phase ^= 1;
        const unsigned long long start = now_ns();
        while (!phase_done(&s.full[stage], phase) && now_ns() - start < kWaitLimitNs) {}
      }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t desc = product_desc<G>(p.p_fmt, p.q_fmt, p.tile_q);
      int stage = 0;
      unsigned phase = 0, sums = 0, turn = 0, turn_phase = 0;
      // Tile j needs its accumulator read out: that of tile j - 2, and, where the accumulators
      // share columns, those of tile j - 1 (the epilogue reads in order, so that implies the rest).
      const unsigned lag = p.tile_q > kSecond ? 1 : 2;
      bool ok = true;
      while (ok && walk.next(&tile)) {
        if (tile.b0 == tile.b1) continue;
        if (sums >= lag) {
          const unsigned j = sums - lag;
          if (!(ok = __all_sync(~0u, wait_phase(&s.sum_empty[j % 2], j / 2 % 2, failed)))) break;
        }
        const uint32_t d = tmem + sums % 2 * accumulator;
        for (int b = tile.b0; b < tile.b1; ++b) {
          const uint32_t sp = scale_columns + turn * kTurnColumns, sq = sp + 4;
          const bool new_word = b == tile.b0 || b % 4 == 0, last = b == tile.b1 - 1, end_word = b % 4 == 3 || last;
          if (new_word && !(ok = __all_sync(~0u, wait_phase(&s.scales_full[turn], turn_phase, failed)))) break;
          if (!(ok = __all_sync(~0u, wait_phase(&s.full[stage], phase, failed)))) break;
          tcgen05_fence_after();
          const uint32_t at = smem_u32(tiles) + stage * stage_bytes;
          const uint64_t pd = operand_desc(at), qd = operand_desc(at + kTileP * kBlock);
          const uint32_t desc_b = with_scale_byte(desc, b % 4);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)  // 32 columns each
              product<G>(d, pd + 2 * i, qd + 2 * i, desc_b, sp, sq, b != tile.b0 || i != 0);
            commit_to<G>(&s.empty[stage]);
            if (end_word) commit_to<G>(&s.scales_empty[turn]);
            if (last) commit_to<G>(&s.sum_full[sums % 2]);
          }
          if (end_word && ++turn == turns) turn = 0, turn_phase ^= 1;
          if (++stage == p.stages) stage = 0, phase ^= 1;
        }
        ++sums;
      }
      if (!ok) {  // given up: the products in flight end before tensor memory is freed
        if (elect_one()) commit_to<G>(&s.drained);
        const unsigned long long start = now_ns();
        while (!phase_done(&s.drained, 0) && now_ns() - start < kWaitLimitNs) {}
      }
    }
  } else if (warp < 4 || warp >= 8) {
    // The scales: one warp for each quarter of the tensor-memory lanes, which all hold the same
    // words.  Next to the tiles' traffic a load takes about 2000 cycles, as long as a word's
    // products, so the words of the next kWordsAhead - 1 are on their way in registers.
    // (By way of shared memory and the copy to tensor memory, a word also cost a proxy fence of
    // 1800 cycles.)
    const uint32_t to = scale_columns + (static_cast<uint32_t>(warp % 4) << 21);
    uint4 vp[kWordsAhead], v0[kWordsAhead], v1[kWordsAhead];
    bool more = walk.next(&tile);
    int b = more ? tile.b0 : 0;
    const auto fetch = [&](uint4& wp, uint4& w0, uint4& w1) {  // the words of the blocks from b on
      while (more && b >= tile.b1) {
        more = walk.next(&tile);
        b = tile.b0;
      }
      if (!more) return false;
      const size_t w = b / 4;
      const uint32_t* q_words = p.q_scales + w * p.q_rows;
      wp = scale_words(p.p_scales + ((p.by_blocks ? 0 : static_cast<size_t>(tile.group) * p.words) + w) * p.p_rows,
                       tile.p0 + first_row, p.p_rows);
      w0 = scale_words(q_words, tile.q0, p.q_rows);
      if (p.tile_q > 128) w1 = scale_words(q_words, tile.q0 + 128, p.q_rows);
      b = (b / 4 + 1) * 4;
      return true;
    };
    bool have[kWordsAhead];
#pragma unroll
    for (int i = 0; i < kWordsAhead; ++i) have[i] = fetch(vp[i], v0[i], v1[i]);
    unsigned turn = 0, phase = 0;
    for (bool ok = true; ok;) {
#pragma unroll
      for (int i = 0; i < kWordsAhead; ++i) {
        ok = ok && have[i] && __all_sync(~0u, wait_phase(&s.scales_empty[turn], phase ^ 1, failed));
        if (!ok) break;
        tcgen05_fence_after();
        const uint32_t at = to + turn * kTurnColumns;
        tmem_store(at, vp[i].x, vp[i].y, vp[i].z, vp[i].w);
        tmem_store(at + 4, v0[i].x, v0[i].y, v0[i].z, v0[i].w);
        if (p.tile_q > 128) tmem_store(at + 8, v1[i].x, v1[i].y, v1[i].z, v1[i].w);
        tmem_store_wait();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at_leader<G>(&s.scales_full[turn]);
        if (++turn == turns) turn = 0, phase ^= 1;
        have[i] = fetch(vp[i], v0[i], v1[i]);
      }
    }
  } else {
    if (p.out_fp32) write_sums<G, float>(p, s, tmem, accumulator, first_row);
    else write_sums<G, __nv_bfloat16>(p, s, tmem, accumulator, first_row);
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (G == 2) cluster_sync();  // the pair's last loads, products and arrivals have landed
  if (warp == 1) {
    __syncwarp();
    tcgen05_fence_after();
    tmem_free<G>(tmem, kColumns);
  }
  if (threadIdx.x == 0 && s.failed) set_error(p.status, ZC_ERR_TIMEOUT);
}

size_t smem_bytes(int load_q, int stages) {
  return 1024 + static_cast<size_t>(stages) * (kTileP + load_q) * kBlock + sizeof(Shared);
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

template <int G>
cudaError_t launch_tiles(TileParams& t, const uint8_t* pv, size_t p_pitch, size_t p_matrices, const uint8_t* qv,
                         size_t q_pitch, const DeviceInfo& dev, cudaStream_t stream) {
  const int load_q = t.tile_q / G;
  t.stages = 2;
  while (t.stages < kMaxStages && smem_bytes(load_q, t.stages + 1) <= kSmemLimit) ++t.stages;
  t.status = dev.status;
  CUtensorMap p_map, q_map;
  cudaError_t err = tile_map(pv, p_pitch, t.p_rows, p_matrices, 3, kTileP, &p_map);
  if (err == cudaSuccess) err = tile_map(qv, q_pitch, t.q_rows, 1, 2, load_q, &q_map);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(matmul_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemLimit));
  if (err != cudaSuccess) return err;
  const size_t most = ceil_div(t.p_rows, kTileP * G) *
                      (t.by_blocks ? ceil_div(t.q_rows, t.tile_q) * t.groups : t.q_rows / t.tile_q + t.groups + 1);
  const size_t room = dev.sm_count / G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(G * (most < room ? most : room)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(load_q, t.stages);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = G;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<G>, t, p_map, q_map);
}

cudaError_t launch_any(TileParams& t, const uint8_t* pv, size_t p_pitch, size_t p_matrices, const uint8_t* qv,
                       size_t q_pitch, const DeviceInfo& dev, cudaStream_t stream) {
  return t.tile_q == kMaxTileQ && t.p_rows > kTileP
             ? launch_tiles<2>(t, pv, p_pitch, p_matrices, qv, q_pitch, dev, stream)
             : launch_tiles<1>(t, pv, p_pitch, p_matrices, qv, q_pitch, dev, stream);
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
  return launch_any(t, p.b, blocks * kBlock, p.groups, p.a, blocks * kBlock, dev, stream);
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
  return launch_any(t, p.b, capacity * kBlock, 1, p.a, capacity * kBlock, dev, stream);
}

}  // namespace ex
}  // namespace zc
