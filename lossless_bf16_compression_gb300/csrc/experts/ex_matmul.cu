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
// each CTA loading half of both, which takes a third off what the SMs read from the L2
// and off the shared-memory traffic that a CTA alone is bound by (8192^3: 304 us against 347).
// Many rows are bound by the tensor cores (32768 rows, 7168 x 4096, 16 groups: 528 us, 3.6 PFLOP/s; back to
// back the power limit brings the clock down to 1.4 GHz and that to 3.1), few by the weights' bytes (32
// rows: 69 us, 6.0 TB/s of the active groups' weights).
// Roles: warp 0 issues the TMA loads (128 columns a stage), warp 1 the products, warps 2, 3, 8 and 9
// bring the scales, warps 4-7 and 10-13 write the results while the next tile's products run.
//
// Scales are kept four blocks to a word, [word][row].  A product's scales lie in tensor memory, row
// r at lane r % 32 (in each quarter of the lanes) and column r / 32, so a warp reads 32 rows' words
// as one coalesced load and stores them as one column; byte b % 4 is picked by the instruction.
#include <cmath>
#include <mutex>

#include "ex_fp8.cuh"
#include "ex_tcgen05.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kThreads = 448;
constexpr int kBand = 2048;  // rows of P: 152 SMs hold 16 x 9.5 tiles of 128 x 256
constexpr int kTileP = 128;
constexpr int kWriters = 8;    // warps of the epilogue
constexpr int kMaxStages = 12;
constexpr int kMaxTurns = 4;   // words of scales in tensor memory; two where accumulators leave no more room
constexpr int kWordsAhead = 4;
constexpr int kTurnColumns = 16;  // 4 of P's scales, and 4 for every 128 rows of Q
constexpr int kColumns = 512;        // tensor memory: all of it (one CTA an SM)
constexpr int kChunk = 32;           // accumulator columns a warp reads at once
// Two accumulators of 256 columns and the scales do not fit in 512 columns: with tiles of 256 the
// second accumulator starts at column 224, and the epilogue reads the 32 columns they share first.
constexpr int kSecond = 224;
// Sharing out takes about 0.27 us for each block that a CTA has less to do and adds up to 8 us (the
// clearing, the parts, the join), so it pays from 24 blocks on: one group of 8 rows, 7168 x 4096, 32 tiles, 44
// blocks less: 17.8 us against 19.4; 14336 x 4096, 88 less: 21 against 34.6; 64 rows of four groups, 4096 x
// 512, 28 less: 11.1 against 13.2; 48 rows of 16 groups, 7168 x 4096, 480 tiles or 24 more than three
// rounds, 47 less: 76.5 against 82; 20 rows of 64 groups, 7168 x 2048, 18 less: 47.4 against 45.6; 100
// rows of eight groups, 2048 x 2048, 2 less: 17.3 against 11.3.
constexpr int kWorthSharing = 24;

struct TileParams {
  const uint32_t *p_scales, *q_scales;  // words
  int p_fmt, q_fmt, groups, out_fp32;
  int p_rows, q_rows;         // rows of P (of one group), and of Q in all
  int blocks;                 // by_blocks: the capacity; else the blocks of a row
  int words;                  // scale words of a row
  bool by_blocks;             // the groups are runs of blocks, and out has a matrix for each
  int tile_q, stages;
  bool out_words;             // rows of out may be stored two 16-bit values at a time
  const int* offsets;         // rows (or blocks) of each group; null: one group
  // Where tiles are few: the blocks of those beyond whole rounds are shared out evenly, so that a CTA
  // begins and ends inside tiles.  Its sums of a part of a tile go to `parts` (two a CTA, [column][128
  // rows]), and whichever warp comes last to its share of a tile, by `arrivals` (eight a tile, zero
  // at the start), adds the parts in their order.  Null: whole tiles.
  float* parts;
  unsigned* arrivals;
  void* out;
  size_t out_pitch;
  int* status;
  unsigned long long wait_ns;  // limit of a wait (for a whole tile: and kWaitBlockNs for each of its blocks)
  int stalled;                 // the CTA that loads nothing, for the test of the waits; -1: none
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t scales_full[kMaxTurns], scales_empty[kMaxTurns];
  uint64_t sum_full[2], sum_empty[2], drained;
  uint32_t tmem;
  unsigned failed;
  unsigned loads;                            // stages that this CTA has loaded
  int start[ZC_MOE_MAX_EXPERTS + 2];         // first row (or block) of each group
  unsigned tiles[ZC_MOE_MAX_EXPERTS + 2];    // tiles before each group
};

struct Tile {
  int group, p0, q0, q1;  // rows p0 .. of P, rows q0 .. q1 - 1 of Q
  int b0, b1;             // blocks
  unsigned index;         // tiles before it
};

// Walks the tiles of this CTA (or pair); every role walks them alike.
// (32-bit arithmetic: the host refuses a product with 2^31 blocks of tiles; 64-bit divisions here
// took 4 us before the first load.)
template <int G>
struct Walk {
  const TileParams& p;
  const Shared& s;
  unsigned t;
  int g = 0;
  const unsigned p_tiles;
  // Shared out: the first tiles, those beyond whole rounds of all the CTAs, where that is worth it.
  unsigned begin = 0, end = 0;  // this CTA's blocks of them
  int phase = 0;
  unsigned ctas = 1;            // that share them: each gets a word of scales, four blocks, at least
  unsigned each = 0, more = 0;  // blocks of a CTA; the first `more` get another one
  __device__ Walk(const TileParams& p_, const Shared& s_)
      : p(p_), s(s_), t(blockIdx.x / G), p_tiles((p_.p_rows + kTileP * G - 1) / (kTileP * G)) {
    if (p.parts) {
      const unsigned tiles = s.tiles[p.groups] % gridDim.x, all = tiles * p.blocks;  // (of tiles that have blocks)
      if (all && (all + gridDim.x - 1) / gridDim.x + kWorthSharing <= static_cast<unsigned>(p.blocks)) {
        ctas = min(gridDim.x, max(all / 4, 1u));
        each = all / ctas;
        more = all - each * ctas;
        begin = begin_of(blockIdx.x);
        end = begin_of(blockIdx.x + 1);
        t += tiles;
      }
    }
  }
  // The first block of a CTA, all tiles' blocks in a row, and the CTA that has a block.
  __device__ unsigned begin_of(unsigned cta) const {
    const unsigned c = min(cta, ctas);
    return c * each + min(c, more);
  }
  __device__ unsigned cta_of(unsigned block) const {
    const unsigned longer = more * (each + 1);
    return block < longer ? block / (each + 1) : more + (block - longer) / each;
  }

  __device__ bool next(Tile* out) {
    const int last = p.by_blocks ? p.groups : p.groups + 1;
    if (begin < end && phase < 2) {
      // The parts of tiles first -- of the one that the CTA ends inside, then of the one that it
      // begins inside -- so that they are joined while the whole tiles are under way.
      const unsigned blocks = p.blocks;
      if (phase == 0) {
        phase = 1;
        const unsigned from = end - end % blocks;
        if (from != end && from >= begin) return part(from, end, out);
      }
      phase = 2;
      if (begin % blocks) return part(begin, min(end, begin - begin % blocks + blocks), out);
    }
    if (t >= s.tiles[last]) return false;
    locate(t, out);
    t += gridDim.x / G;
    return true;
  }

  __device__ bool part(unsigned from, unsigned to, Tile* out) {
    const unsigned tile = from / p.blocks;
    locate(tile, out);
    out->b0 = from - tile * p.blocks;
    out->b1 = out->b0 + (to - from);
    return true;
  }

  __device__ void locate(unsigned tile, Tile* out) {
    // the group, 32 looked at a time (every role's warp walks as a whole)
    if (s.tiles[g] > tile) g = 0;
    const int lane = threadIdx.x % 32, groups = p.by_blocks ? p.groups : p.groups + 1;
    for (;;) {
      const unsigned before = __ballot_sync(~0u, g + lane < groups && s.tiles[min(g + lane, groups - 1) + 1] <= tile);
      if (before != ~0u) {
        g += __ffs(~before) - 1;
        break;
      }
      g += 32;
    }
    // Within a group: bands of kBand rows of P, and in a band all of P's tiles for each of Q's, so
    // that the tiles in flight at a time cover about as many rows of P as of Q.  Shared-out tiles
    // follow one another in a CTA: there Q's tiles for each of P's, whose rows are then in the L2.
    const unsigned local = tile - s.tiles[g], q_tiles = (s.tiles[g + 1] - s.tiles[g]) / p_tiles;
    unsigned q, pt;
    if (p.parts) {
      pt = local / q_tiles;
      q = local - pt * q_tiles;
    } else {
      constexpr unsigned width = kBand / (kTileP * G);
      const unsigned band = local / (width * q_tiles), inside = local - band * width * q_tiles;
      const unsigned here = min(width, p_tiles - band * width);
      q = inside / here;
      pt = band * width + inside - q * here;
    }
    out->index = tile;
    out->group = g;
    out->p0 = pt * kTileP * G;
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
  const unsigned p_tiles = (p.p_rows + kTileP * G - 1) / (kTileP * G);
  unsigned before = 0;
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
    const unsigned q = ((p.by_blocks ? p.q_rows : next - v) + p.tile_q - 1) / p.tile_q;
    unsigned incl = g < n ? q * p_tiles : 0;
    const unsigned mine = incl;
    for (int d = 1; d < 32; d *= 2) {
      const unsigned u = __shfl_up_sync(~0u, incl, d);
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
  const auto word = [&](int i) { return r + 32 * i < rows ? words[r + 32 * i] : 0x7F7F7F7Fu; };
  return make_uint4(word(0), word(1), word(2), word(3));
}

__device__ __forceinline__ void put(float* to, uint32_t v) { *to = __uint_as_float(v); }
__device__ __forceinline__ void put(__nv_bfloat16* to, uint32_t v) { *to = __float2bfloat16_rn(__uint_as_float(v)); }

// Columns c and c + 1 of 32 neighbouring outputs each, as 16 words of column c from the even lanes
// and 16 of column c + 1 from the odd ones: a lane gives its neighbour the value that belongs to
// its word.
__device__ __forceinline__ uint32_t pair_up(uint32_t v0, uint32_t v1) {
  uint32_t own, r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(own) : "f"(__uint_as_float(v1)), "f"(__uint_as_float(v0)));
  const uint32_t other = __shfl_xor_sync(~0u, own, 1);
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(own), "r"(other), "r"(threadIdx.x % 2 ? 0x3276u : 0x5410u));
  return r;
}

// The epilogue: two warps for each quarter of the tensor-memory lanes (32 rows of P), one taking the even
// chunks of a tile's columns and one the odd ones.  A warp reads a chunk, waits and stores it; a second
// chunk in flight made it slower (weights' gradient, 2048 x 7168, 16 groups of 8 blocks: 180 us, 172
// without; of 1 block 150 and 135), the second warp covers the wait (1 block: 110 us, 4.3 TB/s written).

// A warp's share of a part of a tile: to its place among the parts, and the whole if it is the last.
template <typename Out>
__device__ __forceinline__ void write_part(const TileParams& p, Shared& s, const Walk<1>& walk, const Tile& tile,
                                           uint32_t from, unsigned acc, int quarter, int half) {
  const int lane = threadIdx.x % 32, row = 32 * quarter + lane;
  if (16 * half >= p.tile_q) {  // 16 columns: all the other warp's
    if (lane == 0) mbar_arrive(&s.sum_empty[acc]);
    return;
  }
  const unsigned tile_begin = tile.index * p.blocks;
  const size_t part = static_cast<size_t>(kTileP) * p.tile_q;
  // a CTA's first place is for the tile that it begins inside, its second for one that it begins
  const auto place = [&](unsigned cta) {
    return p.parts + (2 * cta + (walk.begin_of(cta) > tile_begin ? 0 : 1)) * part + row;
  };
  float* mine = place(blockIdx.x);
  for (int c = 16 * half; c < p.tile_q; c += 32) {
    uint32_t v[16];
    tmem_load(from + c, v);
    tmem_load_wait(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) __stcg(mine + (c + i) * kTileP, __uint_as_float(v[i]));
  }
  tcgen05_fence_before();
  __threadfence();
  __syncwarp();
  unsigned before = 0;
  if (lane == 0) {
    mbar_arrive(&s.sum_empty[acc]);
    before = atomicAdd(&p.arrivals[static_cast<size_t>(tile.index) * kWriters + 2 * quarter + half], 1u);
  }
  before = __shfl_sync(~0u, before, 0);
  const unsigned first = walk.cta_of(tile_begin), last = walk.cta_of(tile_begin + p.blocks - 1);
  if (before != last - first) return;
  __threadfence();
  const int pr = tile.p0 + row;
  Out* out = static_cast<Out*>(p.out) + static_cast<size_t>(tile.q0) * p.out_pitch + pr;
  for (int c = 16 * half; c < tile.q1 - tile.q0; c += 32) {
    float sum[16] = {};
    for (unsigned cta = first; cta <= last; cta += 4) {  // four parts' loads in flight
      float v[4][16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* from_part = place(min(cta + k, last)) + c * kTileP;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[k][i] = __ldcg(from_part + i * kTileP);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += cta + k <= last ? v[k][i] : 0.f;
    }
    if (pr < p.p_rows)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < tile.q1 - tile.q0) put(out + (c + i) * p.out_pitch, __float_as_uint(sum[i]));
  }
}

template <int G, typename Out>
__device__ __forceinline__ void write_sums(const TileParams& p, Shared& s, uint32_t tmem, uint32_t accumulator,
                                           int first_row) {
  const int quarter = threadIdx.x / 32 % 4, lane = threadIdx.x % 32, half = threadIdx.x / 32 >= 10;
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
        for (int c = half; c < columns; c += 2) put(out + c * p.out_pitch, 0u);
      continue;
    }
    const unsigned long long limit = p.wait_ns + kWaitBlockNs * (tile.b1 - tile.b0);
    if (!__all_sync(~0u, wait_phase<G>(&s.sum_full[sums % 2], sums / 2 % 2, failed, limit))) break;
    tcgen05_fence_after();
    const uint32_t from = tmem + (static_cast<uint32_t>(quarter) << 21) + sums % 2 * accumulator;
    if constexpr (G == 1) {
      if (p.parts && tile.b1 - tile.b0 != p.blocks) {
        write_part<Out>(p, s, walk, tile, from, sums % 2, quarter, half);
        ++sums;
        continue;
      }
    }
    // the first accumulator's shared columns are its last ones, the second's its first
    const int all = p.tile_q / kChunk, turn = shared_columns && sums % 2 == 0 ? all - 1 : 0;
    const auto chunk_at = [&](int i) { return i + turn < all ? i + turn : i + turn - all; };
    const auto store = [&](const uint32_t(&v)[kChunk], int chunk) {
      Out* to = out + static_cast<size_t>(chunk) * kChunk * p.out_pitch;
      const int n = columns - chunk * kChunk;
      if (sizeof(Out) == 2 && p.out_words && n >= kChunk) {
        // two columns a store, half as many stores (16 groups of 8 blocks, 2048 x 7168: 176 -> 170 us,
        // of 1 block 121 -> 110; whole rows by way of shared memory took half as long again, the
        // operands' traffic leaves it no bandwidth)
        uint32_t w[kChunk / 2];
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) w[i] = pair_up(v[2 * i], v[2 * i + 1]);
        if (pr >= p.p_rows) return;
        to += lane % 2 ? static_cast<ptrdiff_t>(p.out_pitch) - 1 : 0;
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) *reinterpret_cast<uint32_t*>(to + 2 * i * p.out_pitch) = w[i];
        return;
      }
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
      if (half == 0) {
        tmem_load(from, v);
        tmem_load_wait(v);
      }
      release();
      if (half == 0 && pr < p.p_rows)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < columns) put(out + i * p.out_pitch, v[i]);
    } else {
      // this warp has done with the columns that the other accumulator shares, or with all, after:
      const int done = shared_columns ? half : (all - 1 - half) / 2 * 2 + half;
      if (half >= all) release();
#pragma unroll 1
      for (int i = half; i < all; i += 2) {
        uint32_t v[kChunk];
        tmem_load(from + chunk_at(i) * kChunk, v);
        tmem_load_wait(v);
        if (i == done) release();
        if (chunk_at(i) < chunks) store(v, chunk_at(i));
        __syncwarp();
      }
    }
    ++sums;
  }
}

// After the roles gave up: the loads in flight still write the CTA's (or pair's) memory, so wait for
// the last one of each stage.  In a pair one CTA may have loaded more stages than the other: the leader's
// barrier expects both's bytes once the leader has loaded, and none before.
template <int G>
__device__ __noinline__ void await_loads(const TileParams& p, Shared& s, uint32_t stage_bytes) {
  const unsigned first = s.loads, second = G == 2 ? seconds_word(&s.loads) : first, all = max(first, second);
  const unsigned stages = p.stages;
  for (unsigned n = all > stages ? all - stages : 0; n < all; ++n) {
    uint64_t* bar = &s.full[n % stages];
    if (n >= second) mbar_complete_tx(bar, stage_bytes);
    if (n >= first) mbar_arrive_expect_tx(bar, stage_bytes);
    const unsigned long long start = now_ns();
    while (!phase_done(bar, n / stages % 2) && now_ns() - start < kWaits.limit_ns) {}
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
  let_next_start();
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
        mbar_init(&s.sum_empty[i], kWriters * G);
      }
      mbar_init(&s.drained, 1);
      s.failed = 0;
      fence_mbar_init();
      prefetch_map(&p_map);
      prefetch_map(&q_map);
    }
  } else if (warp == 1) {
    tmem_alloc<G>(&s.tmem, kColumns);
  } else if (warp == 2) {
    wait_for_previous();
    plan_tiles<G>(p, s);
  }
  // Everything above this line touches only this CTA, so it may run while the kernel before it
  // in the stream ends.
  wait_for_previous();
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
    while (ok && p.stalled != static_cast<int>(blockIdx.x) && walk.next(&tile)) {
      const int z = p.by_blocks ? 0 : tile.group;
      for (int b = tile.b0; b < tile.b1; ++b) {
        if (!(ok = __all_sync(~0u, wait_phase<G>(&s.empty[stage], phase ^ 1, failed, p.wait_ns)))) break;
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
    if (lane == 0) s.loads = loads;
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
          if (!(ok = __all_sync(~0u, wait_phase<G>(&s.sum_empty[j % 2], j / 2 % 2, failed, p.wait_ns)))) break;
        }
        const uint32_t d = tmem + sums % 2 * accumulator;
        for (int b = tile.b0; b < tile.b1; ++b) {
          const uint32_t sp = scale_columns + turn * kTurnColumns, sq = sp + 4;
          const bool new_word = b == tile.b0 || b % 4 == 0, last = b == tile.b1 - 1, end_word = b % 4 == 3 || last;
          if (new_word && !(ok = __all_sync(~0u, wait_phase<G>(&s.scales_full[turn], turn_phase, failed, p.wait_ns))))
            break;
          if (!(ok = __all_sync(~0u, wait_phase<G>(&s.full[stage], phase, failed, p.wait_ns)))) break;
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
        while (!phase_done(&s.drained, 0) && now_ns() - start < kWaits.limit_ns) {}
      }
    }
  } else if (warp < 4 || warp == 8 || warp == 9) {
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
        ok = ok && have[i] && __all_sync(~0u, wait_phase<G>(&s.scales_empty[turn], phase ^ 1, failed, p.wait_ns));
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
  if (s.failed) {  // (the same in both CTAs of a pair)
    if (rank == 0 && threadIdx.x == 0) await_loads<G>(p, s, stage_bytes);
    if (G == 2) cluster_sync();
    if (threadIdx.x == 0) set_error(p.status, ZC_ERR_TIMEOUT);
  }
}

size_t smem_bytes(int load_q, int stages) {
  return 1024 + static_cast<size_t>(stages) * (kTileP + load_q) * kBlock + sizeof(Shared);
}
constexpr size_t kSmemLimit = 227 * 1024;
constexpr size_t kSms = 152;      // of a GB300, where a cut is chosen without asking the device
constexpr size_t kMaxCtas = 160;  // CTAs of a launch, for the size of a workspace
size_t sm_count(const DeviceInfo& dev) { return dev.sm_count < static_cast<int>(kMaxCtas) ? dev.sm_count : kMaxCtas; }

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
                         size_t q_pitch, const Waits& waits, const DeviceInfo& dev, cudaStream_t stream) {
  const int load_q = t.tile_q / G;
  t.stages = 2;
  while (t.stages < kMaxStages && smem_bytes(load_q, t.stages + 1) <= kSmemLimit) ++t.stages;
  t.status = dev.status;
  t.wait_ns = waits.limit_ns;
  t.stalled = waits.stalled;
  t.out_words = reinterpret_cast<uintptr_t>(t.out) % 4 == 0 && t.out_pitch % 2 == 0 && t.p_rows % 2 == 0;
  CUtensorMap p_map, q_map;
  cudaError_t err = tile_map(pv, p_pitch, t.p_rows, p_matrices, 3, kTileP, &p_map);
  if (err == cudaSuccess) err = tile_map(qv, q_pitch, t.q_rows, 1, 2, load_q, &q_map);
  if (err == cudaSuccess) err = allow_shared_memory<matmul_kernel<G>>(kSmemLimit);
  if (err != cudaSuccess) return err;
  const size_t most = ceil_div(t.p_rows, kTileP * G) *
                      (t.by_blocks ? ceil_div(t.q_rows, t.tile_q) * t.groups : t.q_rows / t.tile_q + t.groups + 1);
  if (most * (t.parts ? t.blocks : 1) >= size_t(1) << 31) return cudaErrorInvalidValue;
  const size_t room = sm_count(dev) / G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(t.parts ? room : G * (most < room ? most : room)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(load_q, t.stages);
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = G;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  TimingRecord rec = timing_begin(ZC_KERNEL_FP8_PRODUCT, stream);
  err = cudaLaunchKernelEx(&cfg, matmul_kernel<G>, t, p_map, q_map);
  timing_end(rec, stream);
  return err;
}

__global__ void __launch_bounds__(1024) clear_kernel(uint4* to) {
  let_next_start();
  wait_for_previous();
  to[threadIdx.x] = make_uint4(0, 0, 0, 0);
}

// How a product is cut, from sizes alone (the groups' own sizes are on the device).
struct Shape {
  int tile_q;
  bool pair, share;  // share: tiles may be shared out
};

// Groups of up to 64 rows on average are bound by the weights' bytes: one tile for all of a group's
// rows where they are no more than half again the average.  Sums of more than kWorthSharing blocks
// may be shared out (the kernel knows how many tiles there are).  Larger groups are bound by the
// products: the cut with the least time by the measured cycles of a block, given its waves, and of
// the last tile's writing, which decides where all tiles are under way at once (669 rows of four
// groups, 935 x 166: 10.6 us with tiles of 128 x 128, 12.6 with pairs; 4096 rows of four groups, 4096 x 4096:
// 51 with pairs, 58 with 128 x 256, 91 with 128 x 128).
Shape shape_of(size_t q_rows, size_t groups, size_t p_rows, size_t blocks, bool by_blocks) {
  const size_t active = by_blocks ? groups : q_rows < groups ? q_rows : groups;
  const size_t average = by_blocks ? q_rows : ceil_div(q_rows, active);
  if (!by_blocks && average <= 64) {
    int t = 16;
    while (2 * static_cast<size_t>(t) < 3 * average) t *= 2;
    return {t, false, blocks > kWorthSharing};
  }
  const double sum = by_blocks ? std::fmax(1.0, static_cast<double>(blocks) / groups) : static_cast<double>(blocks);
  struct {
    Shape shape;
    double cycles, end;  // of a block of a tile, and of writing the last one
  } const cuts[] = {{{256, true, false}, 545, 5300}, {{256, false, false}, 722, 4300}, {{128, false, false}, 563, 2200}};
  const Shape* best = nullptr;
  double least = 0;
  for (const auto& c : cuts) {
    const size_t g = c.shape.pair ? 2 : 1;
    const double tiles = static_cast<double>(active) * ceil_div(average, c.shape.tile_q) * ceil_div(p_rows, kTileP * g);
    const double waves = std::ceil(tiles / (kSms / g));
    const double time = waves * sum * c.cycles + c.end;
    if (best == nullptr || time < least) best = &c.shape, least = time;
  }
  return *best;
}

constexpr size_t kArrivals = kMaxCtas * kWriters;
size_t parts_bytes(const Shape& shape) {
  return shape.share ? 2 * kMaxCtas * kTileP * shape.tile_q * sizeof(float) + kArrivals * sizeof(unsigned) : 0;
}

cudaError_t launch_any(TileParams& t, const Shape& shape, const uint8_t* pv, size_t p_pitch, size_t p_matrices,
                       const uint8_t* qv, size_t q_pitch, const Waits& waits, const DeviceInfo& dev,
                       cudaStream_t stream) {
  t.tile_q = shape.tile_q;
  return shape.pair ? launch_tiles<2>(t, pv, p_pitch, p_matrices, qv, q_pitch, waits, dev, stream)
                    : launch_tiles<1>(t, pv, p_pitch, p_matrices, qv, q_pitch, waits, dev, stream);
}

}  // namespace

size_t matmul_workspace(size_t rows, int groups, size_t n, size_t k) {
  return parts_bytes(shape_of(rows, groups, n, ceil_div(k, kBlock), false));
}

cudaError_t launch_matmul(const Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  const size_t blocks = ceil_div(p.k, kBlock);
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
  t.offsets = p.offsets;
  t.out = p.out;
  t.out_pitch = p.out_pitch;
  const Shape shape = shape_of(p.rows, p.groups, p.n, blocks, false);
  if (shape.share) {
    t.arrivals = static_cast<unsigned*>(p.workspace);
    t.parts = reinterpret_cast<float*>(t.arrivals + kArrivals);
    const cudaError_t err = launch(ZC_KERNEL_FP8_PRODUCT, clear_kernel, 1, kArrivals / 4, 0, stream,
                                   static_cast<uint4*>(p.workspace));
    if (err != cudaSuccess) return err;
  }
  return launch_any(t, shape, p.b, blocks * kBlock, p.groups, p.a, blocks * kBlock, p.waits, dev, stream);
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
  t.offsets = p.offsets;
  t.out = p.out;
  t.out_pitch = p.k;
  const Shape shape = shape_of(p.n, p.groups, p.k, capacity, true);
  return launch_any(t, shape, p.b, capacity * kBlock, 1, p.a, capacity * kBlock, p.waits, dev, stream);
}

}  // namespace ex
}  // namespace zc
