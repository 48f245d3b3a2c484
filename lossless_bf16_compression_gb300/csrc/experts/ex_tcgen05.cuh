// ex_tcgen05.cuh -- PTX wrappers for the tensor cores (tcgen05), tensor memory and TMA tile loads.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ex_common.cuh"

namespace zc {
namespace ex {

// ------------------------------------------------------------------ bounded waits

// Nanoseconds that a wait for a whole tile may take longer than another, for each block of its sum: a block takes
// 0.3 us, but the longest sum, a weight gradient's over 2^31 rows in one group, 4.4 s.
constexpr unsigned long long kWaitBlockNs = 2000;

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase of `bar`; false when the limit ran out or another wait of the CTA gave up.
// (Acquires at cluster scope: a pair's barriers are arrived at by both CTAs.)
__device__ __forceinline__ bool phase_done(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The flag of having given up, in this CTA and (with G = 2) in the other one of the pair.
template <int G>
__device__ __forceinline__ void give_up(volatile unsigned* failed) {
  *failed = 1;
  if (G == 2)
    asm volatile(
        "{\n\t.reg .b32 r, a;\n\tmov.u32 r, %%cluster_ctarank;\n\txor.b32 r, r, 1;\n\t"
        "mapa.shared::cluster.u32 a, %0, r;\n\tst.relaxed.cluster.shared::cluster.u32 [a], 1;\n\t}" ::"r"(
            smem_u32(const_cast<unsigned*>(failed)))
        : "memory");
}
template <int G>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, volatile unsigned* failed,
                                           unsigned long long limit) {
  if (phase_done(bar, parity)) return true;
  const unsigned long long start = now_ns();
  for (unsigned i = 1;; ++i) {
    if (phase_done(bar, parity)) return true;
    if (i % 256 == 0 && (*failed || now_ns() - start > limit)) {
      give_up<G>(failed);
      return false;
    }
  }
}
// Bytes taken as arrived, of those that a phase of `bar` was told to expect.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, unsigned bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// A word of the second CTA's shared memory, at the place of this CTA's `word`.
__device__ __forceinline__ unsigned seconds_word(const unsigned* word) {
  unsigned v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, 1;\n\tld.relaxed.cluster.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_u32(word))
      : "memory");
  return v;
}

// One lane of a converged warp.  The tensor-core and TMA instructions take uniform operands: a
// warp that walks its loop together and lets one lane issue them keeps those operands in uniform
// registers, while a lone lane in a loop of its own has to move every one of them there (8192^3
// product: 190 cycles a 128 x 256 x 32 instruction from a lone lane, against the 128 it executes in).
__device__ __forceinline__ bool elect_one() {
  unsigned r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// ------------------------------------------------------------------ CTA pairs
//
// G = 1: a CTA works alone; G = 2: the two CTAs of a cluster share a product (each holds half of
// both operands and 128 rows of the result), issued by the first of them, the leader.

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The leader's barrier at the place of this CTA's `bar`, as a cluster address.
template <int G>
__device__ __forceinline__ uint32_t leaders(uint64_t* bar) {
  uint32_t a = smem_u32(bar);
  if (G == 2) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}
// For what the arrival tells about lies in tensor memory and is ordered by tcgen05 waits and fences,
// so the arrival itself is relaxed: a release at cluster scope would wait for this thread's loads
// and stores in flight (1800 cycles next to the tiles' traffic).
template <int G>
__device__ __forceinline__ void arrive_at_leader(uint64_t* bar) {
  if (G == 1) mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(leaders<G>(bar)) : "memory");
}

// ------------------------------------------------------------------ TMA tile loads (this CTA's memory)

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// The bytes are counted at `bar`, a cluster address (with G = 2, the leader's).
template <int G>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (G == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int G>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (G == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------ tensor memory and products

// By one warp (with G = 2, by one of each CTA of the pair).
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_result, unsigned columns) {
  if (G == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_result)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_result)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, unsigned columns) {
  if (G == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor of an operand tile: rows of 128 bytes, 128-byte swizzle, groups
// of 8 rows 1024 bytes apart.
constexpr uint64_t kDescVersion = 1ull << 46;
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem) {
  return (smem >> 4) | (uint64_t(1024 >> 4) << 32) | kDescVersion | (2ull << 61);
}
// Instruction descriptor of a block-scaled 8-bit product (128 G x n, K = 32, both operands
// K-major, power-of-two scales); the scale byte of the word is picked by `byte` for both operands.
template <int G>
__device__ __forceinline__ uint32_t product_desc(int a_fmt, int b_fmt, int n) {
  return (static_cast<uint32_t>(a_fmt) << 7) | (static_cast<uint32_t>(b_fmt) << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (uint32_t(128 * G >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_scale_byte(uint32_t desc, unsigned byte) {
  return desc | (byte << 4) | (byte << 29);
}

template <int G>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t a_scales,
                                        uint32_t b_scales, bool add) {
  if (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// 4 columns of this warp's 32 lanes; done after tmem_store_wait.
__device__ __forceinline__ void tmem_store(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Arrives at `bar` (with G = 2, in both CTAs of the pair) once every tcgen05 operation that this
// thread issued before is done.
template <int G>
__device__ __forceinline__ void commit_to(uint64_t* bar) {
  if (G == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<unsigned short>(3))
        : "memory");
}

// 16 or 32 columns of this warp's 32 lanes; the values are there after tmem_load_wait.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
      "%23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
// (the registers pass through it, so that nothing uses them before)
template <int N>
__device__ __forceinline__ void tmem_load_wait(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

}  // namespace ex
}  // namespace zc
