// zpp_tcgen05.cuh -- what the tensor-core kernels share: tensor copies into shared memory, the
// fifth-generation matrix unit (tcgen05) with its accumulators in tensor memory, and waits that end.
//
// Operands lie in shared memory in rows of 128 bytes, swizzled in units of 16 bytes within groups
// of 8 rows (1024 bytes, so tiles start at multiples of 1024), as a tensor copy with the 128-byte
// swizzle writes them. An operand whose sum index runs along those rows is "K-major"; one whose rows
// are steps of the sum is "MN-major".
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zpp_device.cuh"

namespace zpp {

constexpr long long kTensorWaitClocks = 2000000000ll;  // about 1 s, then a wait gives up

// ------------------------------------------------------------------ tensor memory and the matrix unit
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_out, uint32_t cols) {  // one whole warp
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(smem_out)),
                 "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(smem_out)),
                 "r"(cols)
                 : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {  // the warp that allocated
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  } else {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
}
// After the last allocation of a CTA: others on the SM may allocate.
template <int CTAS>
__device__ __forceinline__ void tmem_alloc_done() {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  else
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// An arrival on `bar` once every product issued so far by this thread has ended.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}
// The same of a pair of CTAs, on the barrier at this place in both.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
          "r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tc_commit_to(uint64_t* bar) {
  if constexpr (CTAS == 2) tc_commit_pair(bar);
  else tc_commit(bar);
}

// Descriptor of an operand tile at `addr` (a shared-memory address, 1024-byte aligned plus an
// advance along the sum). K-major: groups of 8 rows are `stride` bytes apart, `lead` is not used.
// MN-major: 64-element columns of rows are `lead` bytes apart, groups of 8 sum steps `stride`.
__device__ __forceinline__ uint64_t tc_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// What a product is: fp32 sums of a [rows] x [cols] tile; formats by kind (f16: 0 f16, 1 bf16;
// f8f6f4: 0 e4m3).
__host__ __device__ constexpr uint32_t tc_instruction(int rows, int cols, uint32_t a_format,
                                                      uint32_t b_format, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_format << 7) | (b_format << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(cols >> 3) << 17) |
         (static_cast<uint32_t>(rows >> 4) << 24);
}
#define ZPP_TC_MMA(GROUP, KIND)                                                                     \
  asm volatile(                                                                                     \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                             \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),      \
      "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))                                   \
      : "memory")
// tmem (+)= a b^T over 32 e4m3 steps of the sum, by one thread.
template <int CTAS>
__device__ __forceinline__ void tc_mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t instr,
                                          bool add) {
  if constexpr (CTAS == 1) ZPP_TC_MMA("1", "f8f6f4");
  else ZPP_TC_MMA("2", "f8f6f4");
}
// The same over 16 fp16 steps.
template <int CTAS>
__device__ __forceinline__ void tc_mma_f16(uint32_t tmem, uint64_t a, uint64_t b, uint32_t instr,
                                           bool add) {
  if constexpr (CTAS == 1) ZPP_TC_MMA("1", "f16");
  else ZPP_TC_MMA("2", "f16");
}
#undef ZPP_TC_MMA

// 8, 16 or 32 fp32 columns of this thread's lane: lane 32 (warp % 4) + lane number, the address's
// lane bits set by the caller. Valid after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld(uint32_t tmem, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(tmem));
}
__device__ __forceinline__ void tmem_ld(uint32_t tmem, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(tmem));
}
__device__ __forceinline__ void tmem_ld(uint32_t tmem, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(tmem));
}
// (the loaded registers pass through, so that no use of them moves before the wait)
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// ------------------------------------------------------------------------------- tensor copies
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// A box of the map's tensor, its first element at (x, y[, z]), to shared memory; what lies outside the
// tensor arrives as zeros. x times the element size is a multiple of 16. The bytes of the whole box
// complete on `bar`.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// The way back: a box in shared memory to the map's tensor, what lies outside it left out. By one thread,
// after every writer's tma_store_fence() and a barrier; its stores so far are a group at tma_store_commit().
__device__ __forceinline__ void tma_store_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's groups have read their shared memory; have written.
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ------------------------------------------------------------------------------------ pairs of CTAs
// Two CTAs of a cluster work on one tile of 256 rows: each holds 128 rows of P and half of Q's, the
// first one issues the products for both, and each has its rows' sums in its own tensor memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; what was written before is visible after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared variable of this CTA in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
// The same of a shared-memory address, and a store there.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// (What it tells of is tensor memory that was read, ordered by tc_fence_before: no release of this
// thread's other writes to the cluster is asked for, which takes 1000 clocks and more.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// As tma_load, the bytes counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, int z,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------------------------- warps' parts
// A kernel of 3 warpgroups: the first one copies and issues products, the others work on results. The
// registers of 384 threads with 168 each go 56 to the first and 224 to the others: 128 * 56 + 256 * 224
// = 384 * 168.
constexpr int kTensorThreads = 384;
constexpr int kCopyWarp = 0, kProductWarp = 1, kFirstScaleWarp = 2, kFirstResultWarp = 4, kResultWarps = 8;
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;"); }

// -------------------------------------------------------------------------------- bounded waits
// Waits for a barrier's phase; after so many clocks it sets `bit` of the fault word, and this
// thread's later waits return at once (`alive` is false: what it computes is unspecified, and the
// kernel ends). Inline: a call would hold registers that these kernels do not have.
__device__ __forceinline__ void tc_wait_long(uint64_t* bar, unsigned parity, bool& alive, unsigned* fault,
                                             unsigned bit, long long clocks) {
  if (mbar_try_wait(bar, parity) || !alive) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > clocks) {
      alive = false;
      atomicOr(fault, bit);
      return;
    }
  }
}
__device__ __forceinline__ void tc_wait(uint64_t* bar, unsigned parity, bool& alive, unsigned* fault,
                                        unsigned bit) {
  tc_wait_long(bar, parity, alive, fault, bit, kTensorWaitClocks);
}

// Whether a barrier's phase has completed, without waiting: asked while something else is going on.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One thread of a whole warp (the compiler knows it is one: what it issues takes uniform registers).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A place in a ring of N and the parity of its current round.
template <int N>
struct Ring {
  int at = 0;
  unsigned phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, phase ^= 1u;
  }
};

}  // namespace zpp
