// Fifth-generation tensor core (tcgen05) helpers: tensor memory, descriptors, the
// bf16 product with fp32 accumulators, and bounded barrier waits.
#pragma once

#include "encode.cuh"  // packed fp32 pairs

namespace adamas {

// ---------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_alloc512(uint32_t* slot) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free512(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive 32-bit columns of the lane's row (the warp's quadrant is in addr).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// Waits for the thread's loads; the registers pass through so that nothing uses them before.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---------------------------------------------------------------- operands in shared memory
// A 128 x 128 bf16 tile is two halves of 64 columns, each 128 rows of 128 bytes with
// the 16-byte pieces of a row exchanged by the row number (128-byte swizzle): 16 KB
// a half, 1024-byte aligned.
constexpr int kTileHalf = 128 * 128;
constexpr int kTileBytes = 2 * kTileHalf;

// Byte offset of piece c (0..15, 8 elements) of row r.
__device__ __forceinline__ uint32_t tile_piece(int r, int c) {
  return (uint32_t)((c >> 3) * kTileHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

constexpr uint64_t kDescSw128 = (1ull << 46) | (2ull << 61);
// Rows are the matrix's rows (its product runs along a row): 1024 bytes between groups
// of eight rows.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  return kDescSw128 | (uint64_t)((addr & 0x3FFFF) >> 4) | (1ull << 16) | (64ull << 32);
}
// The product runs down the rows (V: rows are tokens): 1024 bytes between groups of
// eight rows, one half between 64 columns and the next.
__device__ __forceinline__ uint64_t desc_cols(uint32_t addr) {
  return kDescSw128 | (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(kTileHalf >> 4) << 16) | (64ull << 32);
}

// Instruction descriptor: fp32 accumulators, bf16 operands, 128 x 128; B's product
// along its rows or down its rows.
constexpr uint32_t kMma128 = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kMma128Bcols = kMma128 | (1u << 16);

// The barrier is arrived at once when every product this thread issued before is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// S = A B^T of two 128 x 128 tiles in shared memory (8 steps of 16 along the rows).  One
// asm block: the descriptors are formed next to their use and hold no registers between.
__device__ __forceinline__ void mma_rows_rows(uint32_t d, uint32_t a, uint32_t b) {
  const uint64_t da = desc_rows(a), db = desc_rows(b);
  asm volatile(
      "{\n .reg .b64 x, y;\n .reg .pred p, q;\n setp.ne.u32 p, 0, 0;\n setp.eq.u32 q, 0, 0;\n"
      " add.s64 x, %1, 0;\n add.s64 y, %2, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n"
      " add.s64 x, %1, 2;\n add.s64 y, %2, 2;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 4;\n add.s64 y, %2, 4;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 6;\n add.s64 y, %2, 6;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 1024;\n add.s64 y, %2, 1024;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 1026;\n add.s64 y, %2, 1026;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 1028;\n add.s64 y, %2, 1028;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      " add.s64 x, %1, 1030;\n add.s64 y, %2, 1030;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
      "}" ::"r"(d),
      "l"(da), "l"(db), "r"(kMma128)
      : "memory");
}
// O (+)= P V: P bf16 in tensor memory (64 columns), V's rows in shared memory.
__device__ __forceinline__ void mma_probs_rows(uint32_t d, uint32_t p, uint32_t v, bool acc) {
  const uint64_t dv = desc_cols(v);
  asm volatile(
      "{\n .reg .b64 y;\n .reg .b32 a;\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.eq.u32 q, 0, 0;\n"
      " add.u32 a, %1, 0;\n add.s64 y, %2, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, p;\n"
      " add.u32 a, %1, 8;\n add.s64 y, %2, 128;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 16;\n add.s64 y, %2, 256;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 24;\n add.s64 y, %2, 384;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 32;\n add.s64 y, %2, 512;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 40;\n add.s64 y, %2, 640;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 48;\n add.s64 y, %2, 768;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      " add.u32 a, %1, 56;\n add.s64 y, %2, 896;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %3, q;\n"
      "}" ::"r"(d),
      "r"(p), "l"(dv), "r"(kMma128Bcols), "r"((uint32_t)acc)
      : "memory");
}

// ---------------------------------------------------------------- barriers, copies
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for the phase, for two seconds at most: a wait that runs out sets *gave_up
// (shared memory), after which every wait of the block returns at once, so that all its
// loops still end.
__device__ __forceinline__ void mbar_wait_or_give_up(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up) {
  if (mbar_try(bar, parity)) return;
  uint64_t end = 0;
  for (uint32_t i = 0; i < (1u << 26); ++i) {
    if (mbar_try(bar, parity)) return;
    if ((i & 31u) == 31u) {
      if (*gave_up) return;
      const uint64_t now = global_ns();
      if (end == 0) end = now + 2000000000ull;
      else if (now > end) break;
    }
  }
  *gave_up = 1u;
}

// 16 bytes to shared memory, or 16 zero bytes when !live (the source is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// One box of a two-dimensional tensor map (64 columns at x, a multiple of 64, and the
// map's box of rows at y) to shared memory, in the map's 128-byte swizzle; its bytes are
// counted on the barrier.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// The same from a three-dimensional map: 64 columns at x, its box of y and z.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// A box of a three-dimensional map from shared memory; the copies of a thread are committed
// in groups, and it may wait until the last ones have read the memory, or are done.
__device__ __forceinline__ void tma_store_3d(const void* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// The barrier is arrived at once when every cp.async this thread issued before has landed
// (the arrival counts as one of those the barrier expects).  Whoever waits for it runs
// fence_async_smem() before the tensor core reads what landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float fast_exp2(float x) {  // 2 ulp; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace adamas
