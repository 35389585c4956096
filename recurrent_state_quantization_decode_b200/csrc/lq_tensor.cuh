// Tensor-core plumbing of the chunked kernels: mbarriers with bounded waits,
// tiled bulk copies, tcgen05 products with operands in shared or tensor
// memory, and tensor-memory loads and stores.
//
// Tiles are bf16 in shared memory in blocks of 64 columns: block j of a tile
// of R rows is R rows of 128 bytes, 128-byte swizzled (16-byte unit u of row r
// lies at unit u ^ (r % 8)), 1024-byte aligned, at j * R * 128 bytes.  A tile
// serves as an operand whose contraction runs along its columns ("row"
// operands, K-major) or along its rows ("column" operands, MN-major).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lq {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers -----------------------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// Up to 64 polls for the phase, in as few instructions as there can be: waiting
// warps take issue slots from the others.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 64;\n\t"
      "POLL:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra POLL;\n\t"
      "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- bulk copies ---------------------------------------------------------

// 64 columns from x of rows y.. of head h, into one 64-column block.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                          int h, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(h), "r"(row), "r"(bar)
      : "memory");
}

// And out of it.  store_done waits until the block has been read.
__device__ __forceinline__ void store_tile(const CUtensorMap *map, uint32_t src, int x, int h,
                                           int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          map),
      "r"(x), "r"(h), "r"(row), "r"(src)
      : "memory");
}
__device__ __forceinline__ void store_done() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ---- tensor memory -------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Waits for the loads issued so far.  The loaded registers pass through, so
// that no use of them can move above the wait.
__device__ __forceinline__ void wait_loads(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void wait_loads(uint32_t (&r)[16], uint32_t (&s)[16]) {
  wait_loads(r);
  asm volatile("" : "+r"(s[0]), "+r"(s[1]), "+r"(s[2]), "+r"(s[3]), "+r"(s[4]), "+r"(s[5]),
                    "+r"(s[6]), "+r"(s[7]), "+r"(s[8]), "+r"(s[9]), "+r"(s[10]), "+r"(s[11]),
                    "+r"(s[12]), "+r"(s[13]), "+r"(s[14]), "+r"(s[15]));
}
__device__ __forceinline__ void wait_stores() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Columns col .. of the warp's 32 lanes: lane l's register j is column j.
__device__ __forceinline__ void load16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void store8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Transposes on the way into tensor memory.  Four 8 x 8 blocks of a tile, each
// lane giving the address of one row (lanes 0-7 block 0, 8-15 block 1, ...):
// lane l gets, of each block, its column l / 4, rows 2 (l % 4) and the next.
__device__ __forceinline__ void load_transposed(uint32_t row, uint32_t (&r)[8], int at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[at]), "=r"(r[at + 1]), "=r"(r[at + 2]), "=r"(r[at + 3])
               : "r"(row)
               : "memory");
}
// 16 lanes x 16 columns: register 2 g + i of lane l is column 4 g + l % 4 of
// lane 8 i + l / 4 (counted from the address).
__device__ __forceinline__ void store_blocks(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// ---- products ------------------------------------------------------------

// Instruction descriptor: bf16 operands, fp32 result, M x N.
__host__ __device__ constexpr uint32_t product_shape(int m, int n, bool a_column, bool b_column) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_column ? 1u << 15 : 0u) |
         (b_column ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
         (static_cast<uint32_t>(m / 16) << 24);
}

// Operand descriptors of 128-byte swizzled tiles.  Row operand: groups of 8
// rows 1024 bytes apart; 16 columns further is 32 bytes, the next 64 a block.
// Column operand: 64-column blocks `block` bytes apart, groups of 8 rows 1024
// bytes apart; 16 rows further is 2048 bytes.
// The low word; the high one is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t block) {
  return addr >> 4 | (block >> 4) << 16;
}
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// D (tensor memory) = [D +] A B for one step of 16 along the contraction; issued by
// the lane with `lead`.
__device__ __forceinline__ void product_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                           uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %6, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"(static_cast<uint32_t>(add)), "r"(kOperandHigh), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b,
                                           uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %6, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"(static_cast<uint32_t>(add)), "r"(kOperandHigh), "r"(lead)
      : "memory");
}
// One lane of a warp, as 1 there and 0 elsewhere.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
               : "=r"(r));
  return r;
}
// The barrier gets one arrival when all products that the lane has issued so far
// are done.
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
}  // namespace tc
}  // namespace lq
