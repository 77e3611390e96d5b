// tensor_core.cuh -- fifth-generation tensor cores, tensor memory, TMA copies and
// mbarriers for the operators that are products of tiles: PTX wrappers and the waits'
// limit. One block per SM (its shared memory sees to that) uses all of its
// tensor memory.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "op_common.cuh"

namespace rar {
namespace tc {

__device__ __forceinline__ uint32_t shared_address(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

// ---- mbarriers ----
__device__ __forceinline__ void barrier_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_address(b)), "r"(count) : "memory");
}
// Barriers that one thread has initialised, for the copies and products that will arrive on them.
__device__ __forceinline__ void barriers_ready() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_address(b)) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_address(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool try_wait(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(shared_address(b)), "r"(parity)
      : "memory");
  return done != 0;
}

// try_wait may hold the thread for microseconds before it says no; this does not.
__device__ __forceinline__ bool ended(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(shared_address(b)), "r"(parity)
      : "memory");
  return done != 0;
}

// In shared memory: whether a wait of the block has run out, and how long each may take (of the order of a second: no
// tile takes a thousandth of that).
struct Limit {
  int dead;
  uint64_t ns;
};
__device__ __forceinline__ bool wait_lane(uint64_t* b, uint32_t parity, volatile Limit* limit) {
#pragma unroll 1
  for (int i = 0; i < 16; i++)
    if (try_wait(b, parity)) return true;
  const uint64_t since = global_timer_ns();
  while (!try_wait(b, parity)) {
    if (global_timer_ns() - since > limit->ns) limit->dead = 1;
    if (limit->dead) return false;
  }
  return true;
}
// A warp waits for the phase of `parity` to end. False, for all its lanes, once any wait of the block has run past the
// limit: every role then leaves its loops. (Lanes that went by what each of them found could part ahead of what a warp does
// together.)
__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, volatile Limit* limit) {
  return __all_sync(~0u, wait_lane(b, parity, limit));
}
// The same, and what follows is uniform to the compiler. The timer between two looks keeps a waiting warp from the issue
// slots of those that work (without it the gradient of 8192 tokens, heads of 64, took 5 % longer).
__device__ __forceinline__ bool wait_warp(uint64_t* b, uint32_t parity, volatile Limit* limit) {
  if (__all_sync(~0u, try_wait(b, parity))) return true;
  const uint64_t since = global_timer_ns();
#pragma unroll 1
  while (true) {
    if (__all_sync(~0u, try_wait(b, parity))) return true;
    const bool late = global_timer_ns() - since > limit->ns;
    if (late) limit->dead = 1;
    if (__any_sync(~0u, late || limit->dead)) return false;
  }
}
// A number that all lanes of a warp have, as one that the compiler knows they have.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(~0u, x); }

// ---- TMA ----
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void copy_3d(void* to, const CUtensorMap* m, int x, int y, int z, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          shared_address(to)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(shared_address(b))
      : "memory");
}
__device__ __forceinline__ void copy_4d(void* to, const CUtensorMap* m, int x, int y, int z, int w, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          shared_address(to)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(shared_address(b))
      : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* m, int x, int y, int z, const void* from) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m), "r"(x), "r"(y),
               "r"(z), "r"(shared_address(from))
               : "memory");
}
// The thread's stores so far have read shared memory, or have been written as well.
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void stores_written() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---- copies of 16 bytes, the last 16 - bytes of them 0 ----
__device__ __forceinline__ void copy_16(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_of_a_tile() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_done() {  // but for those of the last LEFT tiles
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Ordinary stores to shared memory, for products that read it afterwards.
__device__ __forceinline__ void stores_to_products() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ----
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(where)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void loads_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define RAR_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define RAR_V8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 32 columns of the lane's row of the warp's quarter; valid after loads_done().
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : RAR_R8(r, 0), RAR_R8(r, 8), RAR_R8(r, 16), RAR_R8(r, 24)
      : "r"(at));
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : RAR_R8(r, 0), RAR_R8(r, 8)
               : "r"(at));
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      RAR_V8(r, 0), RAR_V8(r, 8), RAR_V8(r, 16), RAR_V8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
               RAR_V8(r, 0), RAR_V8(r, 8)
               : "memory");
}

// ---- registers of a warpgroup ----
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- products ----
// Operands in shared memory are slabs of 64 elements (128 bytes) a row, swizzled by 128
// bytes as TMA writes them: eight rows are 1024 bytes in a row, `group` bytes lie
// between them and the next eight, `slab` bytes between slabs. A tile is slab by slab
// (groups 1024 bytes apart), or eight rows of all slabs after one another.
// along: the contraction runs along the rows' elements (next 16: 32 bytes on, next 64:
// the next slab). across: it runs across the rows (next 16: two groups on), with results
// along the elements.
// The upper half of a descriptor holds the group's bytes and is the same for both; the
// lower one the address and the bytes between slabs in units of 16, so a step is an
// addition to it.
constexpr uint32_t kGroup = 1024;
__device__ __forceinline__ uint32_t operand_high(uint32_t group) { return group >> 4 | 1u << 14 | 2u << 29; }
__device__ __forceinline__ uint32_t operand_along(uint32_t at) { return at >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t operand_across(uint32_t at, uint32_t slab) { return at >> 4 | (slab >> 4) << 16; }
// bf16 operands, binary32 sums, 128 rows by n columns (a multiple of 16).
__device__ __forceinline__ uint32_t product_of(int n, bool right_across) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (right_across ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
// d (+)= a b over 16 elements, issued by the lane that leads; the whole warp comes here
// together. a in shared memory, or in tensor memory (two elements a column).
__device__ __forceinline__ void multiply(uint32_t lead, uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high,
                                         uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kind), "r"((uint32_t)add), "r"(a_high), "r"(lead), "r"(b_high)
      : "memory");
}
__device__ __forceinline__ void multiply_tmem(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t kind,
                                              bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kind), "r"((uint32_t)add), "r"(b_high), "r"(lead)
      : "memory");
}
// Arrives on b once the leading lane's products so far are done.
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* b) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(shared_address(b)),
      "r"(lead)
      : "memory");
}

// One lane issues all products of a tile, so the instructions around each count: in a
// branch of that lane alone, with descriptors worked out anew, a product took 108 cycles
// to issue and 64 to run. Hence additions to the lower halves only, loops unrolled to
// MOST, and a warp that stays together, whose numbers the compiler keeps in uniform
// registers, where the products want them.
// d = x y^T: 128 rows of x, slab by slab, by n rows of y, `steps` times 16 elements along both.
template <int MOST, int SLAB>
__device__ __forceinline__ void rows_by_rows(uint32_t lead, uint32_t d, uint32_t x, uint32_t y, int n, int steps,
                                             uint32_t slab = SLAB, uint32_t group = kGroup) {
  const uint32_t kind = product_of(n, false), a = operand_along(x), b = operand_along(y), high = operand_high(group);
#pragma unroll
  for (int k = 0; k < MOST; k++)
    if (k < steps)
      multiply(lead, d, a + (((k >> 2) * SLAB + (k & 3) * 32) >> 4), operand_high(kGroup), b + (((k >> 2) * slab + (k & 3) * 32) >> 4),
               high, kind, k > 0);
}
// d (+)= w z: w in tensor memory, 128 rows by 128, its columns in slices of 16 PER elements that begin STRIDE columns
// apart; z has as many rows, n elements each. The part of them from step FIRST to LAST.
template <int PER, int STRIDE, int FIRST = 0, int LAST = 8>
__device__ __forceinline__ void weights_by_rows(uint32_t lead, uint32_t d, uint32_t w, uint32_t z, int n, bool add, uint32_t slab,
                                                uint32_t group = kGroup) {
  const uint32_t kind = product_of(n, true), b = operand_across(z, slab), high = operand_high(group);
#pragma unroll
  for (int k = FIRST; k < LAST; k++)
    multiply_tmem(lead, d, w + k / PER * STRIDE + k % PER * 8, b + k * (group >> 3), high, kind, add || k > 0);
}

// What the bf16 pair `to` leaves of x and y, as another.
__device__ __forceinline__ uint32_t bf16_rest(float x, float y, uint32_t to) {
  const float2 r = unpack(fma2(f2(bf16_lo(to), bf16_hi(to)), f2(-1.f, -1.f), f2(x, y)));
  return bf16_pair(r.x, r.y);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace tc

// TMA descriptors of 2-byte elements, boxes 64 elements wide, swizzled by 128 bytes, zeros outside.
// Three dimensions, the innermost dense: boxes of 64 by `rows` by `planes`.
cudaError_t make_map(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t stride1_bytes,
                     int64_t stride2_bytes, int rows, int planes);
// Dense rows of a multiple of 64 elements, eight by eight: boxes of 64 elements by 8 rows by all slabs by `groups`.
cudaError_t make_grouped_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int groups);

}  // namespace rar
