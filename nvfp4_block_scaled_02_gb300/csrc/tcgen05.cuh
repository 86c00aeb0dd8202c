// tcgen05.cuh -- the few Blackwell tensor-core, tensor-memory, tensor-map and
// mbarrier instructions that the attention and matrix product kernels use, as
// inline PTX.
#pragma once
#include <cstdint>

namespace nvfp4 {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// True in one lane of a converged warp. The compiler knows that a single lane
// goes on, so MMA operands stay in uniform registers: issuing one took 9 clocks
// behind this and 45 behind a comparison of the lane number.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------- mbarriers ---
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.shared::cta.b64 t, [%0];\n\t}" ::"r"(
                   smem_addr(b))
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\t"
               "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(smem_addr(b)), "r"(parity) : "memory");
  return ok != 0;
}
// The same without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(smem_addr(b)), "r"(parity) : "memory");
  return ok != 0;
}

// ---------------------------------------------------------- tensor memory --
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Shared memory written by this thread becomes visible to the tensor cores.
__device__ __forceinline__ void fence_smem_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// 32 consecutive columns of this thread's lane (a warp reaches the 32 lanes of
// its quarter: lanes 32 (warp mod 4) .. + 31).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------- register shares ---
// A warpgroup's share of the registers that the block was launched with.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------- tensor cores ---
// Shared-memory matrix of 16-bit values in 128-byte rows, 8 rows per swizzle
// atom of 1024 bytes (16-byte chunk c of row r stored at chunk c ^ (r & 7)).
// `lead`: bytes between neighbouring 64-value panels (used when the panels lie
// along the operand's M or N dimension), atoms 1024 bytes apart. addr16: its
// shared-memory address / 16.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr16, uint32_t lead) {
  return (uint64_t)addr16 | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// f16 x f16 -> fp32, M = 128; b_mn: B's 128-byte rows run along N, not along K.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn) {
  return 1u << 4 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
// D[tmem] (+)= A[smem] B[smem], K = 16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                       bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
               "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// The same with A in tensor memory (two 16-bit values per column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc,
                                       bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
               "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// The barrier's phase counts one arrival when every MMA issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(b))
               : "memory");
}

// ------------------------------------- products with a scale per block -----
// Descriptor of the scales of 128 rows on their way to tensor memory: 32 lines
// of 16 bytes, line l holds the four bytes of rows l, l + 32, l + 64, l + 96.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr16) {
  return (uint64_t)addr16 | (uint64_t)(128u >> 4) << 32 | (uint64_t)1 << 46;
}
// Those 512 bytes into four columns of tensor memory (the same in each quarter
// of its lanes). Products issued after it by the same thread read them. With
// CG = 2 here and below, one thread acts for a pair of CTAs: each copies from
// its own shared memory to its own tensor memory.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}
// E2M1 x E2M1, a UE4M3 scale per 16 (K = 64), and E4M3 x E4M3, a UE8M0 scale per
// 32 (K = 32); M = 128 m, fp32 accumulators. byte: which of a column's four scale
// bytes the MXFP8 product takes. A pair of CTAs holds 128 rows of A and half of
// B's columns each, B's scales both, and gets its rows' results.
__host__ __device__ constexpr uint32_t nvfp4_mma_desc(int m, int n) {
  return 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m * 128 >> 4) << 24;
}
__host__ __device__ constexpr uint32_t mxfp8_mma_desc(int m, int n, int byte) {
  return (uint32_t)byte << 4 | (uint32_t)(n >> 3) << 17 | 1u << 23 |
         (uint32_t)(m * 128 >> 4) << 24 | (uint32_t)byte << 29;
}
#define NVFP4_SCALED_MMA(CG, KIND)                                            \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"              \
               "tcgen05.mma.cta_group::" CG ".kind::" KIND                   \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a),    \
               "l"(b), "r"(desc), "r"(sa), "r"(sb), "r"((uint32_t)add)       \
               : "memory")
template <int CG>
__device__ __forceinline__ void mma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                          uint32_t sa, uint32_t sb, bool add) {
  if constexpr (CG == 2) NVFP4_SCALED_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  else NVFP4_SCALED_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
}
template <int CG>
__device__ __forceinline__ void mma_mxfp8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                          uint32_t sa, uint32_t sb, bool add) {
  if constexpr (CG == 2) NVFP4_SCALED_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
  else NVFP4_SCALED_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
}
#undef NVFP4_SCALED_MMA

// ---------------------------------------------------------- pairs of CTAs ---
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared object of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
// An arrival at a barrier of another CTA of the cluster. What the caller wrote to
// its own shared memory is ordered before it by fence_smem_async, for the copies
// and products that its own SM then makes on the other CTA's behalf; a release of
// cluster scope would wait for everything that the thread has in flight (a stage
// of 128-value rows then took 2000 clocks where it takes 750).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mma_commit to the barrier at that place in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
               ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(b)), "h"((uint16_t)3)
               : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}

// ------------------------------------------------------------ tensor maps ---
// One arrival, and the phase waits for so many more bytes of copies.
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 t;\n\t"
               "mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(smem_addr(b)),
               "r"(bytes)
               : "memory");
}
// So many bytes that follow one another (a multiple of 16, both addresses too).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* b) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(b))
               : "memory");
}
// A box of a two-dimensional map, its first value at (x, y), to shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const void* map, int x, int y, uint64_t* b) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
               "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y),
               "r"(smem_addr(b))
               : "memory");
}
// The same whose bytes are counted by a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, int x, int y,
                                              uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
               ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map),
               "r"(x), "r"(y), "r"(bar)
               : "memory");
}

// A box of shared memory to global memory, a group of copies of its own.
__device__ __forceinline__ void tma_store(const void* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group "
               "[%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The thread's groups have read shared memory.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

}  // namespace nvfp4
