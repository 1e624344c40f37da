// tcgen05 wrappers of the paged prefill and weights kernels: 128-byte-swizzled operands in
// shared memory, fp32 accumulators in tensor memory, 16-bit operands of one type.
#pragma once

#include "paged.cuh"

namespace dkv {

// Shared-memory descriptor of a 128-byte-swizzled operand.  K-major (rows of 64 channels): `sbo`
// is the stride of 8-row groups (1024), lbo unused.  MN-major (64 channels of the M or N axis a
// row, one row per k): `lbo` is the stride of the next 64 channels, `sbo` of the next 8 k (1024).
__device__ inline uint64_t tc_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3fffu) << 32) | (1ull << 46) | (2ull << 61);
}
// D fp32, A and B of format `fmt` (0 fp16, 1 bf16), A K-major, M = 128
__device__ constexpr uint32_t tc_idesc(uint32_t fmt, bool b_mn, uint32_t n) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
// The lane with `el` issues; the whole warp calls these with the same operands.
// A and B from shared memory
__device__ inline void tc_mma(uint32_t dt, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dt),
      "l"(ad), "l"(bd), "r"(id), "r"(acc), "r"(el)
      : "memory");
}
// A from tensor memory (row = lane, two elements of k a column)
__device__ inline void tc_mma_ta(uint32_t dt, uint32_t at, uint64_t bd, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dt),
      "r"(at), "l"(bd), "r"(id), "r"(acc), "r"(el)
      : "memory");
}
// arrive on `bar` when every product that lane has issued is done
__device__ inline void tc_commit(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
__device__ inline void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
template <int COLS>
__device__ inline void tc_alloc(uint32_t* slot) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "n"(COLS)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
__device__ inline void tc_free(uint32_t tmem) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS) : "memory");
}
// 32 consecutive columns of this thread's lane; tc_ld_wait before use
__device__ inline void tc_ld32(uint32_t ta, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta));
}
__device__ inline void tc_ld16(uint32_t ta, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta));
}
__device__ inline void tc_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ inline void tc_st16(uint32_t ta, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(ta),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ inline void tc_st8(uint32_t ta, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(ta), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ inline void tc_st32(uint32_t ta, const uint32_t* r) {
  tc_st16(ta, r);
  tc_st16(ta + 16, r + 16);
}
__device__ inline void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// named_bar_sync that tells whether x holds for any of the threads
__device__ inline bool named_bar_any(int id, int nthreads, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(nthreads), "r"((uint32_t)x)
      : "memory");
  return any != 0;
}

// two fp32 operations in one instruction (sm_100 and up)
__device__ inline uint64_t f2_bits(float2 x) { return *reinterpret_cast<uint64_t*>(&x); }
__device__ inline float2 fma2(float2 x, float2 y, float2 z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(x)), "l"(f2_bits(y)), "l"(f2_bits(z)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ inline float2 add2(float2 x, float2 y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(x)), "l"(f2_bits(y)));
  return *reinterpret_cast<float2*>(&r);
}

// The queries of one sequence.
struct QuerySpan {
  int len, n, off;  // tokens in the cache, queries, position of query 0 (negative: it sees nothing)
};
__device__ inline QuerySpan query_span(const PagedArgs& a, const int32_t* q_lens, int Tq, int b) {
  QuerySpan s;
  s.len = paged_len(a, b);
  s.n = Tq;
  if (q_lens) {
    s.n = __ldg(q_lens + b);
    if (s.n < 0 || s.n > Tq) {
      raise_error(a.err, DKV_DEVERR_INDEX);
      s.n = min(max(s.n, 0), Tq);
    }
  }
  s.off = s.len - s.n;
  return s;
}

// The keys that the queries at positions [p_lo, p_hi] see between them, in tiles of N.
template <int N>
struct KeySpan {
  int lo, hi, st, wt0, n;  // window start, end, sink tiles, first window tile, tiles
  __device__ int key(int j) const { return (j < st ? j : wt0 + j - st) * N; }
};
template <int N>
__device__ inline KeySpan<N> key_span(const PagedArgs& a, int p_lo, int p_hi) {
  KeySpan<N> s;
  s.hi = max(0, p_hi + 1);
  s.lo = min(paged_window_lo(a, max(p_lo, 0)), s.hi);
  s.wt0 = s.lo / N;
  s.st = min((min(a.sinks, s.hi) + N - 1) / N, s.wt0);
  s.n = s.st + (s.hi + N - 1) / N - s.wt0;
  return s;
}

}  // namespace dkv
