// Shared by the paged-cache kernels: arguments, visibility, page lookup, TMA box
// loads from the pools and the 16-bit helpers of both data types.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include "dkv_internal.cuh"

namespace dkv {

// What every paged kernel knows of the cache (passed by value).
struct PagedArgs {
  int B, Hq, Hkv, G, page_shift, page_mask, n_pages, max_pages, cap;  // cap: tokens a page-table row reaches
  int window, sinks;
  float scale_log2;  // log2(e) / sqrt(d)
  int64_t stride_page, stride_head, stride_token;  // elements
  const int32_t* __restrict__ table;
  const int32_t* __restrict__ lens;
  uint32_t* err;
};

// tokens of sequence b, brought into [0, cap]
__device__ inline int paged_len(const PagedArgs& a, int b) {
  const int n = __ldg(a.lens + b);
  if (n < 0 || n > a.cap) raise_error(a.err, DKV_DEVERR_INDEX);
  return min(max(n, 0), a.cap);
}

// first token of the sliding window of a query at position p (0 without a window)
__device__ inline int paged_window_lo(const PagedArgs& a, int p) {
  return a.window > 0 ? max(0, p - a.window + 1) : 0;
}

// Page of token t of sequence b; n_pages (a box outside the pool, which a TMA load
// fills with zeros) for a page index that is out of range.
__device__ inline int paged_page(const PagedArgs& a, int b, int t) {
  const int page = __ldg(a.table + (size_t)b * a.max_pages + (t >> a.page_shift));
  if (page >= 0 && page < a.n_pages) return page;
  raise_error(a.err, DKV_DEVERR_INDEX);
  return a.n_pages;
}

// ---------------------------------------------------------------------------
// Dealing tiles to CTAs: the tiles of all (sequence, KV head) units in a row, sequence by sequence
// and head by head, are cut into equal runs, one for each CTA.
// ---------------------------------------------------------------------------
// prefix[b] = tiles (of one head) of the sequences before b; every thread of the CTA calls it
template <typename F>
__device__ inline void deal_prefix(int B, int* prefix, F tiles_of) {
  __shared__ int wsum[32];
  __shared__ int carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) { carry = 0; prefix[0] = 0; }
  __syncthreads();
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int v = b < B ? tiles_of(b) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    int add = carry, all = carry;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) add += wsum[w];
      all += wsum[w];
    }
    if (b < B) prefix[b + 1] = v + add;
    __syncthreads();
    if (tid == 0) carry = all;
    __syncthreads();
  }
}
// The run of CTA c of n: tiles [deal_bound(c), deal_bound(c + 1)) of total.
__device__ inline int deal_bound(int total, int n, int c) { return (int)((int64_t)total * c / n); }
// The CTA whose run holds tile x.
__device__ inline int deal_owner(int total, int n, int x) { return (int)((((int64_t)x + 1) * n - 1) / total); }
// The unit of tile x, and its tiles up to x1.
struct DealSeg {
  int b, h, j0, j1, n;  // tiles [j0, j1) of the unit's n
};
__device__ inline DealSeg deal_seg(const int* prefix, int B, int Hkv, int x, int x1) {
  int lo = 0, hi = B - 1;  // the first b whose tiles end behind x
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (prefix[m + 1] * Hkv > x) hi = m;
    else lo = m + 1;
  }
  DealSeg s;
  s.b = lo;
  s.n = prefix[lo + 1] - prefix[lo];
  const int rem = x - prefix[lo] * Hkv;
  s.h = rem / s.n;
  s.j0 = rem - s.h * s.n;
  s.j1 = min(s.n, s.j0 + x1 - x);
  return s;
}

// ---------------------------------------------------------------------------
// Tiles in shared memory: per 64 channels a sub-tile of `rows` rows x 128 bytes,
// written by TMA boxes under the 128-byte swizzle (16-byte chunk index XOR row % 8;
// sub-tiles start on 1024-byte boundaries), so that eight rows of one chunk lie in
// eight different bank groups for ldmatrix and tcgen05.mma alike.
// ---------------------------------------------------------------------------
__device__ inline uint32_t sw128(uint32_t rows, uint32_t row, uint32_t chunk) {  // chunk: 8 channels
  return (chunk >> 3) * rows * 128u + row * 128u + (((chunk & 7u) ^ (row & 7u)) << 4);
}

// One lane of a converged warp (1 in it, 0 in the others).  Asynchronous copies and tensor-core
// instructions take their operands from uniform registers: they are issued by whole warps with the
// same operands in every lane, the elected one executing.  In code that runs lane by lane an issue
// takes 75 to 150 cycles.
__device__ inline uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// one box {64 channels, box rows} of head h of a pool: x = first channel (0 or 64), y = slot
__device__ inline void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int h, int page, uint64_t* bar,
                                   uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n\t}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(h), "r"(page), "r"(smem_u32(bar)), "r"(el)
      : "memory");
}
// the same under an L2 policy
__device__ inline void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int h, int page, uint64_t* bar,
                                   uint32_t el, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5}], [%6], %8;\n\t}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(h), "r"(page), "r"(smem_u32(bar)), "r"(el), "l"(policy)
      : "memory");
}
__device__ inline void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------
// fp16 / bf16
// ---------------------------------------------------------------------------
template <typename T>
struct Num;
template <>
struct Num<__half> {
  static constexpr uint32_t kUmma = 0;  // operand format field of the tcgen05 instruction descriptor
  static __device__ inline float to_float(__half x) { return __half2float(x); }
  static __device__ inline __half from_float(float x) { return __float2half_rn(x); }
  static __device__ inline uint32_t pack(float lo, float hi) { return pack_half2(lo, hi); }
  static __device__ inline void split(float x, float y, uint32_t& hi, uint32_t& lo) { split_half2(x, y, hi, lo); }
  // 0 x + z, two values
  static __device__ inline uint32_t zero_times(uint32_t x, uint32_t z) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(z));
    return r;
  }
  static __device__ inline void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    mma16816(c, a0, a1, a2, a3, b0, b1);
  }
};
template <>
struct Num<__nv_bfloat16> {
  static constexpr uint32_t kUmma = 1;
  static __device__ inline float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ inline __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
  static __device__ inline uint32_t pack(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ inline uint32_t zero_times(uint32_t x, uint32_t z) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(z));
    return r;
  }
  // hi + lo carries 16 bits of each value
  static __device__ inline void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    hi = *reinterpret_cast<uint32_t*>(&h);
    lo = pack(x - f.x, y - f.y);
  }
  static __device__ inline void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

__device__ inline uint4 ldsm_x4(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ inline uint4 ldsm_x4_trans(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ inline void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// a grid that may start before the one in front of it on the stream has finished, and calls
// griddep_wait() before it reads what that one wrote
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic_launch() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct PagedMaps {  // tensor maps of the pools: boxes of 64 channels x min(page_size, 64) slots
  CUtensorMap k, v;
};

// decode: workspace [header][records: two per CTA, fp32 m[8] l[8] o[d][8]]; scores fp32 [units][cap][8]
size_t paged_decode_ws_bytes(int d);
cudaError_t launch_paged_decode(const PagedArgs& a, int d, int dtype, const PagedMaps& m, const void* q,
                                const dkv_strides& qs, void* out, float* lse, float* weights, float* scores, uint8_t* ws,
                                cudaStream_t s);
cudaError_t launch_paged_append(const PagedArgs& a, int d, const void* K, const void* V, const dkv_strides& ns,
                                int n_new, const int32_t* pos, const int32_t* counts, void* k_pool, void* v_pool,
                                cudaStream_t s);
// prefill and weights: qmap boxes of 64 channels x paged_prefill_rows(Tq) tokens of q (weights: x
// paged_weights_rows(G, Tq))
struct PagedQuery {
  const void* q;
  dkv_strides qs;
  int Tq;
  const int32_t* q_lens;
};
cudaError_t launch_paged_prefill(const PagedArgs& a, int d, int dtype, const PagedMaps& m, const CUtensorMap& qmap,
                                 const PagedQuery& q, const void* v_pool, const void* k_pool, void* out,
                                 const dkv_strides& os, float* lse, uint8_t* ws, cudaStream_t s);
int paged_prefill_rows(int Tq);
size_t paged_prefill_ws_bytes(int d);
int paged_weights_rows(int G, int Tq);
cudaError_t launch_paged_weights(const PagedArgs& a, int d, int dtype, const CUtensorMap& kmap, const CUtensorMap& qmap,
                                 const PagedQuery& q, const float* lse, float* weights, cudaStream_t s);
size_t paged_evict_ws_bytes(const PagedArgs& a, int d);
struct PagedEvict {
  int budget, first, recent, new_max_pages;
  const float* weights;
  const int32_t* new_table;
  int32_t* kept;
  int32_t* new_lens;
  float* new_weights;
};
cudaError_t launch_paged_evict(const PagedArgs& a, int d, const PagedEvict& e, void* k_pool, void* v_pool, uint8_t* ws,
                               cudaStream_t s);

}  // namespace dkv
