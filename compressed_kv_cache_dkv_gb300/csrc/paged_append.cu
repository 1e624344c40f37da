// dkv_paged_append: new K and V rows into their pages.
//
// A copy of 2 B Hkv n d 16-bit values, bound by memory (both directions).  One
// 16-byte piece per lane and access, the pieces of one token's heads side by side
// (a projection's output order), kAppendVec independent pieces per thread in
// flight; the page of a piece comes from the table through the read-only cache.
//
// Measured: prompts of 700 to 4096 tokens in 8 sequences, 8 KV heads, d 128 (166 MB read and written):
// 29.0 us, 5.7 TB/s.  One token for each of 16 sequences: 1.9 us in a graph, latency.
#include "paged.cuh"

namespace dkv {
namespace {

constexpr int kAppendThreads = 256, kAppendVec = 4;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(PagedArgs a, const uint4* __restrict__ K,
                                                                     const uint4* __restrict__ V, dkv_strides ns,
                                                                     int n_new, const int32_t* __restrict__ pos,
                                                                     const int32_t* __restrict__ counts,
                                                                     uint4* __restrict__ kp, uint4* __restrict__ vp) {
  constexpr int R = D / 8;  // pieces of a row
  const int b = blockIdx.y;
  const uint4* src = blockIdx.z ? V : K;
  uint4* dst = blockIdx.z ? vp : kp;
  int n = n_new;
  if (counts) {
    n = __ldg(counts + b);
    if (n < 0 || n > n_new) {
      if (threadIdx.x == 0) raise_error(a.err, DKV_DEVERR_INDEX);
      n = min(max(n, 0), n_new);
    }
  }
  const int64_t total = (int64_t)n * a.Hkv * R, p0 = __ldg(pos + b);
  const int64_t base = (int64_t)blockIdx.x * (kAppendThreads * kAppendVec) + threadIdx.x;
  if (base >= total) return;
  uint4 v[kAppendVec];
  int64_t to[kAppendVec];
  // row = i * Hkv + h of the thread's first piece; the next one is kStep rows on
  constexpr int kStep = kAppendThreads / R;
  const int c = (int)(base % R);
  int i = (int)(base / R / a.Hkv), h = (int)(base / R - (int64_t)i * a.Hkv);
  const int di = kStep / a.Hkv, dh = kStep - di * a.Hkv;
#pragma unroll
  for (int x = 0; x < kAppendVec; ++x, i += di, h += dh) {
    if (h >= a.Hkv) { h -= a.Hkv; ++i; }
    to[x] = -1;
    if (base + x * kAppendThreads >= total) continue;
    const int64_t t = p0 + i;
    if (t < 0 || t >= a.cap) {
      raise_error(a.err, DKV_DEVERR_INDEX);
      continue;
    }
    const int page = paged_page(a, b, (int)t);
    if (page >= a.n_pages) continue;
    v[x] = __ldg(src + (b * ns.batch + h * ns.head + i * ns.token) / 8 + c);
    to[x] = ((int64_t)page * a.stride_page + h * a.stride_head + ((int)t & a.page_mask) * a.stride_token) / 8 + c;
  }
#pragma unroll
  for (int x = 0; x < kAppendVec; ++x)
    if (to[x] >= 0) dst[to[x]] = v[x];
}

}  // namespace

cudaError_t launch_paged_append(const PagedArgs& a, int d, const void* K, const void* V, const dkv_strides& ns,
                                int n_new, const int32_t* pos, const int32_t* counts, void* k_pool, void* v_pool,
                                cudaStream_t s) {
  const int64_t per = kAppendThreads * kAppendVec, pieces = (int64_t)n_new * a.Hkv * (d / 8);
  const dim3 grid((unsigned)((pieces + per - 1) / per), a.B, 2);
  auto go = [&](auto kernel) {
    kernel<<<grid, kAppendThreads, 0, s>>>(a, static_cast<const uint4*>(K), static_cast<const uint4*>(V), ns, n_new, pos,
                                           counts, static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool));
  };
  if (d == 128) go(paged_append_kernel<128>);
  else go(paged_append_kernel<64>);
  return cudaGetLastError();
}

}  // namespace dkv
