// dkv_paged_evict: keep the heaviest tokens of every (sequence, KV head) and move them
// together.
//
// select: the k-th largest weight of a unit by radix selection over an order-preserving
// integer image of the weights (three passes of 11, 11 and 10 bits, a histogram in shared
// memory each), then one ordered pass that writes the kept positions, ascending.
// compact: kept rows to positions 0, 1, ...  Position j is filled from a position >= j, so
// a CTA that walks its rows in order, reading a batch before it writes it, can compact in
// place; the CTAs of a unit split the row's bytes, never its tokens.
#include "paged.cuh"

namespace dkv {
namespace {

constexpr int kSelThreads = 1024, kSelBins = 2048;
constexpr int kMoveThreads = 256, kMoveRows = 8;  // rows in flight per thread
constexpr int kMovePiece = 64;                    // bytes of a row one CTA moves

// a < b as floats iff image(a) < image(b); -0 is 0, NaN is -infinity
__device__ inline uint32_t weight_image(float w) {
  if (isnan(w)) w = -INFINITY;
  if (w == 0.f) w = 0.f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(PagedArgs a, PagedEvict e, int32_t* __restrict__ counts) {
  __shared__ int hist[kSelBins];
  __shared__ int wsum[32];
  __shared__ int sh_digit, sh_above;
  const int u = blockIdx.x, b = u / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = paged_len(a, b), n = min(len, e.budget);
  int32_t* kept = e.kept + (size_t)u * e.budget;
  if (u % a.Hkv == 0 && tid == 0) counts[b] = n;
  for (int j = n + tid; j < e.budget; j += kSelThreads) kept[j] = -1;
  if (len <= e.budget) {
    for (int j = tid; j < n; j += kSelThreads) kept[j] = j;
    return;
  }
  // candidates [c0, c1); the tokens around them stay whatever they weigh
  const int c0 = e.first, c1 = len - e.recent;
  const float* w = e.weights + (size_t)u * a.cap;
  int k = e.budget - e.first - e.recent;  // candidates to keep: 0 <= k < c1 - c0
  uint32_t thr = 0, mask = 0;             // the k-th largest image, found from its high bits down
  if (k > 0) {
    const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
    for (int p = 0; p < 3; ++p) {
      const int bins = 1 << bits[p];
      for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = c0 + tid; t < c1; t += kSelThreads) {
        const uint32_t x = weight_image(__ldg(w + t));
        if ((x & mask) == thr) atomicAdd(&hist[(x >> shift[p]) & (bins - 1)], 1);
      }
      __syncthreads();
      // the digit with fewer than k images above it and at least k down to it: thread i takes
      // bins - 1 - (per i), ... downwards
      const int per = (bins + kSelThreads - 1) / kSelThreads, top = bins - 1 - tid * per;
      int sum = 0;
      for (int i = 0; i < per && top - i >= 0; ++i) sum += hist[top - i];
      int scan = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      if (lane == 31) wsum[warp] = scan;
      __syncthreads();
      int above = scan - sum;
      for (int i = 0; i < warp; ++i) above += wsum[i];
      if (above < k && above + sum >= k) {
        int i = 0;
        while (above + hist[top - i] < k) above += hist[top - i++];
        sh_digit = top - i;
        sh_above = above;
      }
      __syncthreads();
      thr |= (uint32_t)sh_digit << shift[p];
      mask |= (uint32_t)(bins - 1) << shift[p];
      k -= sh_above;  // still to find among the images that share thr's high bits
      __syncthreads();
    }
  }
  // every image above thr stays, and the first k that equal it (none when no candidate stays)
  const bool any = e.budget > e.first + e.recent;
  int out = 0, ties = 0;  // kept positions and equal images of the chunks before
  for (int base = 0; base < len; base += kSelThreads) {
    const int t = base + tid;
    int keep = 0, tie = 0;
    if (t < len) {
      if (t < c0 || t >= c1) keep = 1;
      else if (any) {
        const uint32_t x = weight_image(__ldg(w + t));
        keep = x > thr;
        tie = x == thr;
      }
    }
    // both counts at once: ties of the chunk before this token, then kept ones
    auto scan_excl = [&](int v, int* total) {
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      __syncthreads();
      if (lane == 31) wsum[warp] = s;
      __syncthreads();
      int before = s - v, all = 0;
      for (int i = 0; i < 32; ++i) {
        if (i < warp) before += wsum[i];
        all += wsum[i];
      }
      *total = all;
      return before;
    };
    int nt, nk;
    const int tb = scan_excl(tie, &nt);
    if (tie && ties + tb < k) keep = 1;
    const int kb = scan_excl(keep, &nk);
    if (keep) kept[out + kb] = t;
    ties += nt;
    out += nk;
  }
}

// grid (units, 2 * row bytes / kMovePiece + 1): K pieces, V pieces, the weights
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(PagedArgs a, PagedEvict e, int pieces,
                                                                 uint8_t* __restrict__ kp, uint8_t* __restrict__ vp,
                                                                 const int32_t* __restrict__ counts) {
  const int u = blockIdx.x, b = u / a.Hkv, h = u % a.Hkv, tid = threadIdx.x;
  const int n = __ldg(counts + b);
  const int32_t* kept = e.kept + (size_t)u * e.budget;
  if ((int)blockIdx.y == 2 * pieces) {
    const float* w = e.weights + (size_t)u * a.cap;
    float* nw = e.new_weights + (size_t)u * a.cap;
    for (int j0 = 0; j0 < n; j0 += kMoveThreads * kMoveRows) {
      float v[kMoveRows];
#pragma unroll
      for (int x = 0; x < kMoveRows; ++x) {
        const int j = j0 + x * kMoveThreads + tid;
        if (j < n) v[x] = __ldcg(w + __ldg(kept + j));
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < kMoveRows; ++x) {
        const int j = j0 + x * kMoveThreads + tid;
        if (j < n) nw[j] = v[x];
      }
    }
    for (int j = n + tid; j < a.cap; j += kMoveThreads) nw[j] = 0.f;
    if (h == 0 && tid == 0) e.new_lens[b] = n;
    return;
  }
  uint8_t* pool = (int)blockIdx.y < pieces ? kp : vp;
  constexpr int kLanes = kMovePiece / 16, kRows = kMoveThreads / kLanes;  // rows of one access
  const int64_t col = (int64_t)(blockIdx.y % pieces) * kMovePiece + (tid % kLanes) * 16 + h * a.stride_head * 2;
  for (int j0 = 0; j0 < n; j0 += kRows * kMoveRows) {
    uint4 v[kMoveRows];
    uint8_t* to[kMoveRows];
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      const int j = j0 + x * kRows + tid / kLanes;
      to[x] = nullptr;
      if (j >= n) continue;
      const int t = __ldg(kept + j), sp = paged_page(a, b, t);
      const int dp = __ldg(e.new_table + (size_t)b * e.new_max_pages + (j >> a.page_shift));
      if (dp < 0 || dp >= a.n_pages) {
        raise_error(a.err, DKV_DEVERR_INDEX);
        continue;
      }
      v[x] = make_uint4(0, 0, 0, 0);
      if (sp < a.n_pages)
        v[x] = __ldcg(reinterpret_cast<const uint4*>(pool + col + (sp * a.stride_page + (t & a.page_mask) * a.stride_token) * 2));
      to[x] = pool + col + (dp * a.stride_page + (j & a.page_mask) * a.stride_token) * 2;
    }
    __syncthreads();  // the batch is read: its positions may be written
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x)
      if (to[x]) *reinterpret_cast<uint4*>(to[x]) = v[x];
  }
}

}  // namespace

size_t paged_evict_ws_bytes(const PagedArgs& a) { return kWsHeader + (size_t)a.B * 4; }

cudaError_t launch_paged_evict(const PagedArgs& a, int d, const PagedEvict& e, void* k_pool, void* v_pool, uint8_t* ws,
                               cudaStream_t s) {
  int32_t* counts = reinterpret_cast<int32_t*>(ws + kWsHeader);
  const int units = a.B * a.Hkv, pieces = d * 2 / kMovePiece;
  evict_select_kernel<<<units, kSelThreads, 0, s>>>(a, e, counts);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  evict_move_kernel<<<dim3(units, 2 * pieces + 1), kMoveThreads, 0, s>>>(a, e, pieces, static_cast<uint8_t*>(k_pool),
                                                                         static_cast<uint8_t*>(v_pool), counts);
  return cudaGetLastError();
}

}  // namespace dkv
