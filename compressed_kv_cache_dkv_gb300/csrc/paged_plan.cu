// dkv_paged_plan: pages, slots and positions of a step's new tokens, from the requests' lengths.
//
// Everything follows from prefix sums over the requests (pages given back, pages needed, tokens), so one CTA
// makes those and every other value is found from its index: the k-th page handed out is entry top - 1 - k of
// the free list with the pages given back behind it, a row's request is the one whose span of rows holds it
// (a binary search in shared memory).  A page that one request gives back and another takes is read from the
// giver's row of the table, which this call does not write, so that no order among the CTAs is needed.
//
// A step of few rows is one grid of one CTA, bound by its latency; more rows go to a second grid over all
// multiprocessors, which writes 12 bytes for each.
//
// Measured: one token for each of 64 requests 4.3 us in a graph; 256 requests into a million rows (12.6 MB, most of them
// padding) 12.4 us, 10.8 in a graph, of which the sums 4 and the second grid's start and shared copy of the sums 3 (14.2 with
// 1024 threads for the sums).
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kPlanThreads = 1024, kPlanMost = 4;  // requests of a thread at most: 4096 in all
constexpr int kPlanFew = 256;                      // threads for as many requests, and for their rows where one CTA writes them
constexpr int kPlanRows = 4;                       // rows of a thread
constexpr int kPlanAlone = 8192;                   // rows that one CTA takes

// What the prefix sums leave: rows, pages needed and pages given back before each request, its old length.
struct PlanSums {
  int* starts;  // [B + 1]
  int* need;    // [B + 1]
  int* back;    // [B + 1]
  int* lens;    // [B]
};
__host__ __device__ inline PlanSums plan_sums(int* at, int B) { return {at, at + B + 1, at + 2 * (B + 1), at + 3 * (B + 1)}; }
__host__ __device__ inline int plan_ints(int B) { return 4 * (B + 1); }

struct Plan {
  PlanArgs a;
  PlanSums s;
  int n_free, top;  // of the list, without and with the pages given back
  bool vec;         // slots and positions begin on 16-byte boundaries

  __device__ int pages_of(int n) const { return (n >> a.page_shift) + ((n & ((1 << a.page_shift) - 1)) != 0); }
  // the request whose span of `cum` holds x < cum[B]
  __device__ int owner(const int* cum, int x) const {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int m = (lo + hi) >> 1;
      if (cum[m + 1] > x) hi = m;
      else lo = m + 1;
    }
    return lo;
  }
  // the r-th page given back
  __device__ int returned(int r) const {
    const int b = owner(s.back, r), keep = pages_of(s.lens[b]) - (s.back[b + 1] - s.back[b]);
    return __ldcg(a.table + (int64_t)b * a.max_pages + keep + r - s.back[b]);
  }
  // the k-th page handed out
  __device__ int page(int k) const {
    const int at = top - 1 - k;
    return at < n_free ? __ldcg(a.free_pages + at) : returned(at - n_free);
  }
  // slots and positions of rows i0 .. i0 + kPlanRows - 1
  __device__ void fill(int64_t i0) const {
    const int live = s.starts[a.B];
    int b = i0 < live ? owner(s.starts, (int)i0) : a.B;
    int64_t slot[kPlanRows];
    int pos[kPlanRows];
#pragma unroll
    for (int x = 0; x < kPlanRows; ++x) {
      const int64_t i = i0 + x;
      slot[x] = -1;
      pos[x] = -1;
      if (i >= live) continue;
      while (i >= s.starts[b + 1]) ++b;
      const int len = s.lens[b], t = len + (int)i - s.starts[b], have = pages_of(len), j = t >> a.page_shift;
      const int pg = j < have ? __ldcg(a.table + (int64_t)b * a.max_pages + j) : page(s.need[b] + j - have);
      pos[x] = t;
      if (pg >= 0 && pg < a.n_pages) slot[x] = ((int64_t)pg << a.page_shift) + (t & ((1 << a.page_shift) - 1));
      else raise_error(a.err, DKV_DEVERR_INDEX);
    }
    if (vec && i0 + kPlanRows <= a.rows) {
      static_assert(kPlanRows == 4, "two 16-byte stores of slots, one of positions");
      *reinterpret_cast<longlong2*>(a.slots + i0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slots + i0 + 2) = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      return;
    }
#pragma unroll
    for (int x = 0; x < kPlanRows; ++x)
      if (i0 + x < a.rows) {
        a.slots[i0 + x] = slot[x];
        a.positions[i0 + x] = pos[x];
      }
  }
  // the table's new entries and the list's, and all rows, by `n` threads
  __device__ void write(int64_t tid, int64_t n) const {
    for (int64_t k = tid; k < s.need[a.B]; k += n) {
      const int b = owner(s.need, (int)k);
      a.table[(int64_t)b * a.max_pages + pages_of(s.lens[b]) + k - s.need[b]] = page((int)k);
    }
    for (int64_t r = tid; r < s.back[a.B]; r += n) {
      const int pg = returned((int)r);
      if (pg < 0 || pg >= a.n_pages) raise_error(a.err, DKV_DEVERR_INDEX);
      if (n_free + r < a.free_cap) a.free_pages[n_free + r] = pg;
      else if (n_free + r < top - s.need[a.B]) raise_error(a.err, DKV_DEVERR_INDEX);  // no room for it in the list
    }
    for (int64_t i = tid * kPlanRows; i < a.rows; i += n * kPlanRows) fill(i);
  }
};

// exclusive prefix sums over a CTA of THREADS of N values a thread, and their totals
template <int THREADS, int N>
__device__ inline void block_sums(int64_t (&v)[N], int64_t (&total)[N]) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int64_t part[N][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 31) part[i][warp] = x[i];
  }
  __syncthreads();
  if (warp < N) {
    int64_t y = lane < kWarps ? part[warp][lane] : 0;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane < kWarps) part[warp][lane] = y;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = x[i] - v[i] + (warp ? part[i][warp - 1] : 0);
    total[i] = part[i][kWarps - 1];
  }
}
// two counts in one sum (each stays below 2^31: 4096 requests of at most 65536 pages, 2^30 rows)
__device__ inline int64_t both(int hi, int lo) { return ((int64_t)hi << 32) | (uint32_t)lo; }

template <int THREADS>
__global__ void __launch_bounds__(THREADS) plan_kernel(PlanArgs a, int* ws, int alone, bool vec) {
  extern __shared__ int sums[];
  constexpr int kMost = THREADS == kPlanThreads ? kPlanMost : 1;
  if (!alone) griddep_launch();  // the grid that writes
  Plan p;
  p.a = a;
  p.vec = vec;
  p.s = plan_sums(alone ? sums : ws, a.B);
  const int per = (a.B + THREADS - 1) / THREADS, b0 = threadIdx.x * per;
  const int cap = a.max_pages << a.page_shift;
  int n_free = __ldcg(a.n_free);
  if (n_free < 0 || n_free > a.free_cap) {
    if (threadIdx.x == 0) raise_error(a.err, DKV_DEVERR_INDEX);
    n_free = min(max(n_free, 0), a.free_cap);
  }
  int len[kMost], cut[kMost], grow[kMost];
  int64_t v[2] = {0, 0}, all[2];  // pages given back and pages needed; tokens
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int b = b0 + i;
    len[i] = cut[i] = grow[i] = 0;
    if (i >= per || b >= a.B) continue;
    const int n = __ldcg(a.lens + b), m = __ldcg(a.news + b);
    len[i] = min(max(n, 0), cap);
    const bool fits = m <= cap - len[i];
    if (m < 0) cut[i] = m < -len[i] ? len[i] : -m;
    else if (fits) grow[i] = m;
    if (n != len[i] || !fits || m < -len[i]) raise_error(a.err, DKV_DEVERR_INDEX);
    v[0] += both(p.pages_of(len[i]) - p.pages_of(len[i] - cut[i]), p.pages_of(len[i] + grow[i]) - p.pages_of(len[i]));
    v[1] += grow[i];
  }
  block_sums<THREADS>(v, all);
  const int all_back = (int)(all[0] >> 32);
  p.n_free = n_free;
  p.top = n_free + all_back;
  int give[kMost];  // tokens granted
  int back = (int)(v[0] >> 32), asked = (int)v[0];
  int64_t rows = v[1], w[1] = {0}, sum[1];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int need = p.pages_of(len[i] + grow[i]) - p.pages_of(len[i]);
    asked += need;
    rows += grow[i];
    give[i] = (need == 0 || asked <= p.top) && rows <= a.rows ? grow[i] : 0;
    w[0] += both(give[i], give[i] ? need : 0);
  }
  __syncthreads();
  block_sums<THREADS>(w, sum);
  const int all_rows = (int)(sum[0] >> 32), all_need = (int)sum[0];
  int start = (int)(w[0] >> 32), taken = (int)w[0];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= a.B) continue;
    p.s.starts[b] = start;
    p.s.need[b] = taken;
    p.s.back[b] = back;
    p.s.lens[b] = len[i];
    a.starts[b] = start;
    a.granted[b] = give[i];
    a.new_lens[b] = len[i] - cut[i] + give[i];
    start += give[i];
    taken += p.pages_of(len[i] + give[i]) - p.pages_of(len[i]);
    back += p.pages_of(len[i]) - p.pages_of(len[i] - cut[i]);
  }
  if (threadIdx.x == 0) {
    p.s.starts[a.B] = a.starts[a.B] = all_rows;
    p.s.need[a.B] = all_need;
    p.s.back[a.B] = all_back;
    p.s.lens[a.B] = n_free;
    *a.new_n_free = min(p.top - all_need, a.free_cap);
  }
  __syncthreads();
  if (alone) p.write(threadIdx.x, THREADS);
}

__global__ void __launch_bounds__(256) plan_write_kernel(PlanArgs a, const int* ws, bool vec) {
  extern __shared__ int sums[];
  griddep_wait();
  for (int i = threadIdx.x; i < plan_ints(a.B); i += blockDim.x) sums[i] = __ldcg(ws + i);
  __syncthreads();
  Plan p;
  p.a = a;
  p.vec = vec;
  p.s = plan_sums(sums, a.B);
  p.n_free = p.s.lens[a.B];
  p.top = p.n_free + p.s.back[a.B];
  p.write((int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

}  // namespace

size_t plan_ws_bytes(int B) { return kWsHeader + round_up((size_t)plan_ints(B) * 4, 256); }

cudaError_t launch_paged_plan(const PlanArgs& a, uint8_t* ws, cudaStream_t s) {
  int* sums = reinterpret_cast<int*>(ws + kWsHeader);
  const size_t smem = (size_t)plan_ints(a.B) * 4;
  const bool alone = a.rows <= kPlanAlone, few = a.B <= kPlanFew && (!alone || a.rows <= kPlanFew * kPlanRows);
  const bool vec = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  cudaError_t e = ensure_smem_limit(few ? reinterpret_cast<const void*>(plan_kernel<kPlanFew>) : reinterpret_cast<const void*>(plan_kernel<kPlanThreads>), smem);
  if (e != cudaSuccess) return e;
  if (few) plan_kernel<kPlanFew><<<1, kPlanFew, smem, s>>>(a, sums, alone, vec);
  else plan_kernel<kPlanThreads><<<1, kPlanThreads, smem, s>>>(a, sums, alone, vec);
  if ((e = cudaGetLastError()) != cudaSuccess || alone) return e;
  if ((e = ensure_smem_limit(reinterpret_cast<const void*>(plan_write_kernel), smem)) != cudaSuccess) return e;
  const int64_t most = ((int64_t)a.rows + 256 * kPlanRows - 1) / (256 * kPlanRows);
  return launch_dependent(plan_write_kernel, dim3((unsigned)(most < 4 * sm_count() ? most : 4 * sm_count())), 256, smem, s, a, (const int*)sums, vec);
}

}  // namespace dkv
