// dkv_paged_weights: softmax weights summed by key, weights[t] += sum over queries of
// 2^(c q.k_t - lse), on the tcgen05 tensor cores.
//
// S^T = K Q^T for 128 keys and up to 128 query columns puts one key into each TMEM lane: a thread
// sums its key's weights over the columns in registers, every key has one owner, and the order is
// fixed (no atomics).  Four warpgroups sum, each with 128 TMEM columns of its own (with two, the
// latencies of a column's load, lse and exponential stayed in view); warp 16 streams operands with
// TMA, warp 17 issues the products.
//
// Few queries (those of all heads of a group fit 128 columns, padded to 16, 32, 64 or 128 a head):
// a unit's column tile stays while its key tiles are streamed, to the warpgroups in turn; the key
// tiles of all units are dealt out evenly to one CTA per multiprocessor.  Bound by the read of K.
// Many queries: 256 keys stay, two warpgroups in turn to 128 of them, and the query tiles of one
// head after the other are streamed past; a cluster of kCluster CTAs shares the queries of its keys
// and adds the parts in rank order, since the first keys of a prompt are seen by all its queries
// and would take many times the average.  Products and exponentials take 1024 cycles each for 256 keys x
// 128 queries at d 128, and both pipes are busy 55 % of the time: what bounds it is a step's chain of scores,
// lse and exponentials, and the uneven last wave.
//
// Measured (d 128): the last 32 queries of 8 prompts of 2000 to 8192 tokens, 8 KV heads (92 MB): 27 us,
// of which 14 the read, the rest the start and the end.  A prompt of 8192 with all its queries, 12
// heads: 90 to 91 us, 1.13 PFLOP/s.
#include "paged_tc.cuh"

namespace dkv {
namespace {

constexpr int kWtThreads = 576, kWtM = 128, kWtN = 128;  // keys, query columns of a tile at most
constexpr int kCluster = 4;  // CTAs that share the queries of their keys (eight leave a fifth of the GPU's
                             // multiprocessors without a cluster: 125 us for an 8k prompt, four 93 us)
constexpr int kStay = 2, kSlots = 4;  // operand tiles in shared memory: those that stay, and the streamed ones'

template <int D>
struct WtSmem {
  static constexpr uint32_t kTile = 128 * D * 2;                     // 128 keys or query rows
  static constexpr uint32_t kOffSlots = kStay * kTile;
  static constexpr uint32_t kOffLse = kOffSlots + kSlots * kTile;    // [warpgroup][128] minus base-2 lse
  static constexpr uint32_t kOffRank = kOffLse + 4 * kWtN * 4;       // [block % 2][rank][256] sums of the cluster
  static constexpr uint32_t kOffBar = kOffRank + 2 * kCluster * 2 * kWtM * 4;
  static constexpr uint32_t kOffPrefix = kOffBar + 256;              // [B + 1] (few queries)
};

struct WtArgs {
  PagedArgs a;
  PagedQuery q;
  const float* lse;
  float* weights;
  int rows;  // query rows of a box: a head's columns
};

struct WtBars {
  uint64_t *stay_full, *stay_empty, *full, *empty, *s_full, *s_empty;  // [kStay] x 2, [kSlots] x 2, [warpgroup] x 2
  uint64_t* drain;
  uint32_t* tmem_slot;
};

// barriers and tensor memory; returns its address
template <int D>
__device__ inline uint32_t wt_start(uint8_t* smem, WtBars& b, const CUtensorMap* kmap, const CUtensorMap* qmap) {
  b.stay_full = reinterpret_cast<uint64_t*>(smem + WtSmem<D>::kOffBar);
  b.stay_empty = b.stay_full + kStay;
  b.full = b.stay_empty + kStay;
  b.empty = b.full + kSlots;
  b.s_full = b.empty + kSlots;
  b.s_empty = b.s_full + 4;
  b.drain = b.s_empty + 4;
  b.tmem_slot = reinterpret_cast<uint32_t*>(b.drain + 1);
  if (threadIdx.x == 0) {
    tma_prefetch_map(kmap);
    tma_prefetch_map(qmap);
    for (int i = 0; i < 2 * (kStay + kSlots); ++i) mbar_init(&b.stay_full[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.s_empty[i], 128);
    }
    mbar_init(b.drain, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 32) tc_alloc<512>(b.tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *b.tmem_slot;
}
// a wait of the issuing warp gave up, and the sums' may have too: no product outlives the CTA
__device__ inline void wt_drain(const WtBars& b, uint32_t* err, uint32_t el) {
  tc_commit(b.drain, el);
  mbar_wait(b.drain, 0, err);
}
__device__ inline void wt_end(uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x < 32) tc_free<512>(tmem);
}

// Lane i: the page of the i-th run of `rows` keys from key k0 on that is seen by a query from
// window start k_lo on (n_pages, a box of zeros, for a run without a visible key, wherever the table
// points).
__device__ inline int wt_page(const PagedArgs& a, int b, int len, int k_lo, int k0, int rows) {
  const int first = k0 + (threadIdx.x & 31) * rows;
  return (int)(threadIdx.x & 31) * rows < kWtM && first < len && (first + rows > k_lo || first < a.sinks) ? paged_page(a, b, first)
                                                                                                    : a.n_pages;
}
// a tile of 128 keys; whole warp, `page` from wt_page
template <int D>
__device__ inline void wt_load_keys(const PagedArgs& a, const CUtensorMap* kmap, int h, int k0, int rows, int page, uint32_t to,
                                    uint64_t* bar, uint32_t el) {
#pragma unroll 4
  for (int i = 0; i < kWtM / rows; ++i) {
    const int pg = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
      tma_load_4d(to + hf * kWtM * 128 + i * rows * 128, kmap, hf * 64, (k0 + i * rows) & a.page_mask, h, pg, bar, el);
  }
}
// `m` heads' boxes of qn query rows, side by side in one tile; whole warp
template <int D>
__device__ inline void wt_load_queries(const CUtensorMap* qmap, int b, int head, int m, int row, int qn, uint32_t to, uint64_t* bar,
                                       uint32_t el) {
  if (el) mbar_arrive_expect_tx(bar, (uint32_t)(m * qn) * D * 2);
  for (int x = 0; x < m; ++x)
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
      tma_load_4d(to + hf * m * qn * 128 + x * qn * 128, qmap, hf * 64, row, head + x, b, bar, el);
}
// S^T of the key tile and the query tile of ncol columns at these addresses; whole warp
template <int D>
__device__ inline void wt_product(uint32_t td, uint32_t key, uint32_t query, int ncol, uint32_t id, uint32_t el) {
  const uint64_t kd = tc_desc(key, 16, 1024), qd = tc_desc(query, 16, 1024), half = (uint64_t)(ncol * 128 >> 4);
  tc_fence_after();
#pragma unroll
  for (int c = 0; c < D / 16; ++c)  // 16 channels: 32 bytes of a 128-byte row, then the next 64 channels
    tc_mma(td, kd + (uint64_t)(((c >> 2) * kWtM * 128 + (c & 3) * 32) >> 4), qd + (c >> 2) * half + (uint64_t)((c & 3) * 32 >> 4), id,
           c > 0, el);
}
// minus the base-2 log-sum-exp (-inf for a column without a query, so that it adds 0)
__device__ inline float wt_minus_lse2(float lse) { return lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f; }

// Adds to acc the weights of this thread's key t over the columns at TMEM address ts: query rows r0 on
// of head after head, qn columns each, with l2 their minus base-2 lse; `left_out`: it is -inf for some,
// which add nothing whatever their scores are (NaN, for a row that nothing has written).  Waits for the
// scores and gives the columns back.
__device__ inline bool wt_sum(const PagedArgs& a, const QuerySpan& qs, uint32_t ts, int ncol, int qn, int r0, int t, const float* l2, bool left_out,
                              uint64_t* s_full, uint64_t* s_empty, uint32_t parity, float2 (&acc)[2], bool ok) {
  // rows [v_lo, v_hi) of each head see this key
  const int v_lo = max(t - qs.off - r0, 0);
  int v_hi = min(qn, qs.n - r0);
  if (a.window > 0 && t >= a.sinks) v_hi = (int)max((int64_t)0, min((int64_t)v_hi, (int64_t)t + a.window - qs.off - r0));
  const bool all = ncol == kWtN && !left_out && __all_sync(0xffffffffu, v_lo == 0 && v_hi == qn);
  if (ok) ok = mbar_wait(s_full, parity, a.err);
  tc_fence_after();
  if (all) {  // every column counts
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
    for (int c = 0; c < kWtN / 32; ++c) {
      uint32_t s[32];
      tc_ld32(ts + 32 * c, s);
      float4 m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = *reinterpret_cast<const float4*>(l2 + 32 * c + 4 * e);
      tc_ld_wait();
      if (c + 1 == kWtN / 32) {
        tc_fence_before();
        mbar_arrive(s_empty);
      }
      float2 y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        y[e] = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2,
                    e & 1 ? make_float2(m[e >> 1].z, m[e >> 1].w) : make_float2(m[e >> 1].x, m[e >> 1].y));
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = make_float2(fast_exp2(y[e].x), fast_exp2(y[e].y));
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = add2(y[e], y[e + 8]);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = add2(y[e], y[e + 4]);
      acc[0] = add2(acc[0], add2(y[0], y[2]));
      acc[1] = add2(acc[1], add2(y[1], y[3]));
    }
    return ok;
  }
#pragma unroll 1
  for (int c = 0; c < ncol; c += 16) {
    const int r1 = c & (qn - 1);  // (qn is a power of two, 16 at least: the chunk lies in one head)
    if (!__any_sync(0xffffffffu, v_lo < r1 + 16 && v_hi > r1)) continue;
    uint32_t s[16];
    tc_ld16(ts + c, s);
    tc_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float m = l2[c + e], x = fast_exp2(fmaf(__uint_as_float(s[e]), a.scale_log2, m));
      acc[e & 1].x += r1 + e >= v_lo && r1 + e < v_hi && m != -INFINITY ? x : 0.f;  // (what lies in a hidden column is not looked at)
    }
  }
  tc_fence_before();
  mbar_arrive(s_empty);
  return ok;
}
__device__ inline float wt_total(const float2 (&acc)[2]) { return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y); }

// ---------------------------------------------------------------- few queries
template <typename T, int D>
__global__ void __launch_bounds__(kWtThreads, 1)
    paged_weights_few_kernel(WtArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = WtSmem<D>;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, qn = p.rows, ncol = a.G * qn;
  int* prefix = reinterpret_cast<int*>(smem + S::kOffPrefix);
  auto span_of = [&](int b) {
    const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, b);
    return qs.n > 0 ? key_span<kWtM>(a, qs.off, qs.len - 1) : KeySpan<kWtM>{0, 0, 0, 0, 0};
  };
  deal_prefix(a.B, prefix, [&](int b) { return span_of(b).n; });
  __syncthreads();
  const int total = prefix[a.B] * a.Hkv, nc = min((int)gridDim.x, total);
  if ((int)blockIdx.x >= nc) return;
  const int x0 = deal_bound(total, nc, blockIdx.x), x1 = deal_bound(total, nc, blockIdx.x + 1);
  WtBars bar;
  const uint32_t tmem = wt_start<D>(smem, bar, &kmap, &qmap), sb = smem_u32(smem), slots = sb + S::kOffSlots;
  bool ok = true;

  if (warp == 16) {
    // =========================== loads
    const uint32_t el = elect_one();
    const int rows = min(a.page_mask + 1, 64);
    auto wait = [&](uint64_t* b, int parity) { return ok = __all_sync(0xffffffffu, ok && mbar_wait(b, (uint32_t)parity, a.err)); };
    int i = 0, seg = 0;
    for (int x = x0; x < x1 && ok; ++seg) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
      const KeySpan<kWtM> ks = span_of(g.b);
      int page = wt_page(a, g.b, ks.hi, ks.lo, ks.key(g.j0), rows);
      if (seg >= kStay && !wait(&bar.stay_empty[seg % kStay], (seg / kStay - 1) & 1)) break;
      wt_load_queries<D>(&qmap, g.b, g.h * a.G, a.G, 0, qn, sb + (seg % kStay) * S::kTile, &bar.stay_full[seg % kStay], el);
      for (int j = g.j0; j < g.j1; ++j, ++i) {
        const int sl = i % kSlots;
        const int next = j + 1 < g.j1 ? wt_page(a, g.b, ks.hi, ks.lo, ks.key(j + 1), rows) : 0;  // a tile ahead of its use
        if (i >= kSlots && !wait(&bar.empty[sl], (i / kSlots - 1) & 1)) break;
        if (el) mbar_arrive_expect_tx(&bar.full[sl], S::kTile);
        wt_load_keys<D>(a, &kmap, g.h, ks.key(j), rows, page, slots + sl * S::kTile, &bar.full[sl], el);
        page = next;
      }
      x += g.j1 - g.j0;
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    for (int y = max(0, i - kSlots); y < i; ++y) mbar_wait(&bar.full[y % kSlots], (uint32_t)((y / kSlots) & 1), a.err);
    for (int y = max(0, seg - kStay); y < seg; ++y) mbar_wait(&bar.stay_full[y % kStay], (uint32_t)((y / kStay) & 1), a.err);
  } else if (warp == 17) {
    // =========================== products
    const uint32_t el = elect_one(), id = tc_idesc(Num<T>::kUmma, false, (uint32_t)ncol);
    auto wait = [&](uint64_t* b, int parity) { return ok = __all_sync(0xffffffffu, ok && mbar_wait(b, (uint32_t)parity, a.err)); };
    int i = 0, seg = 0;
    for (int x = x0; x < x1 && ok; ++seg) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
      if (!wait(&bar.stay_full[seg % kStay], (seg / kStay) & 1)) break;
      for (int j = g.j0; j < g.j1; ++j, ++i) {
        const int sl = i % kSlots, w = i & 3;
        if (!wait(&bar.full[sl], (i / kSlots) & 1)) break;
        if (i >= 4 && !wait(&bar.s_empty[w], (i / 4 - 1) & 1)) break;
        wt_product<D>(tmem + 128u * w, slots + sl * S::kTile, sb + (seg % kStay) * S::kTile, ncol, id, el);
        tc_commit(&bar.s_full[w], el);
        tc_commit(&bar.empty[sl], el);
      }
      tc_commit(&bar.stay_empty[seg % kStay], el);
      x += g.j1 - g.j0;
    }
    if (!ok) wt_drain(bar, a.err, el);
  } else {
    // =========================== sums: one key per thread
    const int w = warp >> 2, row = threadIdx.x & 127;
    float* l2 = reinterpret_cast<float*>(smem + S::kOffLse) + kWtN * w;
    int i = 0;
    for (int x = x0; x < x1;) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
      const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, g.b);
      const KeySpan<kWtM> ks = span_of(g.b);
      const int u = g.b * a.Hkv + g.h;
      named_bar_sync(1 + w, 128);  // the last unit's lse is read
      {
        const int head = g.h * a.G + row / qn, r = row % qn;
        l2[row] = row < ncol && r < qs.n ? wt_minus_lse2(__ldg(p.lse + ((int64_t)g.b * a.Hq + head) * p.q.Tq + r)) : -INFINITY;
      }
      const bool left_out = named_bar_any(1 + w, 128, l2[row] == -INFINITY);
      for (int j = g.j0; j < g.j1; ++j, ++i) {
        if ((i & 3) != w) continue;
        const int t = ks.key(j) + row;
        float* to = p.weights + (size_t)u * a.cap + t;
        const float old = t < qs.len ? __ldcg(to) : 0.f;  // back before the sum is
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        ok = wt_sum(a, qs, tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128u * w, ncol, qn, 0, t, l2, left_out, &bar.s_full[w], &bar.s_empty[w],
                    (uint32_t)((i >> 2) & 1), acc, ok);
        if (t < qs.len) *to = old + wt_total(acc);
      }
      x += g.j1 - g.j0;
    }
  }
  wt_end(tmem);
}

// ---------------------------------------------------------------- many queries
// A cluster takes 256 keys of one unit (LOOP: blocks y, y + gridDim.y, ... of them; the rings of operand
// tiles and scores run on from block to block, and a block's keys are loaded when the last one's sums are
// done).
template <typename T, int D, bool LOOP>
__global__ void __launch_bounds__(kWtThreads, 1) __cluster_dims__(kCluster, 1, 1)
    paged_weights_kernel(WtArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = WtSmem<D>;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, rank = (int)cluster_ctarank(), qn = p.rows;
  // of all units the earlier keys, which more queries see, first
  const int u = (int)blockIdx.x / kCluster, b = u / a.Hkv, h = u % a.Hkv;
  const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, b);
  // first and last query row that sees one of the keys from k0 on
  auto row_lo = [&](int k0) { return max(0, k0 - qs.off); };
  auto row_hi = [&](int k0) {
    int hi = qs.n - 1;
    if (a.window > 0 && k0 >= a.sinks) hi = (int)min((int64_t)hi, (int64_t)k0 + 2 * kWtM - 2 + a.window - qs.off);
    return hi;
  };
  // the next block from k0 on that a query sees (the same answer in every CTA of a cluster)
  const int step = (int)gridDim.y * 2 * kWtM;
  auto seen_from = [&](int k0) {
    while (k0 < qs.len && row_lo(k0) > row_hi(k0)) k0 += step;
    return k0;
  };
  int k0 = (int)blockIdx.y * 2 * kWtM;
  if (LOOP) k0 = seen_from(k0);
  if (k0 >= qs.len || (!LOOP && row_lo(k0) > row_hi(k0))) return;
  cluster_arrive_relaxed();  // the CTAs that rank 0 hears from may find it not yet started
  WtBars bar;
  const uint32_t tmem = wt_start<D>(smem, bar, &kmap, &qmap), sb = smem_u32(smem), slots = sb + S::kOffSlots;
  cluster_wait();
  float* lse2 = reinterpret_cast<float*>(smem + S::kOffLse);
  bool ok = true;
  int blk = 0, i0 = 0;    // blocks and steps before this block
  int even = 0, odd = 0;  // and the steps among them of warpgroups 0 and 1, and of 2 and 3
  do {
    const int r_lo = row_lo(k0), r_hi = row_hi(k0);
    // this CTA's share of the head-by-head list of query tiles
    const int t_lo = r_lo / qn, per = r_hi / qn - t_lo + 1, all = per * a.G;
    const int c0 = (int)((int64_t)all * rank / kCluster), n = (int)((int64_t)all * (rank + 1) / kCluster) - c0;
    float* ranks = reinterpret_cast<float*>(smem + S::kOffRank) + (blk & 1) * kCluster * 2 * kWtM;  // (rank 0 may still read the last block's)

    if (warp == 16) {
      // =========================== loads
      const uint32_t el = elect_one();
      const int rows = min(a.page_mask + 1, 64), k_lo = paged_window_lo(a, max(qs.off, 0));
      if (!LOOP || ok) {
        if (el) mbar_arrive_expect_tx(bar.stay_full, kStay * S::kTile);
        for (int x = 0; x < kStay; ++x)
          wt_load_keys<D>(a, &kmap, h, k0 + x * kWtM, rows, wt_page(a, b, qs.len, k_lo, k0 + x * kWtM, rows), sb + x * S::kTile,
                          bar.stay_full, el);
        int i = 0, hd = c0 / per, tl = c0 % per;
        for (; i < n; ++i) {
          const int at = i0 + i, sl = at % kSlots;
          if (at >= kSlots) ok = mbar_wait(&bar.empty[sl], (uint32_t)((at / kSlots - 1) & 1), a.err);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          wt_load_queries<D>(&qmap, b, h * a.G + hd, 1, (t_lo + tl) * qn, qn, slots + sl * S::kTile, &bar.full[sl], el);
          if (++tl == per) { tl = 0; ++hd; }
        }
        // every copy has landed before the CTA may end (also after a wait that gave up)
        mbar_wait(bar.stay_full, (uint32_t)(blk & 1), a.err);
        for (int y = max(0, i0 + i - kSlots); y < i0 + i; ++y) mbar_wait(&bar.full[y % kSlots], (uint32_t)((y / kSlots) & 1), a.err);
      }
    } else if (warp == 17) {
      // =========================== products: key tile x of step i to warpgroup 2 (i % 2) + x
      const uint32_t el = elect_one(), id = tc_idesc(Num<T>::kUmma, false, (uint32_t)qn);
      auto wait = [&](uint64_t* b, int parity) { return ok = __all_sync(0xffffffffu, ok && mbar_wait(b, (uint32_t)parity, a.err)); };
      wait(bar.stay_full, blk & 1);
      for (int i = 0; i < n && ok; ++i) {
        const int at = i0 + i, sl = at % kSlots, turn = (i & 1 ? odd : even) + (i >> 1);
        if (!wait(&bar.full[sl], (at / kSlots) & 1)) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int w = 2 * (i & 1) + x;
          if (turn >= 1 && !wait(&bar.s_empty[w], (turn - 1) & 1)) break;
          wt_product<D>(tmem + 128u * w, sb + x * S::kTile, slots + sl * S::kTile, qn, id, el);
          tc_commit(&bar.s_full[w], el);
        }
        tc_commit(&bar.empty[sl], el);
      }
      if (!ok) wt_drain(bar, a.err, el);
    } else {
      // =========================== sums: one key per thread
      const int w = warp >> 2, row = threadIdx.x & 127, t = k0 + (w & 1) * kWtM + row;
      float* l2 = lse2 + kWtN * w;
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // this warpgroup's steps w / 2, w / 2 + 2, ...: head and query tile of each
      int i = w >> 1, hd = (c0 + i) / per, tl = (c0 + i) % per;
      const float* lse = p.lse + ((int64_t)b * a.Hq + h * a.G) * p.q.Tq;
      auto fetch = [&]() {
        const int r = (t_lo + tl) * qn + row;
        return row < qn && r < qs.n ? __ldg(lse + (int64_t)hd * p.q.Tq + r) : -INFINITY;
      };
      float next = i < n ? fetch() : 0.f;
      for (int k = w >> 1 ? odd : even; i < n; i += 2, ++k) {
        const int r0 = (t_lo + tl) * qn;
        l2[row] = wt_minus_lse2(next);
        tl += 2;
        while (tl >= per) { tl -= per; ++hd; }
        if (i + 2 < n) next = fetch();
        const bool left_out = named_bar_any(1 + w, 128, l2[row] == -INFINITY);
        ok = wt_sum(a, qs, tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128u * w, qn, qn, r0, t, l2, left_out, &bar.s_full[w], &bar.s_empty[w],
                    (uint32_t)(k & 1), acc, ok);
        named_bar_sync(1 + w, 128);  // l2 is read
      }
      // the two warpgroups of these keys, then the ranks, in order
      const float sum = wt_total(acc);
      if (w >= 2) l2[row] = sum;
      named_bar_sync(5, 512);
      if (w < 2) st_cluster_f32(ranks + rank * 2 * kWtM + w * kWtM + row, 0, sum + lse2[kWtN * (w + 2) + row]);
    }
    if (LOOP) __syncthreads();
    else wt_end(tmem);
    cluster_sync();
    const int t = k0 + (int)threadIdx.x;
    if (rank == 0 && threadIdx.x < 2 * kWtM && t < qs.len) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) sum += ranks[r * 2 * kWtM + threadIdx.x];
      p.weights[(size_t)u * a.cap + t] += sum;
    }
    if (!LOOP) return;
    ++blk;
    i0 += n;
    even += (n + 1) >> 1;
    odd += n >> 1;
  } while ((k0 = seen_from(k0 + step)) < qs.len);
  wt_end(tmem);
}

// Columns of a head when the queries of all heads of a group fit one tile (0: they do not).
int few_rows(int G, int Tq) {
  for (int r = 16; r <= kWtN; r *= 2)
    if (Tq <= r) return G * r <= kWtN ? r : 0;
  return 0;
}

template <typename T, int D>
cudaError_t launch_td(const WtArgs& p, bool few, const CUtensorMap& kmap, const CUtensorMap& qmap, cudaStream_t s) {
  // Many queries: a cluster for each block of keys of each unit that the table has room for, or, where that
  // is more than four for each place (38 of four multiprocessors), so many that walk the blocks in turn: the
  // table says nothing of the lengths, and a cluster without a block holds its place for 0.7 us.  64 prompts
  // of 2048, 8 heads, d 128: 1464 us in turn, 1510 one by one, and 6950 one by one under a table for 131072
  // tokens; one prompt of 8192, 2 heads: 94 us in turn, 90 one by one (64 clusters, so taken).
  const int units = p.a.B * p.a.Hkv, blocks = (p.a.cap + 2 * kWtM - 1) / (2 * kWtM), most = (sm_count() + units - 1) / units;
  const auto kernel = few ? paged_weights_few_kernel<T, D> : blocks <= most ? paged_weights_kernel<T, D, false> : paged_weights_kernel<T, D, true>;
  const dim3 grid = few ? dim3(sm_count()) : dim3(units * kCluster, blocks < most ? blocks : most);
  const size_t smem = WtSmem<D>::kOffPrefix + (few ? ((size_t)p.a.B + 1) * 4 : 0);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kWtThreads, smem, s>>>(p, kmap, qmap);
  return cudaGetLastError();
}

}  // namespace

int paged_weights_rows(int G, int Tq) {
  const int r = few_rows(G, Tq);
  return r ? r : Tq <= 32 ? 32 : Tq <= 64 ? 64 : kWtN;
}

cudaError_t launch_paged_weights(const PagedArgs& a, int d, int dtype, const CUtensorMap& kmap, const CUtensorMap& qmap,
                                 const PagedQuery& q, const float* lse, float* weights, cudaStream_t s) {
  const WtArgs p = {a, q, lse, weights, paged_weights_rows(a.G, q.Tq)};
  const bool few = few_rows(a.G, q.Tq) > 0;
  if (dtype == DKV_BF16)
    return d == 128 ? launch_td<__nv_bfloat16, 128>(p, few, kmap, qmap, s) : launch_td<__nv_bfloat16, 64>(p, few, kmap, qmap, s);
  return d == 128 ? launch_td<__half, 128>(p, few, kmap, qmap, s) : launch_td<__half, 64>(p, few, kmap, qmap, s);
}

}  // namespace dkv
