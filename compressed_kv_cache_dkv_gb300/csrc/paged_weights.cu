// dkv_paged_weights: softmax weights summed by key, weights[t] += sum over queries of
// 2^(c q.k_t - lse), on the tcgen05 tensor cores.
//
// S^T = K Q^T for 128 keys and up to 128 query columns puts one key into each TMEM lane: a thread
// sums its key's weights over the columns in registers, every key has one owner, and the order is
// fixed (no atomics).  Two warpgroups take column tiles in turn, each with its own 128 TMEM columns;
// warp 8 streams operands with TMA, warp 9 issues the products; two CTAs share a multiprocessor.
//
// Few queries (those of all heads of a group fit 128 columns, padded to 16, 32, 64 or 128 a head):
// the column tile stays, the keys are streamed, a CTA walks a run of key tiles.  Bound by the read of K.
// Many queries: the keys stay, the query tiles of one head after the other are streamed; a cluster of
// kCluster CTAs shares the queries of its keys and adds the parts in rank order, since the first
// keys of a prompt are seen by all its queries and would take many times the average.
// Bound by the products (8 x 64 cycles a tile at d 128) and, close behind, their exponentials.
#include "paged_tc.cuh"

namespace dkv {
namespace {

constexpr int kWtThreads = 320, kWtM = 128, kWtN = 128;  // keys, query columns of a tile at most
constexpr int kSlots = 2;     // of the operand that is streamed
constexpr int kCluster = 8;   // CTAs that share the queries when the keys stay

template <int D>
struct WtSmem {  // [lse][part][rank][barriers], then the operand that stays and the slots
  static constexpr uint32_t kTile = 128 * D * 2;               // a slot: 128 keys or query rows
  static constexpr uint32_t kOffPart = 2 * kWtN * 4;           // [warpgroup][128] sums (before: base-2 lse)
  static constexpr uint32_t kOffRank = kOffPart + 2 * kWtM * 4;  // [rank][128] sums of the cluster
  static constexpr uint32_t kOffBar = kOffRank + kCluster * kWtM * 4;
  static constexpr uint32_t kOffStay = kOffBar + 1024 - kOffBar % 1024;
  static constexpr uint32_t kOffSlot = kOffStay + kTile;
};

struct WtArgs {
  PagedArgs a;
  PagedQuery q;
  const float* lse;
  float* weights;
  int stay;  // the queries stay: `rows` columns a head, all heads of a group in one tile
  int rows;  // query rows of a box
  int run;   // key tiles of a CTA
};

template <typename T, int D>
__global__ void __launch_bounds__(kWtThreads, 2)
    paged_weights_kernel(WtArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = WtSmem<D>;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool stay = p.stay != 0;
  // of all units the earlier keys, which more queries see, first
  const int ncl = stay ? 1 : kCluster, rank = stay ? 0 : (int)cluster_ctarank();
  const int u = (int)blockIdx.x / ncl, b = u / a.Hkv, h = u % a.Hkv, qn = p.rows;
  constexpr int ns = kSlots;
  const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, b);
  const int kt0 = (int)blockIdx.y * p.run, kt1 = min(kt0 + p.run, (qs.len + kWtM - 1) / kWtM);
  // query rows [lo, hi] that see a key of tile kt
  auto rows_of = [&](int kt, int& lo, int& hi) {
    const int k0 = kt * kWtM;
    lo = max(0, k0 - qs.off);
    hi = qs.n - 1;
    if (a.window > 0 && k0 >= a.sinks) hi = (int)min((int64_t)hi, (int64_t)k0 + kWtM - 2 + a.window - qs.off);
  };
  // column tiles of key tile kt: [c0, c0 + n) of the head-by-head list (this CTA's share of it)
  struct Cols { int per, t_lo, c0, n; };
  auto cols_of = [&](int kt) {
    Cols c = {0, 0, 0, 0};
    int lo, hi;
    rows_of(kt, lo, hi);
    if (lo > hi) return c;
    if (stay) { c.n = c.per = 1; return c; }
    c.t_lo = lo / qn;
    c.per = hi / qn - c.t_lo + 1;
    const int all = c.per * a.G;
    c.c0 = all * rank / ncl;
    c.n = all * (rank + 1) / ncl - c.c0;
    return c;
  };
  {
    bool any = false;  // the same answer in every CTA of a cluster
    for (int kt = kt0; kt < kt1; ++kt) {
      int lo, hi;
      rows_of(kt, lo, hi);
      any |= lo <= hi;
    }
    if (!any) return;
  }

  const uint32_t sb = smem_u32(smem);
  float* lse2 = reinterpret_cast<float*>(smem);
  float* part = reinterpret_cast<float*>(smem + S::kOffPart);
  float* ranks = reinterpret_cast<float*>(smem + S::kOffRank);
  uint64_t* stay_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* full = stay_full + 1;    // [slot]
  uint64_t* empty = full + kSlots;   // [slot]
  uint64_t* s_full = empty + kSlots; // [warpgroup]
  uint64_t* s_empty = s_full + 2;  // [warpgroup]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_empty + 2);
  if (threadIdx.x == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&qmap);
    mbar_init(stay_full, 1);
    for (int i = 0; i < ns; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 128);
    }
    fence_mbar_init();
  }
  if (!stay) cluster_arrive_relaxed();  // the CTAs that rank 0 hears from may find it not yet started
  if (warp == 0) tc_alloc<256>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!stay) cluster_wait();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 8) {
    // =========================== loads
    const uint32_t el = elect_one();
    const int rows = min(a.page_mask + 1, 64), pk = kWtM / rows;  // runs of `rows` keys
    const int lo = paged_window_lo(a, max(qs.off, 0));
    auto page_of = [&](int kt) {  // lane i < pk: the page of the tile's i-th run
      const int first = kt * kWtM + lane * rows;
      // runs without a visible key: zeros, wherever the table points
      return lane < pk && first < qs.len && (first + rows > lo || first < a.sinks) ? paged_page(a, b, first) : a.n_pages;
    };
    auto load_k = [&](int kt, int page, uint32_t to, uint64_t* bar) {
      if (el) mbar_arrive_expect_tx(bar, S::kTile);
#pragma unroll 2
      for (int i = 0; i < pk; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
          tma_load_4d(to + hf * kWtM * 128 + i * rows * 128, &kmap, hf * 64, (kt * kWtM + i * rows) & a.page_mask, h, pg, bar, el);
      }
    };
    // `n` heads' boxes of qn rows, side by side in column tiles of `ncol`
    auto load_q = [&](int head, int n, int row, uint32_t to, uint64_t* bar) {
      if (el) mbar_arrive_expect_tx(bar, (uint32_t)(n * qn) * D * 2);
      for (int x = 0; x < n; ++x)
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
          tma_load_4d(to + hf * n * qn * 128 + x * qn * 128, &qmap, hf * 64, row, head + x, b, bar, el);
    };
    int i = 0, page = page_of(kt0);
    if (stay) load_q(h * a.G, a.G, 0, sb + S::kOffStay, stay_full);
    else load_k(kt0, page, sb + S::kOffStay, stay_full);
    for (int kt = kt0; kt < kt1 && ok; ++kt) {
      const Cols c = cols_of(kt);
      const int next = stay && kt + 1 < kt1 ? page_of(kt + 1) : 0;  // looked up a tile ahead of its use
      for (int x = 0; x < c.n; ++x, ++i) {
        const int sl = i % ns;
        if (i >= ns) ok = mbar_wait(&empty[sl], (uint32_t)((i / ns - 1) & 1), a.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        if (stay) load_k(kt, page, sb + S::kOffSlot + sl * S::kTile, &full[sl]);
        else load_q(h * a.G + (c.c0 + x) / c.per, 1, (c.t_lo + (c.c0 + x) % c.per) * qn, sb + S::kOffSlot + sl * S::kTile, &full[sl]);
      }
      page = next;
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    mbar_wait(stay_full, 0, a.err);
    for (int x = max(0, i - ns); x < i; ++x) mbar_wait(&full[x % ns], (uint32_t)((x / ns) & 1), a.err);
  } else if (warp == 9) {
    // =========================== products
    const uint32_t el = elect_one();
    const int ncol = stay ? a.G * qn : qn;
    const uint32_t id = tc_idesc(Num<T>::kUmma, false, (uint32_t)ncol);
    ok = __all_sync(0xffffffffu, mbar_wait(stay_full, 0, a.err));
    int i = 0;
    for (int kt = kt0; kt < kt1 && ok; ++kt) {
      const Cols c = cols_of(kt);
      for (int x = 0; x < c.n; ++x, ++i) {
        const int w = i & 1, sl = i % ns;
        ok = ok && mbar_wait(&full[sl], (uint32_t)((i / ns) & 1), a.err);
        if (i >= 2) ok = ok && mbar_wait(&s_empty[w], (uint32_t)((i / 2 - 1) & 1), a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t slot = sb + S::kOffSlot + sl * S::kTile;
        const uint64_t kd = tc_desc(stay ? slot : sb + S::kOffStay, 16, 1024), qd = tc_desc(stay ? sb + S::kOffStay : slot, 16, 1024);
        const uint64_t half = (uint64_t)(ncol * 128 >> 4);  // the query tile's second 64 channels
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma(tmem + 128u * w, kd + (uint64_t)(((k >> 2) * kWtM * 128 + (k & 3) * 32) >> 4),
                 qd + (k >> 2) * half + (uint64_t)((k & 3) * 32 >> 4), id, k > 0, el);
        tc_commit(&s_full[w], el);
        tc_commit(&empty[sl], el);
      }
    }
  } else {
    // =========================== sums: one key per thread and warpgroup
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128u * w;
    float* l2 = lse2 + kWtN * w;
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    auto sync_group = [&]() { if (w == 0) named_bar_sync(1, 128); else named_bar_sync(2, 128); };
    // minus the base-2 lse of column `row` of a tile (-inf for a column without a query, so that it adds 0)
    auto column = [&](int head, int r, bool live) {
      if (!live || r >= qs.n) return -INFINITY;
      const float v = __ldg(p.lse + ((int64_t)b * a.Hq + head) * p.q.Tq + r);
      return v == -INFINITY ? -INFINITY : v * -1.4426950408889634f;
    };
    if (stay) {
      l2[row] = column(h * a.G + row / qn, row % qn, row < a.G * qn);
      sync_group();
    }
    int i = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      const Cols c = cols_of(kt);
      const int t = kt * kWtM + row;
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      float next = 0.f, old = 0.f;
      if (stay && t < qs.len) old = __ldcg(p.weights + (size_t)u * a.cap + t);  // back before the sum is
      auto fetch = [&](int x) { return column(h * a.G + (c.c0 + x) / c.per, (c.t_lo + (c.c0 + x) % c.per) * qn + row, row < qn); };
      const int x0 = (w ^ i) & 1;  // this warpgroup's first column tile
      if (!stay && x0 < c.n) next = fetch(x0);
      for (int x = x0; x < c.n; x += 2) {
        const int at = (i + x) / 2;  // tiles of this warpgroup so far
        const int r0 = stay ? 0 : (c.t_lo + (c.c0 + x) % c.per) * qn;
        if (!stay) {
          l2[row] = next;
          if (x + 2 < c.n) next = fetch(x + 2);
          sync_group();
        }
        if (ok) ok = mbar_wait(&s_full[w], (uint32_t)(at & 1), a.err);
        tc_fence_after();
        // rows [v_lo, v_hi) of the tile see this key
        const int v_lo = max(t - qs.off - r0, 0);
        int v_hi = min(qn, qs.n - r0);
        const bool bound = a.window > 0 && t >= a.sinks;
        if (bound) v_hi = (int)max((int64_t)0, min((int64_t)v_hi, (int64_t)t + a.window - qs.off - r0));
        const int ncol = stay ? a.G * qn : qn;
        const bool all = __all_sync(0xffffffffu, v_lo == 0 && v_hi == qn);
#pragma unroll
        for (int ch = 0; ch < kWtN / 32; ++ch) {
          if (32 * ch >= ncol) break;
          if (!stay && !__any_sync(0xffffffffu, v_lo < 32 * ch + 32 && v_hi > 32 * ch)) continue;
          uint32_t s[32];
          tc_ld32(ts + 32 * ch, s);
          tc_ld_wait();
          if (all && 32 * ch + 32 <= ncol) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 m = *reinterpret_cast<const float4*>(l2 + 32 * ch + e);
              const float2 y0 = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), scale2, make_float2(m.x, m.y));
              const float2 y1 = fma2(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), scale2, make_float2(m.z, m.w));
              acc[0] = add2(acc[0], make_float2(fast_exp2(y0.x), fast_exp2(y0.y)));
              acc[1] = add2(acc[1], make_float2(fast_exp2(y1.x), fast_exp2(y1.y)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int r = stay ? (32 * ch + e) & (qn - 1) : 32 * ch + e;
              const float x2 = fast_exp2(fmaf(__uint_as_float(s[e]), a.scale_log2, l2[32 * ch + e]));
              // (what lies in a hidden column, or beyond the last, is not looked at)
              acc[e & 1].x += r >= v_lo && r < v_hi && 32 * ch + e < ncol ? x2 : 0.f;
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&s_empty[w]);
        if (!stay) sync_group();  // l2 is read
      }
      i += c.n;
      const float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      if (stay) {  // a key tile is one column tile, and so one warpgroup's
        if (c.n > 0 && x0 == 0 && t < qs.len) p.weights[(size_t)u * a.cap + t] = old + sum;
      } else {
        part[w * kWtM + row] = sum;
        named_bar_sync(3, 256);
        if (w == 0) st_cluster_f32(ranks + rank * kWtM + row, 0, part[row] + part[kWtM + row]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tc_free<256>(tmem);
  if (!stay) {
    cluster_sync();
    const int t = kt0 * kWtM + (int)threadIdx.x;
    if (rank == 0 && threadIdx.x < kWtM && t < qs.len) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) sum += ranks[r * kWtM + threadIdx.x];
      p.weights[(size_t)u * a.cap + t] += sum;
    }
  }
}

// Columns of a head when the queries of all heads of a group fit one tile (0: they do not).
int stay_rows(int G, int Tq) {
  for (int r = 16; r <= 128; r *= 2)
    if (Tq <= r) return G * r <= kWtN ? r : 0;
  return 0;
}

template <typename T, int D>
cudaError_t launch_td(const WtArgs& p, const CUtensorMap& kmap, const CUtensorMap& qmap, cudaStream_t s) {
  const void* kernel = reinterpret_cast<const void*>(paged_weights_kernel<T, D>);
  constexpr uint32_t smem = WtSmem<D>::kOffSlot + kSlots * WtSmem<D>::kTile;
  cudaError_t e = ensure_smem_limit(kernel, smem);
  if (e != cudaSuccess) return e;
  const int units = p.a.B * p.a.Hkv, tiles = (p.a.cap + kWtM - 1) / kWtM;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.stay ? units : units * kCluster, (tiles + p.run - 1) / p.run);
  cfg.blockDim = dim3(kWtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.stay ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, paged_weights_kernel<T, D>, p, kmap, qmap);
}

}  // namespace

int paged_weights_rows(int G, int Tq) {
  const int r = stay_rows(G, Tq);
  return r ? r : Tq <= 32 ? 32 : Tq <= 64 ? 64 : kWtN;
}

cudaError_t launch_paged_weights(const PagedArgs& a, int d, int dtype, const CUtensorMap& kmap, const CUtensorMap& qmap,
                                 const PagedQuery& q, const float* lse, float* weights, cudaStream_t s) {
  WtArgs p;
  p.a = a;
  p.q = q;
  p.lse = lse;
  p.weights = weights;
  p.stay = stay_rows(a.G, q.Tq) > 0;
  p.rows = paged_weights_rows(a.G, q.Tq);
  // runs long enough to hide a CTA's start behind its loads, short enough for every multiprocessor to have two
  const int64_t tiles = (int64_t)a.B * a.Hkv * ((a.cap + kWtM - 1) / kWtM), share = tiles / (2 * sm_count());
  p.run = p.stay ? (int)(share < 1 ? 1 : share > 16 ? 16 : share) : 1;
  if (dtype == DKV_BF16)
    return d == 128 ? launch_td<__nv_bfloat16, 128>(p, kmap, qmap, s) : launch_td<__nv_bfloat16, 64>(p, kmap, qmap, s);
  return d == 128 ? launch_td<__half, 128>(p, kmap, qmap, s) : launch_td<__half, 64>(p, kmap, qmap, s);
}

}  // namespace dkv
