// dkv_paged_decode: attention of one new token per sequence over a paged cache.
//
// The visible tokens of a sequence are cut into 64-token tiles (the tiles of its
// sinks, then those of its window); the tiles of all (sequence, KV head) units in a
// row are dealt out evenly to the CTAs, one per multiprocessor, whatever the
// sequences' lengths.  A CTA walks its run of tiles unit by unit; a unit that lies
// wholly in one run is finished there, the others leave one partial record per run
// they touch, which the combine grid merges in run order (deterministic).
//
// One producer warp streams tiles of K and V with TMA boxes (one per page, 64
// channels wide, 128-byte swizzle) into a ring of kDecStages stages; its lanes look up
// the tile's pages, one elected lane issues.  Eight consumer warps in two teams take tiles in turn, warp w of
// a team 16 tokens:
//   S = K q      ldmatrix K fragments, mma.sync m16n8k16, tokens in M, heads in N
//   o += V^T p   ldmatrix.trans V^T fragments, p as hi + lo 16-bit halves
// with an online softmax per warp in base 2, merged over the warps at a unit's end.
// Bound by HBM: 4 d bytes per token and KV head; the products need 2 x 8 columns of
// which G are used, on a path that has time to spare.  Even runs of tiles keep all multiprocessors
// reading to the end whatever the lengths are; two teams of consumers hide one tile's chain of products,
// softmax and products behind the other's; four stages of 32 KB keep more bytes on their way than the
// latency of the reads takes.
//
// Measured (d 128): 64 sequences of 300 to 8000 tokens, 8 KV heads, a window of 4096 and 4 sinks,
// pages of 16 (841 MB): 137 to 141 us, 6.0 TB/s.  16 of 64k tokens, 2 KV heads, with their weights (1.09 GB):
// 193 us, 5.6 TB/s.  One of 1000 tokens: 7.4 us in a graph, the latency of two launches.
//
// Rows of V that the query does not see inside a tile are zeroed in shared memory
// before the product: their weight is 0, but 0 x NaN from a slot never written would not be.
#include "paged.cuh"

namespace dkv {
namespace {

constexpr int kDecTile = 64, kDecStages = 4, kDecConsumers = 8;
// a stage always belongs to the same team, which so sees every phase of its barrier
static_assert(kDecStages % 2 == 0, "two teams take the stages in turn");
constexpr int kDecThreads = 32 * (kDecConsumers + 1);
constexpr int kCombThreads = 512, kCombCols = 32;  // combine: channels per CTA
constexpr int kScoreThreads = 256, kScoreBatch = 8, kScoreTokens = 2048;
static_assert(kScoreTokens % (kScoreBatch * kScoreThreads / 2) == 0, "whole rounds");

// p, its sums and so o carry a factor 2^kDecShift.  A fp16 value below 2^-25 would be lost, and a long
// cache can hold tens of thousands of such weights beside one of 1: with the factor, and the low half
// behind the high one, weights down to e^-18 of the largest keep 11 bits and those to e^-27 count.
template <typename T>
constexpr float kDecShift = 0.f;
template <>
constexpr float kDecShift<__half> = 14.f;

template <int D>
constexpr int rec_floats() { return 16 + 8 * D; }

// The tiles of a sequence that its last token sees.
struct Span {
  int len, lo, st, wt0, n;  // tokens, window start, sink tiles, first window tile, tiles in all
  __device__ int token(int j) const { return (j < st ? j : wt0 + j - st) * kDecTile; }
};
__device__ inline Span dec_span(const PagedArgs& a, int b) {
  Span s;
  s.len = paged_len(a, b);
  s.lo = paged_window_lo(a, s.len - 1);
  s.wt0 = s.lo / kDecTile;
  s.st = min((min(a.sinks, s.len) + kDecTile - 1) / kDecTile, s.wt0);
  s.n = s.st + (s.len + kDecTile - 1) / kDecTile - s.wt0;
  return s;
}

struct DecArgs {
  PagedArgs a;
  const void* q;
  int64_t q_batch, q_head;
  void* out;
  float* lse;
  float* records;
  float* scores;  // [units][cap][8] base-2 scores, or null
};

template <typename T, int D>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_decode_kernel(DecArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedArgs& a = p.a;
  constexpr int KT = D / 16;
  constexpr uint32_t TILE = kDecTile * D * 2;  // bytes of one K (or V) tile
  float* merge = reinterpret_cast<float*>(smem + kDecStages * 2 * TILE);    // o [warp][D][8]
  float* stats = merge + kDecConsumers * D * 8;                             // m, l [warp][2][8]
  uint64_t* full = reinterpret_cast<uint64_t*>(stats + kDecConsumers * 16);  // [stage]
  uint64_t* empty = full + kDecStages;
  int* prefix = reinterpret_cast<int*>(empty + kDecStages);                 // [B + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem);

  if (threadIdx.x == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
    for (int i = 0; i < kDecStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);  // the four warps of the team that read the stage
    }
    fence_mbar_init();
  }
  deal_prefix(a.B, prefix, [&](int b) { return dec_span(a, b).n; });
  __syncthreads();
  griddep_launch();
  // sequences without a token: zeros and -inf
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) {
      T* o = static_cast<T*>(p.out) + (size_t)b * a.Hq * D;
      for (int e = threadIdx.x; e < a.Hq * D; e += kDecThreads) o[e] = Num<T>::from_float(0.f);
      if (p.lse)
        for (int e = threadIdx.x; e < a.Hq; e += kDecThreads) p.lse[(size_t)b * a.Hq + e] = -INFINITY;
    }
  const int total = prefix[a.B] * a.Hkv, nc = min((int)gridDim.x, total), c = blockIdx.x;
  if (c >= nc) return;
  const int x0 = deal_bound(total, nc, c), x1 = deal_bound(total, nc, c + 1);

  if (warp == kDecConsumers) {
    // =========================== producer
    const uint32_t el = elect_one();
    const uint64_t policy = policy_evict_first();  // a cache is read once a step
    const int rows = min(a.page_mask + 1, kDecTile), ppt = kDecTile / rows;  // boxes of `rows` slots, runs per tile
    bool ok = true;
    int it = 0;
    for (int x = x0; x < x1 && ok;) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
      const Span s = dec_span(a, g.b);
      for (int j = g.j0; j < g.j1; ++j, ++it) {
        const int st = it % kDecStages, y = s.token(j) & a.page_mask, first = s.token(j) + lane * rows;
        int page = a.n_pages;  // runs without a visible token: zeros, wherever the table points
        if (lane < ppt && first < s.len && (first + rows > s.lo || first < a.sinks)) page = paged_page(a, g.b, first);
        if (it >= kDecStages) ok = mbar_wait(&empty[st], (uint32_t)((it / kDecStages - 1) & 1), a.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        if (el) mbar_arrive_expect_tx(&full[st], 2 * TILE);
        const uint32_t dst = sb + (uint32_t)(2 * st) * TILE;
#pragma unroll 1
        for (int i = 0; i < ppt; ++i) {
          const int pg = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf) {
            const uint32_t at = dst + (uint32_t)hf * kDecTile * 128u + (uint32_t)(i * rows) * 128u;
            tma_load_4d(at, &kmap, hf * 64, y, g.h, pg, &full[st], el, policy);
            tma_load_4d(at + TILE, &vmap, hf * 64, y, g.h, pg, &full[st], el, policy);
          }
        }
      }
      x += g.j1 - g.j0;
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    for (int i = max(0, it - kDecStages); i < it; ++i) mbar_wait(&full[i % kDecStages], (uint32_t)((i / kDecStages) & 1), a.err);
    return;
  }

  // =========================== consumers
  const int team = warp >> 2, wr = 16 * (warp & 3);  // this warp's rows of a tile
  const int t = lane & 3, gq = lane >> 2, mi = lane >> 3, mr = lane & 7;
  const float slog2 = a.scale_log2;
  bool ok = true;
  int it = 0;
  for (int x = x0; x < x1;) {
    const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
    const Span s = dec_span(a, g.b);
    const int u = g.b * a.Hkv + g.h;
    // q as B fragments (k = channels, n = heads of the group; heads past the group read zeros)
    uint32_t qb[KT][2];
    {
      const bool live = gq < a.G;
      const uint32_t* qrow = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + g.b * p.q_batch +
                                                               (int64_t)(g.h * a.G + (live ? gq : 0)) * p.q_head);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        qb[kt][0] = live ? __ldg(qrow + 8 * kt + t) : 0u;
        qb[kt][1] = live ? __ldg(qrow + 8 * kt + 4 + t) : 0u;
      }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[KT][4];
#pragma unroll
    for (int i = 0; i < KT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int j = g.j0; j < g.j1; ++j, ++it) {
      if ((it & 1) != team) continue;
      const int st = it % kDecStages, tok0 = s.token(j);
      if (ok) ok = mbar_wait(&full[st], (uint32_t)((it / kDecStages) & 1), a.err);
      const uint32_t kb = sb + (uint32_t)(2 * st) * TILE, vb = kb + TILE;
      float ac[2][4] = {};  // even and odd k tiles: two shorter chains
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const uint4 kf = ldsm_x4(kb + sw128(kDecTile, wr + (mi & 1) * 8 + mr, 2 * kt + (mi >> 1)));
        Num<T>::mma(ac[kt & 1], kf.x, kf.y, kf.z, kf.w, qb[kt][0], qb[kt][1]);
      }
      float sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = (ac[0][i] + ac[1][i]) * slog2;
      const int tk = tok0 + wr + gq;
      if (!((tok0 >= s.lo && tok0 + kDecTile <= s.len) || tok0 + kDecTile <= min(a.sinks, s.len))) {  // a tile at an edge
        auto seen = [&](int y) { return y < s.len && (y >= s.lo || y < a.sinks); };
        if (!seen(tk)) sc[0] = sc[1] = -INFINITY;
        if (!seen(tk + 8)) sc[2] = sc[3] = -INFINITY;
        const int row = wr + (lane >> 1);
        if (!seen(tok0 + row))
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch)
            sts128(vb + sw128(kDecTile, row, (lane & 1) * (D / 16) + ch), make_uint4(0, 0, 0, 0));
        fence_proxy_async();
        __syncwarp();
      }
      if (p.scores) {
        float* row = p.scores + ((size_t)u * a.cap + tk) * 8 + 2 * t;
        if (tk < s.len) *reinterpret_cast<float2*>(row) = make_float2(sc[0], sc[1]);
        if (tk + 8 < s.len) *reinterpret_cast<float2*>(row + 64) = make_float2(sc[2], sc[3]);
      }
      // ---- online softmax over the warp's tokens (columns 2t, 2t + 1)
      float y0 = fmaxf(sc[0], sc[2]), y1 = fmaxf(sc[1], sc[3]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, off));
        y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, off));
      }
      const float n0 = fmaxf(m0, y0), n1 = fmaxf(m1, y1);
      const float ms0 = n0 == -INFINITY ? 0.f : n0, ms1 = n1 == -INFINITY ? 0.f : n1;
      const float f0 = fast_exp2(m0 - ms0), f1 = fast_exp2(m1 - ms1);
      m0 = n0;
      m1 = n1;
      // (the shift behind the difference: in front of it a large maximum would round it away)
      const float p0 = fast_exp2((sc[0] - ms0) + kDecShift<T>), p1 = fast_exp2((sc[1] - ms1) + kDecShift<T>);
      const float p2 = fast_exp2((sc[2] - ms0) + kDecShift<T>), p3 = fast_exp2((sc[3] - ms1) + kDecShift<T>);
      l0 = l0 * f0 + (p0 + p2);
      l1 = l1 * f1 + (p1 + p3);
      if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
        for (int i = 0; i < KT; ++i) { o[i][0] *= f0; o[i][1] *= f1; o[i][2] *= f0; o[i][3] *= f1; }
      }
      // p (C fragment: rows = tokens) -> B fragments (k = tokens, n = heads), hi + lo halves:
      // a single 16-bit p would be the only rounding of the call coarser than its output's
      uint32_t h01, r01, h23, r23;
      Num<T>::split(p0, p1, h01, r01);
      Num<T>::split(p2, p3, h23, r23);
      const uint32_t bh0 = movtrans(h01), bl0 = movtrans(r01), bh1 = movtrans(h23), bl1 = movtrans(r23);
#pragma unroll
      for (int md = 0; md < KT; ++md) {
        const uint4 v = ldsm_x4_trans(vb + sw128(kDecTile, wr + (mi >> 1) * 8 + mr, 2 * md + (mi & 1)));
        Num<T>::mma(o[md], v.x, v.y, v.z, v.w, bh0, bh1);
        Num<T>::mma(o[md], v.x, v.y, v.z, v.w, bl0, bl1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    x += g.j1 - g.j0;

    // ---- merge the eight warps
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (lane < 4) {
      *reinterpret_cast<float2*>(stats + warp * 16 + 2 * t) = make_float2(m0, m1);
      *reinterpret_cast<float2*>(stats + warp * 16 + 8 + 2 * t) = make_float2(l0, l1);
    }
#pragma unroll
    for (int md = 0; md < KT; ++md) {
      float* ow = merge + (warp * D + md * 16 + gq) * 8 + 2 * t;
      *reinterpret_cast<float2*>(ow) = make_float2(o[md][0], o[md][1]);
      *reinterpret_cast<float2*>(ow + 64) = make_float2(o[md][2], o[md][3]);
    }
    named_bar_sync(1, 32 * kDecConsumers);
    {
      const int gg = threadIdx.x & 7;
      float M = -INFINITY, L = 0.f, f[kDecConsumers];
#pragma unroll
      for (int w = 0; w < kDecConsumers; ++w) M = fmaxf(M, stats[w * 16 + gg]);
      const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kDecConsumers; ++w) {
        f[w] = fast_exp2(stats[w * 16 + gg] - Ms);
        L += f[w] * stats[w * 16 + 8 + gg];
      }
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no weight at all: zeros; a NaN stays one
      float* rec = p.records + (size_t)(2 * c + (g.j0 == 0 ? 1 : 0)) * rec_floats<D>();
      const size_t head = (size_t)g.b * a.Hq + g.h * a.G + gg;
#pragma unroll
      for (int dd = threadIdx.x >> 3; dd < D; dd += 4 * kDecConsumers) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kDecConsumers; ++w) v += f[w] * merge[(w * D + dd) * 8 + gg];
        if (!whole) rec[16 + dd * 8 + gg] = v;
        else if (gg < a.G) static_cast<T*>(p.out)[head * D + dd] = Num<T>::from_float(v * inv);
      }
      if (threadIdx.x < 8) {
        if (!whole) {
          rec[gg] = M;
          rec[8 + gg] = L;
        } else if (gg < a.G && p.lse) {
          p.lse[head] = (M - kDecShift<T> + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    named_bar_sync(1, 32 * kDecConsumers);
  }
}

// Merge of the units that lie in several runs.  CTA (c, y) looks at the run of decode
// CTA c: where its last unit begins in it and goes on in the next runs, it merges that
// unit's records (slot 1 of c, slot 0 of the following CTAs) for 32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(DecArgs p, int ncta) {
  const PagedArgs& a = p.a;
  extern __shared__ float csm[];
  constexpr int kGroups = kCombThreads / (8 * kCombCols);  // records taken side by side
  __shared__ float part[kCombThreads];
  int* prefix = reinterpret_cast<int*>(csm);
  float* fac = csm + a.B + 1;  // [record][8]
  float* red = fac + 8 * ncta;  // M, L [8] each
  deal_prefix(a.B, prefix, [&](int b) { return dec_span(a, b).n; });
  __syncthreads();
  griddep_wait();
  const int total = prefix[a.B] * a.Hkv, nc = min(ncta, total), c = blockIdx.x;
  if (c >= nc) return;
  const int x0 = deal_bound(total, nc, c), x1 = deal_bound(total, nc, c + 1);
  const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x1 - 1, x1);  // the last tile's unit
  const int begin = x1 - 1 - g.j0;                        // its first tile
  if (begin < x0 || g.j0 + 1 == g.n) return;
  const int nrec = deal_owner(total, nc, begin + g.n - 1) - c + 1;
  auto rec = [&](int i) { return p.records + (size_t)(2 * (c + i) + (i == 0 ? 1 : 0)) * rec_floats<D>(); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < 8) {
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < nrec; i += 32) M = fmaxf(M, __ldcg(rec(i) + warp));
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float Ms = M == -INFINITY ? 0.f : M;
    for (int i = lane; i < nrec; i += 32) {
      const float f = fast_exp2(__ldcg(rec(i) + warp) - Ms);
      fac[i * 8 + warp] = f;
      L += f * __ldcg(rec(i) + 8 + warp);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (lane == 0) { red[warp] = M; red[8 + warp] = L; }
  }
  __syncthreads();
  const int e = threadIdx.x % (8 * kCombCols), grp = threadIdx.x / (8 * kCombCols), gg = e & 7;
  const int dd = blockIdx.y * kCombCols + (e >> 3);
  float v = 0.f;
#pragma unroll 8
  for (int i = grp; i < nrec; i += kGroups) v += fac[i * 8 + gg] * __ldcg(rec(i) + 16 + dd * 8 + gg);
  part[threadIdx.x] = v;
  __syncthreads();
  if (grp == 0 && gg < a.G) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) v += part[i * 8 * kCombCols + e];
    const float L = red[8 + gg], inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const size_t head = (size_t)g.b * a.Hq + g.h * a.G + gg;
    static_cast<T*>(p.out)[head * D + dd] = Num<T>::from_float(v * inv);
    if (p.lse && dd == 0) p.lse[head] = (red[gg] - kDecShift<T> + log2f(L)) * 0.6931471805599453f;
  }
}

// weights[unit][t] += sum over the group's heads of 2^(score - lse), from the scores the decode
// kernel left: 32 bytes a token beside the 4 d of its key and value.  Two neighbouring threads take
// the two halves of a token's scores, so that a warp reads whole lines; kScoreBatch of them in flight.
__global__ void __launch_bounds__(kScoreThreads) paged_score_kernel(DecArgs p, float* __restrict__ weights) {
  const PagedArgs& a = p.a;
  griddep_wait();
  const int u = blockIdx.y, b = u / a.Hkv, h = u % a.Hkv, len = paged_len(a, b), lo = paged_window_lo(a, len - 1);
  const int first = blockIdx.x * kScoreTokens;
  if (first >= len) return;
  const int half = threadIdx.x & 1, g0 = 4 * half;
  float l2[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float l = g0 + g < a.G ? __ldcg(p.lse + (size_t)b * a.Hq + h * a.G + g0 + g) * 1.4426950408889634f : -INFINITY;
    l2[g] = l == -INFINITY ? INFINITY : l;  // (a head without a weight, or none: adds 0)
  }
  float* wu = weights + (size_t)u * a.cap;
#pragma unroll 1
  for (int base = first + (threadIdx.x >> 5) * 16; base < min(first + kScoreTokens, len); base += kScoreBatch * kScoreThreads / 2) {
    const int t0 = base + ((threadIdx.x & 31) >> 1);  // (base is the warp's: its lanes go round together)
    float4 s[kScoreBatch];
    float old[kScoreBatch];
    bool sees[kScoreBatch];
#pragma unroll
    for (int x = 0; x < kScoreBatch; ++x) {
      const int t = t0 + x * kScoreThreads / 2;
      sees[x] = t < len && (t >= lo || t < a.sinks);
      s[x] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (sees[x] && g0 < a.G) s[x] = __ldcg(reinterpret_cast<const float4*>(p.scores + ((size_t)u * a.cap + t) * 8 + g0));
      old[x] = sees[x] && half == 0 ? __ldcg(wu + t) : 0.f;
    }
#pragma unroll
    for (int x = 0; x < kScoreBatch; ++x) {
      const float v[4] = {s[x].x, s[x].y, s[x].z, s[x].w};
      float w = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g0 + g < a.G) w += fast_exp2(v[g] - l2[g]);
      w += __shfl_xor_sync(0xffffffffu, w, 1);
      if (sees[x] && half == 0) wu[t0 + x * kScoreThreads / 2] = old[x] + w;
    }
  }
}

template <typename T, int D>
cudaError_t launch_decode_td(const DecArgs& p, const PagedMaps& m, float* weights, cudaStream_t s) {
  const int ncta = sm_count();
  const size_t smem = (size_t)kDecStages * 4 * kDecTile * D + kDecConsumers * (D * 8 + 16) * 4 + kDecStages * 16 +
                      ((size_t)p.a.B + 1) * 4;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(paged_decode_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<T, D><<<ncta, kDecThreads, smem, s>>>(p, m.k, m.v);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(paged_combine_kernel<T, D>, dim3(ncta, D / kCombCols), kCombThreads,
                 ((size_t)p.a.B + 1 + 8 * ncta + 16) * 4, s, p, ncta);
  if (e != cudaSuccess || !weights) return e;
  return launch_dependent(paged_score_kernel, dim3((p.a.cap + kScoreTokens - 1) / kScoreTokens, p.a.B * p.a.Hkv), kScoreThreads, 0, s, p, weights);
}

}  // namespace

size_t paged_decode_ws_bytes(int d) { return kWsHeader + (size_t)2 * sm_count() * (16 + 8 * d) * 4; }

cudaError_t launch_paged_decode(const PagedArgs& a, int d, int dtype, const PagedMaps& m, const void* q,
                                const dkv_strides& qs, void* out, float* lse, float* weights, float* scores, uint8_t* ws,
                                cudaStream_t s) {
  DecArgs p;
  p.a = a;
  p.q = q;
  p.q_batch = qs.batch;
  p.q_head = qs.head;
  p.out = out;
  p.lse = lse;
  p.records = reinterpret_cast<float*>(ws + kWsHeader);
  p.scores = weights ? scores : nullptr;
  if (dtype == DKV_BF16)
    return d == 128 ? launch_decode_td<__nv_bfloat16, 128>(p, m, weights, s) : launch_decode_td<__nv_bfloat16, 64>(p, m, weights, s);
  return d == 128 ? launch_decode_td<__half, 128>(p, m, weights, s) : launch_decode_td<__half, 64>(p, m, weights, s);
}

}  // namespace dkv
