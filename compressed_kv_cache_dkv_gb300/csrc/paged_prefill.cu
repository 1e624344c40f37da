// dkv_paged_prefill: causal attention of the last tokens of each sequence over a paged cache,
// with an optional sliding window and sinks, on the tcgen05 tensor cores.
//
// A CTA owns two groups of 128 query rows that share every K and V tile: two heads of one
// KV head at the same tokens where the group size is even, else 256 tokens of one head; up to 64
// queries stand in rows of 8, 16, 32 or 64 a head, so that a group holds several heads.  A grid
// that would leave half of the multiprocessors idle is multiplied by cutting the key tiles of
// each CTA into parts, which a second grid joins by their maxima and sums.  Per 64-key tile j and
// group g
//   S_g = Q_g K_j^T   M = 128 queries, N = 64 keys   (64 TMEM columns, two buffers a group)
//   O_g += P_g V_j    M = 128, N = d, P from TMEM (16-bit, over the first 32 columns of its S)
// One row per softmax thread (warps 0-3 group A, 4-7 group B).  Warps 8 and 11 stream K and V
// with TMA boxes, one per page and 64 channels, into five slots each; warps 9 and 10 issue
// the products of groups A and B: S of tile j + 1 goes out while the rows still turn S_j into P,
// so that neither the rows nor the tensor cores wait for the other's latency.  (With 128-key
// tiles, which read Q half as often from shared memory, there is room for one S only, and the
// chain S - P - O - next S of a group takes 3700 cycles per 128 keys, of which 1024 products.)
// S_{j+2} overwrites P_j, so it is issued once O_j is done.  The row maximum moves only when a
// score exceeds it by kPfSlack (base 2), and only then is O rescaled in tensor memory.
//
// P is rounded once to the type of V.  The output is rounded to that type too, and the error of
// p enters it with about the same size: sqrt(2) of the unavoidable error instead of twice the
// work for P V.  For fp16 p is scaled by 2^7 first (2^15 with the slack): weights down to e^-14 of
// the largest keep 11 bits and smaller ones are off by 2^-32 of it at most, 2^-12 for all of the longest
// cache's tokens together; the scale cancels in the division.  (A slack of 4 and a scale of 2^11 would
// give them four bits more, and took 3 % longer on a 16k prompt under a window of 1024, 12 heads.)
//
// Tiles in which some row sees a key that another does not (the diagonal, the window's edge, the
// sinks' end) go past warp 11 first: it zeroes the V rows that no row of the CTA sees, and, since
// a masked weight of 0 would still carry a NaN or infinity of V into the sum, the rows that are
// not finite; those are kept in a bit set, and the rows that do see them add them at the end.
//
// Bound by the tensor cores: a 128 x 64 tile at d 128 takes 8 x 50 cycles for S (6 KB of shared
// memory a product) and 4 x 64 for P V.
//
// Measured (d 128): a prompt of 8191, 32 query and 8 KV heads, pages of 16: 413 to 420 us, 1.3 PFLOP/s.  One
// of 16384 under a window of 1024, 12 heads: 137 to 139 us, 730 TFLOP/s; its 768 CTAs of 19 tiles take five
// waves and a remainder, and the start and end of a CTA, which nothing overlaps, a fifth of the time.  At d 64
// the same prompts take 360 and 113 us: a tile's chain of waits and its exponentials stay, half of the products go.
// 32 queries over 300 to 2000 keys, d 64: 16.4 to 17.3 us.
#include "paged_tc.cuh"

namespace dkv {
namespace {

constexpr int kPfThreads = 384, kPfM = 128, kPfN = 64;
constexpr float kPfSlack = 8.f;
// Rows with scores from here on (in base 2) are left to large_tiles.
constexpr float kPfLarge = 0x1p20f;
constexpr int kPfEdges = 12;  // edge tiles of a CTA (255 positions): 5 on the diagonal, 5 at the window's edge, 1 at the sinks' end

template <typename T>
constexpr float kPfShift = 0.f;
template <>
constexpr float kPfShift<__half> = 7.f;

template <int D>
struct PfSmem {
  static constexpr int kR = 5;                          // slots for K, and for V
  static constexpr uint32_t kQ = kPfM * D * 2;          // one group's Q
  static constexpr uint32_t kTile = kPfN * D * 2;       // one K or V tile
  static constexpr uint32_t kOffK = 2 * kQ;
  static constexpr uint32_t kOffV = kOffK + kR * kTile;
  static constexpr uint32_t kOffBar = kOffV + kR * kTile;
  static constexpr uint32_t kBytes = kOffBar + 512;
};

struct PfKernelArgs {
  PagedArgs a;
  PagedQuery q;
  const void* k_pool;
  const void* v_pool;
  void* out;
  dkv_strides os;
  float* lse;
  int rows;      // query rows of a head in a group: 128, or 8, 16, 32, 64 with 128 / rows heads a group
  int rows_shift;
  int by_heads;  // the groups hold different heads (else two 128-token tiles of one head)
  int heads;     // heads of a CTA
  int per_kv;    // CTAs that share the heads of a KV head
  int parts;     // parts of a row tile's keys at most
  float tile_us, part_us, ratio;  // times of a key tile, and of a part; the first over the second
  float* part_o;     // [CTA][part][256 rows][d] and
  float2* part_stat; // [CTA][part][256 rows] maximum and sum, when parts > 1 (a log-sum-exp would lose a sum
                     // beside a large maximum)
};

// Parts of `tiles` key tiles: as many as take the least time by the model, with kPfJoin us for the join, one
// where that takes no longer.  The grid and its join have to agree, so the roundings are spelled out.
constexpr float kPfJoin = 2.5f;
__device__ inline int pf_parts(const PfKernelArgs& p, int tiles) {
  if (p.parts < 2) return 1;
  const int parts = min(min((int)rintf(__fsqrt_rn(__fmul_rn(p.ratio, (float)tiles))), p.parts), tiles);
  if (parts < 2) return 1;
  const float whole = __fmul_rn(p.tile_us, (float)tiles), cut = __fadd_rn(__fmul_rn(p.tile_us, (float)((tiles + parts - 1) / parts)), __fadd_rn(__fmul_rn(p.part_us, (float)parts), kPfJoin));
  return cut < whole ? parts : 1;
}

// Row `row` of group g of a CTA's 256: its head and token.
struct PfRow {
  int head, token;
  bool live;
};
__device__ inline PfRow pf_row(const PfKernelArgs& p, int kvh, int h0, int row0, int n, int g, int row) {
  PfRow r;
  const int h = h0 + (p.by_heads ? (g * kPfM + row) >> p.rows_shift : 0);  // within the KV head's group
  r.head = kvh * p.a.G + h;
  r.token = row0 + (p.by_heads ? row & (p.rows - 1) : g * kPfM + row);
  r.live = h < p.a.G && r.token < n;
  return r;
}

// natural log-sum-exp of a row's maximum and sum (-inf for a row that sees no key)
template <typename T>
__device__ inline float lse_of(float m, float l) { return (m - kPfShift<T> + log2f(l)) * 0.6931471805599453f; }

// every query at positions [p_lo, p_hi] sees every key of [k0, k0 + kPfN)
__device__ inline bool all_seen(const PagedArgs& a, int k0, int p_lo, int p_hi) {
  return k0 + kPfN - 1 <= p_lo && (a.window == 0 || k0 > p_hi - a.window || k0 + kPfN <= a.sinks);
}

// bit c: the query at position pos sees key k0 + c
__device__ inline unsigned long long pf_sees(const PagedArgs& a, int pos, int k0) {
  const int hi = pos - k0, lo = a.window ? pos - a.window + 1 - k0 : 0, sk = a.sinks - k0;
  auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
  return below(hi + 1) & (~below(lo) | below(sk));
}

// Tiles j .. n - 1 of a row, in the softmax loop's place, where scores are large (rare, so in rolled
// loops).  That loop's fma of score, scale and minus the maximum leaves the rounding of the maximum in the
// exponent: 2^-4 at kPfLarge, but 1 at 2^24, which with slack and shift is past fp16, and hundreds at
// 2^32.  Here the product is rounded as the maximum's was, and the maximum moves at once.  Returns it and
// the sum.
template <typename T, int D>
__device__ __noinline__ float2 large_tiles(const PagedArgs& a, const KeySpan<kPfN>& ks, int t0, int j, int n, int pos, uint32_t tg,
                                           uint64_t* s_full, uint64_t* p_full, uint64_t* o_done, float m, float l) {
  bool ok = true;
#pragma unroll 1
  for (; j < n; ++j) {
    const int buf = j & 1;
    const uint32_t ts = tg + kPfN * buf, to = tg + 128u;
    if (ok) ok = mbar_wait(&s_full[buf], (uint32_t)((j >> 1) & 1), a.err);
    tc_fence_after();
    const unsigned long long sees = pf_sees(a, pos, ks.key(t0 + j));
    float top = m;
#pragma unroll 1
    for (int c = 0; c < kPfN; c += 16) {
      uint32_t s[16];
      tc_ld16(ts + c, s);
      tc_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (sees >> (c + e) & 1ull) top = fmaxf(top, __fmul_rn(__uint_as_float(s[e]), a.scale_log2));
    }
    const float al = top > m ? fast_exp2(m - top) : 1.f;
    m = top;
    if (j > 0 && __any_sync(0xffffffffu, al != 1.f)) {
      if (ok) ok = mbar_wait(&o_done[buf ^ 1], (uint32_t)(((j - 1) >> 1) & 1), a.err);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc_ld16(to + c, o);
        tc_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
        tc_st16(to + c, o);
      }
    }
    const float ms = m == -INFINITY ? 0.f : m;
    l *= al;
#pragma unroll 1
    for (int c = 0; c < kPfN; c += 16) {  // (P's columns c / 2 .. c / 2 + 7 lie over scores that have been read)
      uint32_t s[16], w[8];
      tc_ld16(ts + c, s);
      tc_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float y[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float d = __fadd_rn(__fmul_rn(__uint_as_float(s[e + x]), a.scale_log2), -ms);
          y[x] = sees >> (c + e + x) & 1ull ? fast_exp2(d + kPfShift<T>) : 0.f;
          l += y[x];
        }
        w[e / 2] = Num<T>::pack(y[0], y[1]);
      }
      tc_st8(ts + c / 2, w);
    }
    tc_st_wait();
    tc_fence_before();
    mbar_arrive(&p_full[buf]);
  }
  return make_float2(m, l);
}

// f = the sum of p v in fp32 over the V rows that are not finite and that this row sees, for channels
// c0 .. c0 + 31 (rare, so in plain loops)
template <typename T, int D>
__device__ __noinline__ void add_bad_rows(const PfKernelArgs& p, const PagedArgs& a, int b, int head, int kvh, int qrow, int pos,
                                          int bads, const int* bad_key, const uint32_t* bad_bits, int c0, float m, float il,
                                          float* f) {
  for (int e = 0; e < 32; ++e) f[e] = 0.f;
  const T* qr = static_cast<const T*>(p.q.q) + (int64_t)b * p.q.qs.batch + (int64_t)head * p.q.qs.head + (int64_t)qrow * p.q.qs.token;
  for (int x = 0; x < bads * kPfN; ++x) {
    const int t = bad_key[x / kPfN] + x % kPfN;
    if (!((bad_bits[x / 32] >> (x % 32)) & 1u)) continue;
    if (t > pos || (a.window && t <= pos - a.window && t >= a.sinks)) continue;
    const int page = paged_page(a, b, t);
    if (page >= a.n_pages) continue;
    const int64_t at = page * a.stride_page + kvh * a.stride_head + (t & a.page_mask) * a.stride_token;
    const T* kr = static_cast<const T*>(p.k_pool) + at;
    const T* vr = static_cast<const T*>(p.v_pool) + at + c0;
    float dot = 0.f;
    for (int e = 0; e < D; ++e) dot = fmaf(Num<T>::to_float(qr[e]), Num<T>::to_float(kr[e]), dot);
    const float w = fast_exp2(__fadd_rn(__fmul_rn(dot, a.scale_log2), -m) + kPfShift<T>) * il;
    for (int e = 0; e < 32; ++e) f[e] += w * Num<T>::to_float(vr[e]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPfThreads, 1)
    paged_prefill_kernel(PfKernelArgs p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = PfSmem<D>;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, b);
  // the groups: head and first query row (of all heads the later rows, with more keys, first)
  const int tile = (int)gridDim.z - 1 - (int)blockIdx.z;
  const int row0 = tile * (p.by_heads ? p.rows : 2 * kPfM);
  if (p.parts > 1) griddep_launch();  // the join; without it the next grid on the stream may be anyone's
  if (row0 >= qs.n) return;
  const int part = (int)blockIdx.x % p.parts, hg = (int)blockIdx.x / p.parts;
  const int kvh = hg / p.per_kv, h0 = hg % p.per_kv * p.heads;  // h0: within the KV head's group
  // tokens of the groups, heads of each (0: an empty group)
  const int tokA = min(p.by_heads ? p.rows : kPfM, qs.n - row0), tokB = p.by_heads ? tokA : max(0, min(kPfM, qs.n - row0 - kPfM));
  const int hdA = p.by_heads ? min(kPfM / p.rows, a.G - h0) : 1;
  const int hdB = p.by_heads ? max(0, min(kPfM / p.rows, a.G - h0 - kPfM / p.rows)) : (tokB > 0 ? 1 : 0);
  const int p_lo = qs.off + row0, p_hi = p_lo + (p.by_heads ? tokA : tokA + tokB) - 1;
  const KeySpan<kPfN> ks = key_span<kPfN>(a, p_lo, p_hi);
  const int parts = pf_parts(p, ks.n);
  if (part >= parts) return;  // fewer than a sequence of the table's length would take
  // this part's key tiles; group A's may end a tile or two before B's
  const int t0 = (int)((int64_t)ks.n * part / parts), t1 = (int)((int64_t)ks.n * (part + 1) / parts);
  const int endA = p.by_heads ? ks.n : min(ks.n, max(0, ks.st + (max(0, p_lo + tokA) + kPfN - 1) / kPfN - ks.wt0));
  const int nA = max(0, min(endA, t1) - t0), nB = hdB > 0 ? t1 - t0 : 0;
  const int nt = max(nA, nB);
  auto key_of = [&](int j) { return ks.key(t0 + j); };  // first key of tile j

  const uint32_t sb = smem_u32(smem);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);  // [slot]
  uint64_t* v_full = k_full + S::kR;   // [slot]
  uint64_t* empty = v_full + S::kR;    // [slot] O_j, and so S_j, of both groups are done
  uint64_t* landed = empty + S::kR;    // [edge tile] its V landed, for warp 11 (used once)
  uint64_t* q_full = landed + kPfEdges;
  uint64_t* s_full = q_full + 1;       // [group][buffer]
  uint64_t* p_full = s_full + 4;       // [group][buffer]
  uint64_t* o_done = p_full + 4;       // [group][buffer]
  uint64_t* drain = o_done + 4;        // [group] after a wait that gave up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  int* n_bad = reinterpret_cast<int*>(tmem_slot + 1);
  int* bad_key = n_bad + 1;                                              // [edge] first key of an edge tile with bad rows
  uint32_t* bad_bits = reinterpret_cast<uint32_t*>(bad_key + kPfEdges);  // [edge][2]

  if (threadIdx.x == 0) {
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
    for (int i = 0; i < S::kR; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&empty[i], 2);  // one commit per group
    }
    for (int i = 0; i < kPfEdges; ++i) mbar_init(&landed[i], 1);
    mbar_init(q_full, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kPfM);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
    *n_bad = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc_alloc<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  // K or V tiles; whole warp
  const int rows = min(a.page_mask + 1, kPfN), runs = kPfN / rows;
  auto page_of = [&](int j) {  // lane i < runs: the page of the tile's i-th run of `rows` keys
    const int first = key_of(j) + lane * rows;
    // runs without a visible key: zeros, wherever the table points
    return j < nt && lane < runs && first < ks.hi && (first + rows > ks.lo || first < a.sinks) ? paged_page(a, b, first) : a.n_pages;
  };
  auto load = [&](const CUtensorMap* map, uint32_t to, int j, int page, uint64_t* bar, uint32_t el) {
    if (el) mbar_arrive_expect_tx(bar, S::kTile);
    const int y = key_of(j) & a.page_mask;
#pragma unroll 1  // (here as below: what is short stays in the instruction cache)
    for (int i = 0; i < runs; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
        tma_load_4d(sb + to + hf * kPfN * 128 + i * rows * 128, map, hf * 64, y, kvh, pg, bar, el);
    }
  };
  auto slot_free = [&](int j) {  // the slots of tile j - kR
    if (j >= S::kR) ok = mbar_wait(&empty[j % S::kR], (uint32_t)((j / S::kR - 1) & 1), a.err);
    return ok = __all_sync(0xffffffffu, ok);
  };

  if (warp == 8) {
    // =========================== Q and K
    const uint32_t el = elect_one();
    int j = 0;
    if (nt > 0) {
      const int boxesA = nA > 0 ? hdA : 0;  // (the rows of a group without a tile go out through its place meanwhile)
      if (el) mbar_arrive_expect_tx(q_full, (uint32_t)((boxesA + hdB) * p.rows) * D * 2);
      for (int x = 0; x < boxesA + hdB; ++x) {  // a box of p.rows rows for each head (or 128-token tile)
        const int g = x < boxesA ? 0 : 1, slot = x - g * boxesA;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
          tma_load_4d(sb + g * S::kQ + hf * kPfM * 128 + slot * p.rows * 128, &qmap, hf * 64, p.by_heads ? row0 : row0 + g * kPfM,
                      kvh * a.G + h0 + (p.by_heads ? x : 0), b, q_full, el);
      }
    }
    for (int page = page_of(0); j < nt; ++j) {
      const int next = page_of(j + 1);  // looked up a tile ahead of its use
      if (!slot_free(j)) break;
      load(&kmap, S::kOffK + (j % S::kR) * S::kTile, j, page, &k_full[j % S::kR], el);
      page = next;
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    if (nt > 0) mbar_wait(q_full, 0, a.err);
    for (int x = max(0, j - S::kR); x < j; ++x) mbar_wait(&k_full[x % S::kR], (uint32_t)((x / S::kR) & 1), a.err);
  } else if (warp == 9 || warp == 10) {
    // =========================== products of group g
    // The whole warp walks through here and one elected lane issues: in code that one lane runs
    // alone the operands are not known to be uniform, and an issue took 75 to 150 cycles.  The code
    // is kept short: between two tiles the other warps' code has taken its place in the
    // instruction cache.
    constexpr uint32_t id_s = tc_idesc(Num<T>::kUmma, false, kPfN), id_o = tc_idesc(Num<T>::kUmma, true, D);
    const uint32_t el = elect_one();
    const int g = warp - 9, n = g ? nB : nA, n_other = g ? nA : nB;
    const uint32_t tg = tmem + 256u * g;
    const uint64_t qd = tc_desc(sb + g * S::kQ, 16, 1024);
    uint64_t* const sf = s_full + 2 * g;
    uint64_t* const pf = p_full + 2 * g;
    uint64_t* const od = o_done + 2 * g;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = mbar_wait(bar, parity, a.err);
      __syncwarp();
    };
    int k_sl = 0, v_sl = 0;             // slots of the next K and V tile
    uint32_t k_ph = 0, v_ph = 0;        // and their phases
    auto scores = [&](int j) {
      const int buf = j & 1;
      wait(&k_full[k_sl], k_ph);
      if (j >= 2) wait(&od[buf], (uint32_t)((j - 2) >> 1) & 1u);  // the buffer holds P_{j-2}
      tc_fence_after();
      const uint64_t kd = tc_desc(sb + S::kOffK + k_sl * S::kTile, 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)  // 16 channels: 32 bytes of a 128-byte row, then the next 64 channels
        tc_mma(tg + kPfN * buf, qd + (uint64_t)(((k >> 2) * kPfM * 128 + (k & 3) * 32) >> 4),
               kd + (uint64_t)(((k >> 2) * kPfN * 128 + (k & 3) * 32) >> 4), id_s, k > 0, el);
      tc_commit(&sf[buf], el);
      if (++k_sl == S::kR) { k_sl = 0; k_ph ^= 1u; }
    };
    if (n > 0) {
      wait(q_full, 0);
      scores(0);
      for (int j = 0; j < n; ++j) {
        if (j + 1 < n) scores(j + 1);
        const int buf = j & 1;
        wait(&v_full[v_sl], v_ph);
        wait(&pf[buf], (uint32_t)(j >> 1) & 1u);
        tc_fence_after();
        const uint64_t vd = tc_desc(sb + S::kOffV + v_sl * S::kTile, kPfN * 128, 1024);
        const uint32_t ts = tg + kPfN * buf;
#pragma unroll
        for (int k = 0; k < kPfN / 16; ++k)  // 16 keys: 16 rows of 128 bytes
          tc_mma_ta(tg + 128u, ts + 8u * k, vd + (uint64_t)(k * 16 * 128 >> 4), id_o, k > 0 ? 1u : (j > 0 ? 1u : 0u), el);
        tc_commit(&od[buf], el);
        // once for this group, once more where the other has no tile j
        tc_commit(&empty[v_sl], el);
        if (j >= n_other) tc_commit(&empty[v_sl], el);
        if (++v_sl == S::kR) { v_sl = 0; v_ph ^= 1u; }
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {  // a wait gave up, and the rows may have too: no product outlives the CTA
      tc_commit(&drain[g], el);
      mbar_wait(&drain[g], 0, a.err);
    }
  } else if (warp == 11) {
    // =========================== V, and the rows of its edge tiles
    const uint32_t el = elect_one();
    auto clean = [&](int j, int edge) {
      const int k0 = key_of(j), sl = j % S::kR;
      // (waited for also when another wait has given up: the copy must not outlive the CTA)
      if (!__all_sync(0xffffffffu, mbar_wait(&landed[edge], 0, a.err))) { ok = false; return; }
      const uint32_t vb = sb + S::kOffV + sl * S::kTile;
      uint32_t bad = 0;  // rows lane, lane + 32 with a value that is not finite
      for (int x = 0; x < kPfN / 32; ++x) {
        const int r = 32 * x + lane, t = k0 + r;
        const bool some = t < ks.hi && (t >= ks.lo || t < a.sinks);  // a row of the CTA sees it
        bool odd = false;
        if (some) {  // 0 x is NaN for every x that is not finite, and stays one in the sum
          uint32_t z[2] = {0u, 0u};
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint4 v = lds128(vb + sw128(kPfN, r, ch));
            z[0] = Num<T>::zero_times(v.x, z[0]);
            z[1] = Num<T>::zero_times(v.y, z[1]);
            z[0] = Num<T>::zero_times(v.z, z[0]);
            z[1] = Num<T>::zero_times(v.w, z[1]);
          }
          odd = ((z[0] | z[1]) & 0x7fff7fffu) != 0u;
        }
        if (!some || odd)
          for (int ch = 0; ch < D / 8; ++ch) sts128(vb + sw128(kPfN, r, ch), make_uint4(0, 0, 0, 0));
        const uint32_t bits = __ballot_sync(0xffffffffu, odd);
        if (lane == x) bad = bits;
      }
      if (__any_sync(0xffffffffu, bad)) {
        const int at = *n_bad;
        __syncwarp();
        if (at < kPfEdges) {
          if (lane < kPfN / 32) bad_bits[kPfN / 32 * at + lane] = bad;
          if (lane == 0) { bad_key[at] = k0; *n_bad = at + 1; }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[sl]);
    };
    // V of an edge tile lands on a barrier of its own, and fills its slot once it has been looked over.
    // That is done up to two tiles later, so that the loads behind it go out meanwhile (the slot of tile
    // j is waited for only by tile j + kR).
    int edges = 0, j = 0, todo[2] = {-1, -1}, first = 0, cleaned = 0;  // edge tiles loaded and not yet clean
    auto clean_next = [&]() {
      clean(todo[first], cleaned++);
      todo[first] = -1;
      first ^= 1;
    };
    for (int page = page_of(0); j < nt; ++j) {
      const int next = page_of(j + 1);
      if (!slot_free(j)) break;
      const bool edge = !all_seen(a, key_of(j), p_lo, p_hi);
      load(&vmap, S::kOffV + (j % S::kR) * S::kTile, j, page, edge ? &landed[edges] : &v_full[j % S::kR], el);
      page = next;
      if (todo[first] >= 0 && (todo[first] <= j - 2 || todo[first ^ 1] >= 0)) clean_next();
      if (edge) {
        todo[todo[first] < 0 ? first : first ^ 1] = j;
        ++edges;
      }
    }
    while (todo[first] >= 0) clean_next();
    for (int x = max(0, j - S::kR); x < j; ++x) mbar_wait(&v_full[x % S::kR], (uint32_t)((x / S::kR) & 1), a.err);
  } else if (warp < 8) {
    // =========================== softmax: one query row per thread
    const int g = warp >> 2, rw = warp & 3, row = 32 * rw + lane;
    const int n = g ? nB : nA;
    const PfRow me = pf_row(p, kvh, h0, row0, qs.n, g, row);
    const int pos = qs.off + me.token;
    // positions of the group's rows (the tile is unmasked when all of them see all of it)
    const int g_lo = p.by_heads ? p_lo : p_lo + g * kPfM, g_hi = g_lo + (g ? tokB : tokA) - 1;
    const uint32_t tg = tmem + ((uint32_t)(32 * rw) << 16) + 256u * g, to = tg + 128u;
    const float slog2 = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const int buf = j & 1;
      const uint32_t ts = tg + kPfN * buf;
      if (ok) ok = mbar_wait(&s_full[2 * g + buf], (uint32_t)((j >> 1) & 1), a.err);
      tc_fence_after();
      uint32_t s[kPfN];
#pragma unroll
      for (int c = 0; c < kPfN / 32; ++c) tc_ld32(ts + 32 * c, s + 32 * c);
      tc_ld_wait();
      const int k0 = key_of(j);
      if (!all_seen(a, k0, g_lo, g_hi)) {
        const unsigned long long sees = pf_sees(a, pos, k0);
        if (__any_sync(0xffffffffu, sees != ~0ull)) {
          const uint32_t half[2] = {(uint32_t)sees, (uint32_t)(sees >> 32)};
#pragma unroll
          for (int c = 0; c < kPfN; ++c) s[c] = half[c >> 5] >> (c & 31) & 1u ? s[c] : 0xff800000u;
        }
      }
      float mx[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
      for (int c = 8; c < kPfN; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(s[c]));
      const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * slog2;
      const bool up = top > m + kPfSlack, moved = __any_sync(0xffffffffu, up);
      // (rows that are not live hold whatever was there)
      if (moved && __any_sync(0xffffffffu, me.live && fabsf(top) >= kPfLarge && top > -INFINITY)) {
        const float2 ml = large_tiles<T, D>(a, ks, t0, j, n, pos, tg, s_full + 2 * g, p_full + 2 * g, o_done + 2 * g, m, l);
        m = ml.x;
        l = ml.y;
        break;
      }
      const float al = up ? fast_exp2(m - top) : 1.f;
      if (up) m = top;
      if (j > 0 && moved) {  // rescale O once O_{j-1} is done
        if (ok) ok = mbar_wait(&o_done[2 * g + (buf ^ 1)], (uint32_t)(((j - 1) >> 1) & 1), a.err);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tc_ld32(to + 32 * c, o);
          tc_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
          tc_st32(to + 32 * c, o);
        }
      }
      const float ms = (m == -INFINITY ? 0.f : m) - kPfShift<T>;
      const float2 scale2 = make_float2(slog2, slog2), shift2 = make_float2(-ms, -ms);
      float2 lp[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t w[kPfN / 2];
#pragma unroll
      for (int e = 0; e < kPfN / 2; ++e) {
        const float2 x = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, shift2);
        const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
        lp[e & 1] = add2(lp[e & 1], y);
        w[e] = Num<T>::pack(y.x, y.y);
      }
      tc_st32(ts, w);
      l = fmaf(l, al, (lp[0].x + lp[1].x) + (lp[0].y + lp[1].y));
      tc_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[2 * g + buf]);
    }
    if (n > 0 && ok) ok = mbar_wait(&o_done[2 * g + ((n - 1) & 1)], (uint32_t)(((n - 1) >> 1) & 1), a.err);
    tc_fence_after();
    const bool live = me.live;
    const float il = n == 0 || l == 0.f ? 0.f : 1.f / l;  // a row that sees no key: zeros
    // (every edge tile's product, and so warp 11's work on it, is behind o_done)
    const int bads = n > 0 ? *reinterpret_cast<volatile int*>(n_bad) : 0;
    // The rows go through the group's Q, which no product reads any more, so that a warp then writes
    // whole rows of the output.
    const uint32_t stage = sb + g * S::kQ;
    const int64_t rec = (((int64_t)b * gridDim.z + tile) * (gridDim.x / p.parts) + hg) * p.parts + part;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (n > 0) {
        tc_ld32(to + 32 * c, o);
        tc_ld_wait();
      }
      float f[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) f[e] = n > 0 && l != 0.f ? __uint_as_float(o[e]) * il : 0.f;
      if (bads && live) {
        float more[32];
        add_bad_rows<T, D>(p, a, b, me.head, kvh, me.token, pos, bads, bad_key, bad_bits, 32 * c, m, il, more);
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] += more[e];
      }
      if (parts > 1) {
        if (live) {
          float* o32 = p.part_o + (rec * 2 * kPfM + g * kPfM + row) * D + 32 * c;
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(o32 + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
        continue;
      }
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        sts128(stage + sw128(kPfM, row, (32 * c + e) / 8),
               make_uint4(Num<T>::pack(f[e], f[e + 1]), Num<T>::pack(f[e + 2], f[e + 3]), Num<T>::pack(f[e + 4], f[e + 5]),
                          Num<T>::pack(f[e + 6], f[e + 7])));
    }
    if (parts > 1) {
      if (live) p.part_stat[rec * 2 * kPfM + g * kPfM + row] = make_float2(m, l);
    } else {
      __syncwarp();
      const int ch = lane % (D / 8);  // a row's piece; D / 8 lanes a row
      T* out = static_cast<T*>(p.out) + (int64_t)b * p.os.batch + 8 * ch;
      auto store = [&](const PfRow& first, int r0, int n_rows) {  // rows r0 .. r0 + n_rows - 1, of one head
        if (!first.live) return;
        T* at = out + (int64_t)first.head * p.os.head + (int64_t)first.token * p.os.token;
        const int live_rows = min(n_rows, qs.n - first.token);
#pragma unroll 4
        for (int r = lane / (D / 8); r < live_rows; r += 256 / D)
          *reinterpret_cast<uint4*>(at + (int64_t)r * p.os.token) = lds128(stage + sw128(kPfM, r0 + r, ch));
      };
      const int step = min(p.rows, 32);
      for (int r = 32 * rw; r < 32 * rw + 32; r += step) store(pf_row(p, kvh, h0, row0, qs.n, g, r), r, step);
      if (live && p.lse) p.lse[((int64_t)b * a.Hq + me.head) * p.q.Tq + me.token] = lse_of<T>(m, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tc_free<512>(tmem);
}

// The parts of a row joined: weights l_part 2^(m_part - M), in part order.  A warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_prefill_join_kernel(PfKernelArgs p, int tiles, int hgs) {
  constexpr int V = D / 32;  // channels of a lane
  const PagedArgs& a = p.a;
  griddep_wait();
  const int b = blockIdx.z, tile = (int)blockIdx.y / hgs, hg = (int)blockIdx.y % hgs, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const QuerySpan qs = query_span(a, p.q.q_lens, p.q.Tq, b);
  const int row0 = tile * (p.by_heads ? p.rows : 2 * kPfM), p_lo = qs.off + row0;
  const PfRow me = pf_row(p, hg / p.per_kv, hg % p.per_kv * p.heads, row0, qs.n, row / kPfM, row % kPfM);
  if (!me.live) return;
  const int parts = pf_parts(p, key_span<kPfN>(a, p_lo, p_lo + min(p.by_heads ? p.rows : 2 * kPfM, qs.n - row0) - 1).n);
  if (parts < 2) return;  // written by its one part
  const int64_t rec = (((int64_t)b * tiles + tile) * hgs + hg) * p.parts;
  auto at = [&](int i) { return (rec + i) * 2 * kPfM + row; };
  float M = -INFINITY;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(p.part_stat + at(i)).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float f[V] = {}, L = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 ml = __ldcg(p.part_stat + at(i));
    if (ml.y == 0.f) continue;  // (a NaN goes on)
    const float w = ml.y * fast_exp2(ml.x - M);
    L += w;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 o = __ldcg(reinterpret_cast<const float2*>(p.part_o + at(i) * D + V * lane + e));
      f[e] = fmaf(w, o.x, f[e]);
      f[e + 1] = fmaf(w, o.y, f[e + 1]);
    }
  }
  const float il = L == 0.f ? 0.f : 1.f / L;
  T* out = static_cast<T*>(p.out) + (int64_t)b * p.os.batch + (int64_t)me.head * p.os.head + (int64_t)me.token * p.os.token + V * lane;
#pragma unroll
  for (int e = 0; e < V; e += 2) *reinterpret_cast<uint32_t*>(out + e) = Num<T>::pack(f[e] * il, f[e + 1] * il);
  if (p.lse && lane == 0) p.lse[((int64_t)b * a.Hq + me.head) * p.q.Tq + me.token] = lse_of<T>(M, L);
}

template <typename T, int D>
cudaError_t launch_td(const PfKernelArgs& p, const PagedMaps& m, const CUtensorMap& qmap, cudaStream_t s) {
  constexpr uint32_t smem = PfSmem<D>::kBytes;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(paged_prefill_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.q.Tq + (p.by_heads ? p.rows : 2 * kPfM) - 1) / (p.by_heads ? p.rows : 2 * kPfM);
  const int hgs = p.a.Hkv * p.per_kv;
  paged_prefill_kernel<T, D><<<dim3(hgs * p.parts, p.a.B, tiles), kPfThreads, smem, s>>>(p, qmap, m.k, m.v);
  if ((e = cudaGetLastError()) != cudaSuccess || p.parts == 1) return e;
  return launch_dependent(paged_prefill_join_kernel<T, D>, dim3(2 * kPfM / 8, tiles * hgs, p.a.B), 256, 0, s, p, tiles, hgs);
}

}  // namespace

// Rows of a head in a group.  Up to 64 queries: a power of two, so that a group holds several heads.
int paged_prefill_rows(int Tq) {
  int r = 8;
  while (r < Tq && r < kPfM) r *= 2;
  return r;
}

size_t paged_prefill_ws_bytes(int d) { return kWsHeader + (size_t)sm_count() * 2 * kPfM * (d + 2) * 4; }

cudaError_t launch_paged_prefill(const PagedArgs& a, int d, int dtype, const PagedMaps& m, const CUtensorMap& qmap,
                                 const PagedQuery& q, const void* v_pool, const void* k_pool, void* out,
                                 const dkv_strides& os, float* lse, uint8_t* ws, cudaStream_t s) {
  PfKernelArgs p;
  p.a = a;
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.out = out;
  p.os = os;
  p.lse = lse;
  p.rows = paged_prefill_rows(q.Tq);
  p.rows_shift = 0;
  while ((1 << p.rows_shift) < p.rows) ++p.rows_shift;
  p.by_heads = a.G % 2 == 0 || p.rows < kPfM;
  p.heads = p.by_heads ? 2 * kPfM / p.rows : 1;
  p.per_kv = (a.G + p.heads - 1) / p.heads;
  // Parts of the key tiles, when the grid would fill at most half of the multiprocessors (records for one
  // grid of them are what the workspace holds).  A tile takes 0.85 us; the join 2.5, 0.65 a part, and 2 ps
  // for every value that a part leaves and the join reads.  That fits these times (us; the number of parts
  // in front) of 32 heads at d 128 to within 1.5: 16 queries over 1024 keys 1: 17.9, 2: 15.6, 4: 13.2; over
  // 4096 keys 4: 21.7, 8: 18.0, 16: 23.2; 128 over 1024 1: 20.7, 2: 20.9, 4: 19.3; 512 over 1024 1: 20.6,
  // 2: 25.2.  At d 64 a tile takes 0.6 and the rule is not refitted: 16 queries over 1024 keys 1: 15.4, 2: 13.1,
  // 4: 10.7, 8: 10.6, the rule's 11.1; over 4096 keys 1: 44.6, 4: 18.3, 8: 14.1, 16: 14.9, the rule's 15.2.  Under
  // a window of 1024 the same as over 1024 keys (d 128 4: 13.7, the rule's 13.9).  The grid has room for the parts
  // of the longest sequence that the table allows; how many there are goes by the keys that are there.
  const int tokens = p.by_heads ? p.rows : 2 * kPfM;
  const int64_t ctas = (int64_t)a.Hkv * p.per_kv * a.B * ((q.Tq + tokens - 1) / tokens);
  const int64_t keys = a.window > 0 && (int64_t)a.window + a.sinks + tokens < a.cap ? (int64_t)a.window + a.sinks + tokens : a.cap;
  const int64_t fit = sm_count() / ctas;
  p.tile_us = 0.85f;
  p.part_us = 0.65f + 2e-6f * (float)d * (float)a.B * (float)a.Hq * (float)q.Tq;
  p.ratio = p.tile_us / p.part_us;
  p.parts = 1;
  if (fit > 1) {
    const float tiles = (float)((keys + kPfN - 1) / kPfN);
    float parts = rintf(sqrtf(p.ratio * tiles));
    parts = fminf(fmaxf(parts, 1.f), fminf((float)fit, tiles));
    if (p.tile_us * ceilf(tiles / parts) + kPfJoin + p.part_us * parts < p.tile_us * tiles) p.parts = (int)parts;
  }
  p.part_o = reinterpret_cast<float*>(ws + kWsHeader);
  p.part_stat = reinterpret_cast<float2*>(p.part_o + (size_t)sm_count() * 2 * kPfM * d);
  if (dtype == DKV_BF16)
    return d == 128 ? launch_td<__nv_bfloat16, 128>(p, m, qmap, s) : launch_td<__nv_bfloat16, 64>(p, m, qmap, s);
  return d == 128 ? launch_td<__half, 128>(p, m, qmap, s) : launch_td<__half, 64>(p, m, qmap, s);
}

}  // namespace dkv
