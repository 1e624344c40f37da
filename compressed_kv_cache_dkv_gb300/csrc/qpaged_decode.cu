// dkv_qpaged_decode: attention of one new token per sequence over a cache held in 4 bits.
//
// With key values s c + b (scale, code, bias of a token's group of 64 channels)
//   q . k = sum over groups of  s (q . c) + b (sum of q)         and
//   o = sum over tokens of  (p s) c + p b
// so no value is ever made: the products take the codes themselves as fp16 operands, which the four bits are
// already (c 2^-24 in the low bits of a half, c 2^-20 four bits up, both subnormal and exact; the factor 16 is
// taken out of q, and out of o at the end).  Scales and biases meet scores and weights in fp32.
//
//   S = C_K q    mma.sync m16n8k16, tokens in M, heads in N; a token's 32 bytes a group are a lane's operand as
//                they lie, with q's channels in the same order
//   o = C_V^T w  channels in M; two tokens' words interleaved by byte permutes give the pairs along k
// q is brought to at most 2^15 by a power of two, so that it is an fp16 operand whatever its type (channels above 2^-24
// of the largest without loss).  w = p s 2^-E, with a running power of two E for each head and group, is rounded once to
// fp16 (relative error 2^-11, or 2^-32 of the head's largest product).  That rounding falls on codes less 8 (the sum of
// the rounded weights, times 8, goes off again, and the bias is b + 8 s), so that it is one of about the size of the
// values, as in the 16-bit prefill.  One value is a choice: a second one for what the first leaves took 9 % longer (16
// of 64k: 77.8 us, 71.6 without), and with one the outputs are as far from the definition (2.1e-4 in fp16, 1.7e-3 in
// bf16, root mean square) as a plain form's with fp32 weights.
//
// The visible tokens of a sequence are cut into 32-token tiles; the tiles of all (sequence, KV head) units in a row
// are dealt out evenly, to CTAs and in them to warps.  A warp walks its run of tiles unit by unit with stages, copies
// and an online softmax of its own: it looks up the pages of its next tiles, a lane for each, and fetches a tile with
// one bulk copy per page as soon as a stage is free.  A unit that lies wholly in one warp's run is finished there;
// what lies in several is left in shared memory (a warp's last unit in its own stages, which are free by then, its
// first one beside them) and merged once, at the CTA's end; units that lie in several CTAs' runs leave a record for
// each, and the CTA that is last to leave one merges them in run order, so that equal calls give equal bits.
//
// Bound: memory at 9/8 d bytes a token and KV head; right beside it the instructions that cut codes out of words and
// scale weights (317 a warp for 16 tokens, start and end among them; 0.54 of the issue slots, 0.52 of the integer pipe).  What it took, on 16
// sequences of 64k tokens, 2 KV heads, d 128 (302 MB, floor 45 us): one producer warp with a page look-up for each
// tile 157 us; a look-up for a batch of tiles 96; every warp its own tiles and copies, sixteen warps 78; one fp16
// weight, biases by a product, packed arithmetic 72; one merge a CTA, the join in the same grid 68.  The loop
// streams at 5.8 TB/s (0.87 of the measured copy rate); 4 us at the start (lengths, then the page table, then
// the first copies) and 6 at the end (uneven finish, merge, join) are what is left.  64 sequences of 300 to 8000
// under a window of 4096, 8 KV heads, pages of 16 (237 MB): 65 us.  One of 1000 tokens: 11.3 us in a graph.  The join
// of many records with all loads in flight: one sequence of 65536 tokens, 2 KV heads 18.9 us (23.8 with eight at a
// time, merged as they came).
#include "paged_tc.cuh"
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kQdTile = 32, kQdBlocks = kQdTile / kQBlock;
constexpr int kQdWarps = 16, kQdDepth = 2;  // warps, and stages of each
constexpr int kQdThreads = 32 * kQdWarps;
// Tiles of a CTA, as long as there are enough for all.  In a graph: one sequence of 100 tokens, 8 KV heads 7.9 us
// (with 8: 8.7, with 12: 13.6), of 2000, 2 KV heads 11.4 (11.3, 12.1), 16 of 200, 8 KV heads 9.0 (12.6, 13.8).
constexpr int kQdLeast = 4;
// Sequences of one length (one alone, or all beyond their window) get a number of CTAs that cuts units at equal parts,
// so that no CTA has to join two units one after the other, as long as that adds fewer than so many tiles to a run: one
// sequence of 9000 tokens, 2 KV heads, in a graph 15.0 us (19.9 without), 16 of 200, 8 KV heads, 9.4 (13.1), 10 of
// 1600 15.6 (17.1; below 24 they gained, and 4 of 16000 lost 0.2 of 27.7).  With uneven lengths the whole grid is
// better: 10 of 100 to 1500 14.1 us, 17.3 so.
constexpr int kQdEven = 24;
// Weights are 2^(score - ref).  A head's reference lies kQdShift below a maximum and moves only when a score exceeds
// that by kQdSlack (at once where scores are so large that their rounding shows): weights are at most 2^15, and those
// down to e^-14 of the largest keep 11 bits.
constexpr float kQdShift = 7.f, kQdSlack = 8.f, kQdLarge = 0x1p20f;
// A weight times its token's scale is held times 2^-E as a half.  E, of each head and group of channels, lies 7 below a
// product's exponent, goes with the reference, and moves when a product is above 2^15 (kQdMost, a half's bits).  It follows
// the products, not the scales: with E from the largest scale a token of no weight with values 2^27 times the others'
// left these 4 bits.  A piece's first tile always moves it: 0.3 us of a short call (one of 1000 tokens, 12 / 2 heads, in a
// graph 11.3 us, 11.0 with the scales'), 49.7 us for 512 sequences of 10 to 200 tokens, 8 KV heads (46.9), nothing of long
// ones.  A start by the first tile's largest scale, checked against the products: 48.9 of the 512, but 66.3 us for 16 of
// 64k, 65.8 without.  -E goes up to 96: products below 2^-89, a weight being 2^7 at least, are off by 2^-121.
constexpr uint32_t kQdMost = 0x7800u;
constexpr float kQdFinest = 0x1p96f;
__device__ inline float qd_one_over(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }  // x a power of two

template <int D>
constexpr int qrec_floats() { return 16 + 8 * D; }

struct QSpan {
  int len, lo, st, wt0, n;  // tokens, window start, sink tiles, first window tile, tiles in all
  __device__ int token(int j) const { return (j < st ? j : wt0 + j - st) * kQdTile; }
};
__device__ inline QSpan qd_span(const PagedArgs& a, int b) {
  QSpan s;
  s.len = paged_len(a, b);
  s.lo = paged_window_lo(a, s.len - 1);
  s.wt0 = s.lo / kQdTile;
  s.st = min((min(a.sinks, s.len) + kQdTile - 1) / kQdTile, s.wt0);
  s.n = s.st + (s.len + kQdTile - 1) / kQdTile - s.wt0;
  return s;
}

struct QdArgs {
  PagedArgs a;
  const void* q;
  int64_t q_batch, q_head;
  const uint8_t* cache;
  void* out;
  float* lse;
  float* records;
};

template <int D>
struct QdSmem {
  static constexpr uint32_t kStage = kQdBlocks * qblock_bytes(D);
  static constexpr uint32_t kOffFirst = kQdWarps * kQdDepth * kStage;        // o [warp][D][8] of first units
  static constexpr uint32_t kOffStats = kOffFirst + kQdWarps * D * 32;       // [warp][first, last](ref [8], l [8])
  static constexpr uint32_t kOffBar = kOffStats + kQdWarps * 128;            // [warp][stage]
  static constexpr uint32_t kOffUnit = kOffBar + kQdWarps * kQdDepth * 8;    // [warp] its last unit; the CTA's first one
  static constexpr uint32_t kOffPrefix = kOffUnit + (kQdWarps + 1) * 16;     // [B + 1]
  static_assert(kQdDepth * kStage >= D * 32, "a warp's last unit fits its stages");
};
// Counters of the CTAs that have left a record of a unit: a byte for each CTA in which such a unit can begin, behind
// the header's two words.  They are zero between calls (the last CTA takes its unit's away).
constexpr int kQdMostCtas = 160;

// the (scale, bias) pairs of a token
template <int G>
__device__ inline void lds_params(uint32_t at, uint32_t (&x)[G]) {
  if (G == 2) {
    const uint2 y = lds64(at);
    x[0] = y.x;
    x[G - 1] = y.y;
  } else {
    x[0] = lds32(at);
  }
}
// a product that begins a sum
__device__ inline void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ inline float half_lo(uint32_t x) { return __low2float(*reinterpret_cast<__half2*>(&x)); }
__device__ inline float half_hi(uint32_t x) { return __high2float(*reinterpret_cast<__half2*>(&x)); }

template <typename T, int D>
__global__ void __launch_bounds__(kQdThreads, 1) qpaged_decode_kernel(QdArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using S = QdSmem<D>;
  const PagedArgs& a = p.a;
  constexpr int G = D / 64, BB = qblock_bytes(D);
  float* firsts = reinterpret_cast<float*>(smem + S::kOffFirst);
  float* stats = reinterpret_cast<float*>(smem + S::kOffStats);
  int4* units = reinterpret_cast<int4*>(smem + S::kOffUnit);  // first tile, tiles, sequence, head
  int* prefix = reinterpret_cast<int*>(smem + S::kOffPrefix);
  const int lane = threadIdx.x & 31;
  // (a run of few tiles goes to every fourth of these: to warps of different schedulers)
  const int warp = (threadIdx.x >> 5) % 4 * (kQdWarps / 4) + (threadIdx.x >> 7);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBar) + warp * kQdDepth;
  const uint32_t stages = smem_u32(smem) + warp * kQdDepth * S::kStage;
  auto lasts = [&](int w) { return reinterpret_cast<float*>(smem + w * kQdDepth * S::kStage); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kQdWarps * kQdDepth; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + S::kOffBar) + i, 1);
    fence_mbar_init();
  }
  deal_prefix(a.B, prefix, [&](int b) { return qd_span(a, b).n; });
  __syncthreads();
  // sequences without a token: zeros and -inf
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) {
      T* o = static_cast<T*>(p.out) + (size_t)b * a.Hq * D;
      for (int e = threadIdx.x; e < a.Hq * D; e += kQdThreads) o[e] = Num<T>::from_float(0.f);
      if (p.lse)
        for (int e = threadIdx.x; e < a.Hq; e += kQdThreads) p.lse[(size_t)b * a.Hq + e] = -INFINITY;
    }
  const int total = prefix[a.B] * a.Hkv, c = blockIdx.x;
  int nc = min((int)gridDim.x, (total + kQdLeast - 1) / kQdLeast);
  const int one = prefix[1];  // of one length: a look at the middle and the end will do (all of them took 1 us more)
  if (prefix[a.B] == (int64_t)a.B * one && prefix[a.B / 2] == (int64_t)(a.B / 2) * one) {
    const int units = a.B * a.Hkv, fewer = nc - nc % units;
    if ((float)total * (float)(nc - fewer) < (float)kQdEven * (float)nc * (float)fewer) nc = fewer;
  }
  if (c >= nc) return;
  const int x0 = deal_bound(total, nc, c), x1 = deal_bound(total, nc, c + 1);
  auto bound = [&](int w) { return x0 + (x1 - x0) * w / kQdWarps; };  // of the warps' runs
  const int y0 = bound(warp), y1 = bound(warp + 1);

  // ---- the warp's tiles [y0, y1): a lane looks after one run of slots of a page
  const uint64_t policy = policy_evict_first();  // a cache is read once a step
  const int rows = min(a.page_mask + 1, kQdTile), runs = kQdTile / rows, bpr = rows / kQBlock, batch = 32 / runs;
  const int run_shift = runs == 2 ? 1 : 0, part = lane & (runs - 1);
  uint64_t src = 0;       // of the lane's run: address, bytes, place in the stage
  uint32_t bytes = 0, to = 0, all = 0, none = 0;  // all: the tile's bytes; none: lanes whose page is out of range
  auto look = [&](int xb) {
    const int x = xb + (lane >> run_shift);
    bool bad = false;
    bytes = 0;
    if (x < y1) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, y1);
      const QSpan s = qd_span(a, g.b);
      const int first = s.token(g.j0) + part * rows;
      int b0 = bpr, b1 = 0;  // blocks with a visible token
#pragma unroll 1
      for (int i = 0; i < bpr; ++i) {
        const int t = first + i * kQBlock;
        if (t < s.len && (t + kQBlock > s.lo || t < a.sinks)) {
          b0 = min(b0, i);
          b1 = i + 1;
        }
      }
      if (b0 < b1) {
        const int page = paged_page(a, g.b, first);
        bad = page >= a.n_pages;
        if (!bad) {
          bytes = (uint32_t)(b1 - b0) * BB;
          src = reinterpret_cast<uint64_t>(p.cache) + page * a.stride_page + g.h * a.stride_head +
                (int64_t)((first & a.page_mask) / kQBlock + b0) * BB;
        }
      }
      to = (uint32_t)(part * bpr + b0) * BB;
    }
    none = __ballot_sync(0xffffffffu, bad);
    all = bytes;
    if (runs == 2) all += __shfl_xor_sync(0xffffffffu, bytes, 1);
  };
  bool ok = true;
  int next = y0, slot = batch, in = 0;  // the next tile to fetch, its place in the batch, its stage
  auto fetch = [&]() {
    if (next >= y1 || !ok) return;
    if (slot == batch) {
      look(next);
      slot = 0;
    }
    const uint32_t st = stages + in * S::kStage;
    if (lane >> run_shift == slot) {
      if (part == 0) mbar_arrive_expect_tx(&full[in], all);
      if (bytes)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(st + to),
            "l"(src), "r"(bytes), "r"(smem_u32(&full[in])), "l"(policy)
            : "memory");
    }
    __syncwarp();
    if (none >> (slot << run_shift) & (runs == 2 ? 3u : 1u)) {  // pages of zeros: no scales, no biases
      for (int k = 0; k < kQdBlocks; ++k)
        if (none >> ((slot << run_shift) + k / bpr) & 1u)
          for (int i = lane; i < D / 2; i += 32)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + k * BB + 16 * D + 4 * i), "r"(0u) : "memory");
      fence_proxy_async();
      __syncwarp();
    }
    ++next;
    ++slot;
    if (++in == kQdDepth) in = 0;
  };
  for (int i = 0; i < kQdDepth; ++i) fetch();

  constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u, kOnes = 0x3c003c00u;
  const int t = lane & 3, gq = lane >> 2;
  // the tokens of this lane's rows gq and gq + 8 of a block: in this order a lane's words of V lie four tokens apart
  const int r0 = (gq >> 1) + 4 * (gq & 1), r1 = r0 + 8;
  int out = 0;  // the stage of the next tile
  uint32_t phase = 0;
  for (int x = y0; x < y1;) {
    const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, y1);
    const QSpan s = qd_span(a, g.b);
    // q as B fragments: lane (gq, t) holds channels 16 t .. 16 t + 15 of each group of head gq
    uint32_t qb[G][2][2][2];      // [group][word][even, odd nibbles][b0, b1]
    uint32_t qz;                  // the groups' sums of q, for the biases: t = 0 the fp16 value, t = 1 what it leaves
    float2 kf;                    // factor of the products, heads 2t and 2t + 1
    {
      const bool live = gq < a.G;
      const T* row = static_cast<const T*>(p.q) + g.b * p.q_batch + (int64_t)(g.h * a.G + (live ? gq : 0)) * p.q_head + 16 * t;
      float f[G][16], top = 0.f, sum[2] = {0.f, 0.f};
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        const uint4 v[2] = {__ldg(reinterpret_cast<const uint4*>(row + 64 * gg)), __ldg(reinterpret_cast<const uint4*>(row + 64 * gg + 8))};
        const T* h = reinterpret_cast<const T*>(v);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[gg][e] = live ? Num<T>::to_float(h[e]) : 0.f;
          top = fmaxf(top, fabsf(f[gg][e]));
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int ex = max((int)(__float_as_uint(top) >> 23), 15);   // top < 2^(ex - 126)
      const float up = __uint_as_float((uint32_t)(268 - ex) << 23);  // 2^(141 - ex): top up < 2^15
      const float down = __uint_as_float((uint32_t)(ex - 14) << 23) * 0x1p24f * a.scale_log2;  // 2^(ex - 141), the codes' 2^24
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[gg][e] *= up;
          sum[gg] += f[gg][e];
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], o);
        sum[gg] *= 0x1p-10f;  // (codes carry 2^-24: the other 2^-14 follow the product, so that both parts are normal)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float* y = f[gg] + 8 * w;
          qb[gg][w][0][0] = pack_half2(y[0], y[4]);
          qb[gg][w][0][1] = pack_half2(y[2], y[6]);
          qb[gg][w][1][0] = pack_half2(y[1] * 0.0625f, y[5] * 0.0625f);
          qb[gg][w][1][1] = pack_half2(y[3] * 0.0625f, y[7] * 0.0625f);
        }
      }
      uint32_t hi, lo;
      split_half2(sum[0], sum[1], hi, lo);
      qz = t == 0 ? hi : t == 1 ? lo : 0u;
      kf = make_float2(__shfl_sync(0xffffffffu, down, 8 * t), __shfl_sync(0xffffffffu, down, 8 * t + 4));
    }
    float ref[2] = {-INFINITY, -INFINITY}, lim[2] = {-INFINITY, -INFINITY};
    float2 l = make_float2(0.f, 0.f);
    float o[G][4][4], ow[G][4];  // products with the codes; sums of the rounded weights (the same in all rows)
    float2 ob[G];                // sums of p (b + 8 s)
    float2 inv[G];               // 2^-E
#pragma unroll
    for (int gg = 0; gg < G; ++gg) {
      inv[gg] = make_float2(kQdFinest, kQdFinest);
      ob[gg] = make_float2(0.f, 0.f);
      ow[gg][0] = ow[gg][1] = ow[gg][2] = ow[gg][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[gg][i][0] = o[gg][i][1] = o[gg][i][2] = o[gg][i][3] = 0.f;
    }

    for (int j = g.j0; j < g.j1; ++j) {
      const int tok0 = s.token(j);
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&full[out], phase, a.err))) {
        ok = false;  // nothing more is fetched, and what is on its way has landed before the CTA may end
        for (int i = 0; i < kQdDepth; ++i)
          if (x + j - g.j0 + i < next)
            mbar_wait(&full[(out + i) % kQdDepth], phase ^ (out + i >= kQdDepth ? 1u : 0u), a.err);
      }
      const uint32_t tb = stages + out * S::kStage;
      const bool edge = !((tok0 >= s.lo && tok0 + kQdTile <= s.len) || tok0 + kQdTile <= min(a.sinks, s.len));
      auto seen = [&](int y) { return y < s.len && (y >= s.lo || y < a.sinks); };
      // ---- scores
      float2 sc[kQdBlocks][2];
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k) {
        const uint32_t kb = tb + k * BB;
        uint32_t sbk[2][G];  // scale and bias of the rows' tokens
        lds_params<G>(kb + qparam_off(D, 0, 0, 0) + r0 * 4 * G, sbk[0]);
        lds_params<G>(kb + qparam_off(D, 0, 0, 0) + r1 * 4 * G, sbk[1]);
        float ac[G][4], z[4];
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          const uint2 y0 = lds64(kb + qcode_off(D, 0, gg, 0) + r0 * 32 + 8 * t), y1 = lds64(kb + qcode_off(D, 0, gg, 0) + r1 * 32 + 8 * t);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u0 = w ? y0.y : y0.x, u1 = w ? y1.y : y1.x, v0 = u0 >> 8, v1 = u1 >> 8;
            if (w == 0) mma16816_first(ac[gg], u0 & M0, u1 & M0, v0 & M0, v1 & M0, qb[gg][w][0][0], qb[gg][w][0][1]);
            else mma16816(ac[gg], u0 & M0, u1 & M0, v0 & M0, v1 & M0, qb[gg][w][0][0], qb[gg][w][0][1]);
            mma16816(ac[gg], u0 & M1, u1 & M1, v0 & M1, v1 & M1, qb[gg][w][1][0], qb[gg][w][1][1]);
          }
        }
        // biases (of both groups) times sums of q
        mma16816_first(z, __byte_perm(sbk[0][0], sbk[0][G - 1], 0x7632), __byte_perm(sbk[1][0], sbk[1][G - 1], 0x7632), 0u, 0u, qz, 0u);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 y = mul2(make_float2(z[2 * e], z[2 * e + 1]), make_float2(0x1p-14f, 0x1p-14f));
#pragma unroll
          for (int gg = 0; gg < G; ++gg) {
            const float f = half_lo(sbk[e][gg]);
            y = make_float2(fmaf(f, ac[gg][2 * e], y.x), fmaf(f, ac[gg][2 * e + 1], y.y));
          }
          sc[k][e] = mul2(y, kf);
        }
      }
      if (edge) {
#pragma unroll
        for (int k = 0; k < kQdBlocks; ++k) {
          const int at = tok0 + k * kQBlock;
          if (!seen(at + r0)) sc[k][0] = make_float2(-INFINITY, -INFINITY);
          if (!seen(at + r1)) sc[k][1] = make_float2(-INFINITY, -INFINITY);
        }
        // nothing of V where a weight is 0: its scale and bias may be anything
        if (!seen(tok0 + lane))
#pragma unroll
          for (int gg = 0; gg < G; ++gg)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(tb + lane / kQBlock * BB + qparam_off(D, 1, gg, lane % kQBlock)), "r"(0u) : "memory");
        fence_proxy_async();
        __syncwarp();
      }
      // ---- references (columns 2t, 2t + 1)
      const float top[2] = {fmaxf(fmaxf(sc[0][0].x, sc[0][1].x), fmaxf(sc[1][0].x, sc[1][1].x)),
                            fmaxf(fmaxf(sc[0][0].y, sc[0][1].y), fmaxf(sc[1][0].y, sc[1][1].y))};
      if (__any_sync(0xffffffffu, top[0] > lim[0] || top[1] > lim[1])) {
        float al[2], up[2];  // up: a power of two, al up in [1, 2)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = top[e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
          al[e] = 1.f;
          if (y > lim[e]) {
            al[e] = fast_exp2(ref[e] - (y - kQdShift));
            ref[e] = y - kQdShift;
            lim[e] = ref[e] + (fabsf(y) < kQdLarge ? kQdShift + kQdSlack : kQdShift);
          }
          up[e] = __uint_as_float((254u << 23) - (__float_as_uint(al[e]) & 0x7f800000u));
        }
        l = mul2(l, make_float2(al[0], al[1]));
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {  // the products' power of two goes with the reference
          const float2 to = make_float2(fminf(inv[gg].x * up[0], kQdFinest), fminf(inv[gg].y * up[1], kQdFinest));
          const float f0 = al[0] * (to.x * qd_one_over(inv[gg].x)), f1 = al[1] * (to.y * qd_one_over(inv[gg].y));
          inv[gg] = to;
          ob[gg] = mul2(ob[gg], make_float2(al[0], al[1]));
          ow[gg][0] *= f0;
          ow[gg][1] *= f1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[gg][i][0] *= f0;
            o[gg][i][1] *= f1;
            o[gg][i][2] *= f0;
            o[gg][i][3] *= f1;
          }
        }
      }
      const float2 off = make_float2(ref[0] == -INFINITY ? 0.f : -ref[0], ref[1] == -INFINITY ? 0.f : -ref[1]);
      // ---- weights p, and p s 2^-E as halves
      uint32_t wt[kQdBlocks][2][G], most = 0;
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k) {
        uint32_t sv[2][G];
        lds_params<G>(tb + k * BB + qparam_off(D, 1, 0, 0) + r0 * 4 * G, sv[0]);
        lds_params<G>(tb + k * BB + qparam_off(D, 1, 0, 0) + r1 * 4 * G, sv[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // rows gq and gq + 8
          const float2 x = add2(sc[k][e], off);
          sc[k][e] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          l = add2(l, sc[k][e]);
#pragma unroll
          for (int gg = 0; gg < G; ++gg) {
            const float s1 = half_lo(sv[e][gg]), mid = fmaf(8.f, s1, half_hi(sv[e][gg]));
            ob[gg] = fma2(sc[k][e], make_float2(mid, mid), ob[gg]);
            const float2 w = mul2(sc[k][e], mul2(inv[gg], make_float2(s1, s1)));
            wt[k][e][gg] = pack_half2(w.x, w.y);
            most = __vmaxu2(most, wt[k][e][gg]);
          }
        }
      }
      if (__any_sync(0xffffffffu, (most & 0xffffu) > kQdMost || most >> 16 > kQdMost)) {  // E follows the largest product
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          float2 m = make_float2(0.f, 0.f);
          float s1[kQdBlocks][2];
#pragma unroll
          for (int k = 0; k < kQdBlocks; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s1[k][e] = half_lo(lds32(tb + k * BB + qparam_off(D, 1, gg, 0) + (e ? r1 : r0) * 4 * G));
              const float2 w = mul2(sc[k][e], mul2(inv[gg], make_float2(s1[k][e], s1[k][e])));
              m = make_float2(fmaxf(m.x, w.x), fmaxf(m.y, w.y));
            }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            m = make_float2(fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, off)), fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, off)));
          // (each head by its own products alone; the factor brings the largest into [2^7, 2^8))
          const uint32_t h = pack_half2(m.x, m.y);
          const float f0 = (h & 0xffffu) > kQdMost ? __uint_as_float((261u << 23) - (__float_as_uint(m.x) & 0x7f800000u)) : 1.f;
          const float f1 = h >> 16 > kQdMost ? __uint_as_float((261u << 23) - (__float_as_uint(m.y) & 0x7f800000u)) : 1.f;
          inv[gg] = mul2(inv[gg], make_float2(f0, f1));
          ow[gg][0] *= f0;
          ow[gg][1] *= f1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[gg][i][0] *= f0;
            o[gg][i][1] *= f1;
            o[gg][i][2] *= f0;
            o[gg][i][3] *= f1;
          }
#pragma unroll
          for (int k = 0; k < kQdBlocks; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 w = mul2(sc[k][e], mul2(inv[gg], make_float2(s1[k][e], s1[k][e])));
              wt[k][e][gg] = pack_half2(w.x, w.y);
            }
        }
      }
      // ---- the product with V's codes
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k) {
        const uint32_t vb = tb + k * BB;
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          const uint32_t bw[2] = {movtrans(wt[k][0][gg]), movtrans(wt[k][1][gg])};
          mma16816(ow[gg], kOnes, kOnes, kOnes, kOnes, bw[0], bw[1]);
          uint32_t y[4], z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = lds32(vb + qcode_off(D, 1, gg, 0) + (4 * i + t) * 32 + 4 * gq);
          z[0] = __byte_perm(y[0], y[1], 0x5410);
          z[1] = __byte_perm(y[0], y[1], 0x7632);
          z[2] = __byte_perm(y[2], y[3], 0x5410);
          z[3] = __byte_perm(y[2], y[3], 0x7632);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (i < 2 ? z[e] : z[e] >> 8) & (i & 1 ? M1 : M0);
            mma16816(o[gg][i], f[0], f[1], f[2], f[3], bw[0], bw[1]);
          }
        }
      }
      __syncwarp();
      fetch();  // into the stage just read
      if (++out == kQdDepth) {
        out = 0;
        phase ^= 1u;
      }
    }
    // ---- the piece's sums: l and ob over the rows, o as [gg][i, i + 4]
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l.x += __shfl_xor_sync(0xffffffffu, l.x, off);
      l.y += __shfl_xor_sync(0xffffffffu, l.y, off);
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        ob[gg].x += __shfl_xor_sync(0xffffffffu, ob[gg].x, off);
        ob[gg].y += __shfl_xor_sync(0xffffffffu, ob[gg].y, off);
      }
    }
    float2 v[G][8];  // channels 64 gg + 8 gq + 0 .. 7 of heads 2t, 2t + 1
#pragma unroll
    for (int gg = 0; gg < G; ++gg) {
      const float F0 = qd_one_over(inv[gg].x), F1 = qd_one_over(inv[gg].y);  // 2^E
      const float m0 = fmaf(-8.f * F0, ow[gg][0], ob[gg].x), m1 = fmaf(-8.f * F1, ow[gg][1], ob[gg].y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f0 = F0 * (i & 1 ? 0x1p20f : 0x1p24f), f1 = F1 * (i & 1 ? 0x1p20f : 0x1p24f);
        v[gg][i] = make_float2(fmaf(o[gg][i][0], f0, m0), fmaf(o[gg][i][1], f1, m1));
        v[gg][i + 4] = make_float2(fmaf(o[gg][i][2], f0, m0), fmaf(o[gg][i][3], f1, m1));
      }
    }
    if (g.j0 == 0 && g.j1 == g.n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (2 * t + e >= a.G) continue;
        const float L = e ? l.y : l.x, il = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no weight at all: zeros; a NaN stays one
        const size_t head = (size_t)g.b * a.Hq + g.h * a.G + 2 * t + e;
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = Num<T>::pack((e ? v[gg][2 * i].y : v[gg][2 * i].x) * il, (e ? v[gg][2 * i + 1].y : v[gg][2 * i + 1].x) * il);
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + head * D + 64 * gg + 8 * gq) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (p.lse && gq == 0) p.lse[head] = (ref[e] + log2f(L)) * 0.6931471805599453f;
      }
    } else {
      const bool last = x + g.j1 - g.j0 == y1;
      float* at = last ? lasts(warp) : firsts + warp * D * 8;
      float* st = stats + warp * 32 + (last ? 16 : 0);
      if (lane < 4) {
        *reinterpret_cast<float2*>(st + 2 * t) = make_float2(ref[0], ref[1]);
        *reinterpret_cast<float2*>(st + 8 + 2 * t) = l;
      }
#pragma unroll
      for (int gg = 0; gg < G; ++gg)
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float2*>(at + ((gg * 8 + i) * 8 + gq) * 8 + 2 * t) = v[gg][i];
    }
    if (lane == 0) {
      const int4 u = make_int4(x - g.j0, g.n, g.b, g.h);
      if (x + g.j1 - g.j0 == y1) units[warp] = u;
      if (x == x0) units[kQdWarps] = u;
    }
    x += g.j1 - g.j0;
  }
  __syncthreads();

  // ---- units that lie in several warps' runs, or are cut by the CTA's.  Lane w looks after warp w.
  const int gg = threadIdx.x & 7, b0 = bound(min(lane, kQdWarps)), b1 = bound(min(lane + 1, kQdWarps));
  const uint32_t used = __ballot_sync(0xffffffffu, b0 < b1);
  const int4 cta_first = units[kQdWarps], cta_last = units[31 - __clz(used)];
  // each unit once: as the CTA's first one, or with the first warp whose last unit it is
  const int4 mine = units[min(lane, kQdWarps)];
  const uint32_t todo = __ballot_sync(0xffffffffu, b0 < b1 && mine.x != cta_first.x && b0 <= mine.x);
  const int n_units = __popc(todo) + 1;
  int team = kQdWarps;  // warps of a unit: as many units side by side as there are
  while (team > 1 && kQdWarps / team < n_units) team >>= 1;
  for (int k = (threadIdx.x >> 5) / team; k < n_units; k += kQdWarps / team) {
    uint32_t bits = todo;
    for (int i = 1; i < k; ++i) bits &= bits - 1;
    const int4 u = units[k == 0 ? kQdWarps : __ffs(bits) - 1];
    const int xs = max(u.x, x0), xe = min(u.x + u.y, x1);
    const uint32_t mask = __ballot_sync(0xffffffffu, b0 < b1 && b0 < xe && b1 > xs);      // warps with a piece
    const uint32_t ends = __ballot_sync(0xffffffffu, b1 <= xe);                           // whose last unit it is
    if (__any_sync(0xffffffffu, b0 < b1 && b0 <= u.x && u.x + u.y <= b1)) continue;       // written already
    float M = -INFINITY, L = 0.f, f[kQdWarps];
#pragma unroll
    for (int i = 0; i < kQdWarps; ++i) {
      f[i] = -INFINITY;
      if (mask >> i & 1u) f[i] = stats[i * 32 + (ends >> i & 1u ? 16 : 0) + gg];
      M = fmaxf(M, f[i]);
    }
    const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int i = 0; i < kQdWarps; ++i)
      if (mask >> i & 1u) {
        f[i] = fast_exp2(f[i] - Ms);
        L += f[i] * stats[i * 32 + (ends >> i & 1u ? 16 : 0) + 8 + gg];
      }
    const bool whole = u.x >= x0 && u.x + u.y <= x1;
    const float il = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    float* rec = p.records + (size_t)(2 * c + (u.x >= x0 ? 1 : 0)) * qrec_floats<D>();
    const size_t head = (size_t)u.z * a.Hq + u.w * a.G + gg;
    const int e0 = threadIdx.x % (32 * team);
#pragma unroll 2
    for (int e = e0; e < D * 8; e += 32 * team) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kQdWarps; ++i)
        if (mask >> i & 1u) v += f[i] * (ends >> i & 1u ? lasts(i) : firsts + i * D * 8)[e];
      const int dd = e >> 3, ch = (dd & ~63) + 8 * (dd & 7) + (dd >> 3 & 7);
      if (!whole) rec[16 + ch * 8 + gg] = v;
      else if (gg < a.G) static_cast<T*>(p.out)[head * D + ch] = Num<T>::from_float(v * il);
    }
    if (e0 < 8) {
      if (!whole) {
        rec[gg] = M;
        rec[8 + gg] = L;
      } else if (gg < a.G && p.lse) {
        p.lse[head] = (M + log2f(L)) * 0.6931471805599453f;
      }
    }
  }

  // ---- units that lie in several CTAs' runs: the last to leave its record merges them
  __shared__ int joins[2];  // the records of the CTA's first and last unit, if it is the one
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    for (int i = 0; i < 2; ++i) {
      const int4 u = i ? cta_last : cta_first;
      joins[i] = 0;
      if (u.x >= x0 && u.x + u.y <= x1) continue;
      if (i && u.x == cta_first.x) continue;
      const int c0 = deal_owner(total, nc, u.x), n = deal_owner(total, nc, u.x + u.y - 1) - c0 + 1, at = 8 * (c0 & 3);
      uint32_t* word = a.err + 2 + c0 / 4;
      if ((int)(atomicAdd(word, 1u << at) >> at & 255u) + 1 == n) {
        atomicSub(word, (uint32_t)n << at);
        joins[i] = n;
      }
    }
    __threadfence();
  }
  __syncthreads();
  if (joins[0] | joins[1]) {  // with both, each has half the warps
    const bool both = joins[0] && joins[1];
    const int threads = both ? kQdThreads / 2 : kQdThreads, tid = threadIdx.x & (threads - 1);
    const int k = both ? threadIdx.x >> 8 : joins[1] ? 1 : 0, n = joins[k];
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + k), "r"(threads) : "memory"); };
    const int4 u = k ? cta_last : cta_first;
    const int c0 = deal_owner(total, nc, u.x);
    constexpr int kStep = 2 * qrec_floats<D>();  // from a CTA's record to the next one's; the first is a CTA's second
    auto rec = [&](int i) { return p.records + (size_t)(c0 + i) * kStep + (i == 0 ? kStep / 2 : 0); };
    // Eight warps turn a head's references into factors each while the first records are on their way; groups of
    // threads take records in turn, four values a thread (loads that wait for one another cost a microsecond each).
    // The sums are over every kParts-th record, whichever threads make them.
    constexpr int kDeep = 8, kQuads = D * 2, kParts = kQdThreads / kQuads, kStats = (kQdMostCtas + 31) / 32;
    constexpr int kRoom = 8 * kQdMostCtas + 16 > 4 * kQdThreads ? 8 * kQdMostCtas + 16 : 4 * kQdThreads;
    static_assert(2 * kRoom <= kQdWarps * D * 8, "the factors of two units");
    float* fac = firsts + k * kRoom;                           // [record][8]
    float* red = fac + 8 * kQdMostCtas;                        // M, L [8] each
    float* part = reinterpret_cast<float*>(smem) + k * kRoom;  // [kParts][D][8]
    const int groups = threads / kQuads, pw = tid >> 5, grp = tid / kQuads;
    const int at = tid % kQuads;  // heads 4 (at % 2) .. + 3 of a channel
    const int n4 = 4 * (at & 1) < a.G ? n : 0;                              // (those that are not there are not read)
    float4 y[kDeep], sum = make_float4(0.f, 0.f, 0.f, 0.f), odd = sum;
    auto fetch = [&](int i0) {
      const float4* from = reinterpret_cast<const float4*>(rec(i0) + 16) + at;
#pragma unroll
      for (int i = 0; i < kDeep; ++i)
        if (i0 + i * groups < n4) y[i] = __ldcg(from + i * (groups * kStep / 4) - (i && i0 == 0 ? kStep / 8 : 0));
    };
    float m[kStats], l[kStats];
    if (pw < 8) {
#pragma unroll
      for (int i = 0; i < kStats; ++i) {
        const bool is = lane + 32 * i < n;
        m[i] = is ? __ldcg(rec(lane + 32 * i) + pw) : -INFINITY;
        l[i] = is ? __ldcg(rec(lane + 32 * i) + 8 + pw) : 0.f;
      }
    }
    fetch(grp);
    if (pw < 8) {
      float M = m[0], L = 0.f;
#pragma unroll
      for (int i = 1; i < kStats; ++i) M = fmaxf(M, m[i]);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int i = 0; i < kStats; ++i) {
        const float f = fast_exp2(m[i] - Ms);
        if (lane + 32 * i < n) fac[(lane + 32 * i) * 8 + pw] = f;
        L += f * l[i];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (lane == 0) {
        red[pw] = M;
        red[8 + pw] = L;
      }
    }
    sync();
    for (int i0 = grp;;) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        if (i0 + i * groups >= n4) continue;
        const float4 f = reinterpret_cast<const float4*>(fac + (i0 + i * groups) * 8)[at & 1];
        float4& to = both && i % 2 ? odd : sum;
        to = make_float4(fmaf(f.x, y[i].x, to.x), fmaf(f.y, y[i].y, to.y), fmaf(f.z, y[i].z, to.z), fmaf(f.w, y[i].w, to.w));
      }
      if ((i0 += kDeep * groups) >= n4) break;
      fetch(i0);
    }
    reinterpret_cast<float4*>(part)[tid] = sum;
    if (both) reinterpret_cast<float4*>(part)[threads + tid] = odd;
    sync();
    const float M = red[gg], L = red[8 + gg], il = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const size_t head = (size_t)u.z * a.Hq + u.w * a.G + gg;
    if (gg < a.G) {
      for (int e = tid; e < D * 8; e += threads) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) v += part[i * D * 8 + e];
        static_cast<T*>(p.out)[head * D + (e >> 3)] = Num<T>::from_float(v * il);
      }
      if (p.lse && tid < 8) p.lse[head] = (M + log2f(L)) * 0.6931471805599453f;
    }
  }
}

template <typename T, int D>
cudaError_t launch_qdecode_td(const QdArgs& p, cudaStream_t s) {
  const int ncta = sm_count() < kQdMostCtas ? sm_count() : kQdMostCtas;
  const size_t smem = QdSmem<D>::kOffPrefix + ((size_t)p.a.B + 1) * 4;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(qpaged_decode_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  qpaged_decode_kernel<T, D><<<ncta, kQdThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t qpaged_decode_ws_bytes(int d) { return kWsHeader + (size_t)2 * sm_count() * (16 + 8 * d) * 4; }

cudaError_t launch_qpaged_decode(const PagedArgs& a, int d, int dtype, const void* q, const dkv_strides& qs,
                                 const uint8_t* cache, void* out, float* lse, uint8_t* ws, cudaStream_t s) {
  QdArgs p;
  p.a = a;
  p.q = q;
  p.q_batch = qs.batch;
  p.q_head = qs.head;
  p.cache = cache;
  p.out = out;
  p.lse = lse;
  p.records = reinterpret_cast<float*>(ws + kWsHeader);
  if (dtype == DKV_BF16)
    return d == 128 ? launch_qdecode_td<__nv_bfloat16, 128>(p, s) : launch_qdecode_td<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_qdecode_td<__half, 128>(p, s) : launch_qdecode_td<__half, 64>(p, s);
}

}  // namespace dkv
