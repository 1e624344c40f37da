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
// q is brought to at most 2^15 by a power of two (bf16 queries become fp16 without loss above 2^-24 of the largest),
// w = p s 2^(14 - E) with a running power of two E over the scales seen, as the sum of two fp16 values (22 bits).
//
// The visible tokens of a sequence are cut into 64-token tiles, dealt out evenly to the CTAs as in the
// 16-bit decode; a producer warp streams tiles with bulk copies (one per page, or for larger pages one per tile),
// kQdWarps consumer warps take tiles in turn, each with its own online softmax, merged at a unit's end; units
// that lie in several CTAs' runs leave records that a second grid joins in run order.
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kQdTile = 64, kQdBlocks = kQdTile / kQBlock;
constexpr int kQdWarps = 8;
constexpr int kQdStages = 2 * kQdWarps;  // a multiple of it: a stage belongs to one warp, which so sees each of its phases
constexpr int kQdThreads = 32 * (kQdWarps + 1);
constexpr int kQdCombThreads = 512, kQdCombCols = 32;
constexpr float kQdShift = 14.f;  // weights carry 2^14: those down to e^-18 of the largest keep 11 bits

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
  static constexpr uint32_t kOffMerge = kQdStages * kStage;                  // o [warp][D][8]
  static constexpr uint32_t kOffStats = kOffMerge + kQdWarps * D * 32;       // m, l [warp][2][8]
  static constexpr uint32_t kOffBar = kOffStats + kQdWarps * 64;             // full, empty [stage]
  static constexpr uint32_t kOffBad = kOffBar + kQdStages * 16;              // [stage] blocks on bad pages
  static constexpr uint32_t kOffPrefix = kOffBad + kQdStages * 4;            // [B + 1]
};

__device__ inline float half_lo(uint32_t x) { return __low2float(*reinterpret_cast<__half2*>(&x)); }
__device__ inline float half_hi(uint32_t x) { return __high2float(*reinterpret_cast<__half2*>(&x)); }

template <typename T, int D>
__global__ void __launch_bounds__(kQdThreads, 1) qpaged_decode_kernel(QdArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = QdSmem<D>;
  const PagedArgs& a = p.a;
  constexpr int G = D / 64, BB = qblock_bytes(D);
  float* merge = reinterpret_cast<float*>(smem + S::kOffMerge);
  float* stats = reinterpret_cast<float*>(smem + S::kOffStats);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* empty = full + kQdStages;
  volatile uint32_t* bad_blocks = reinterpret_cast<uint32_t*>(smem + S::kOffBad);
  int* prefix = reinterpret_cast<int*>(smem + S::kOffPrefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = smem_u32(smem);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kQdStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    fence_mbar_init();
  }
  deal_prefix(a.B, prefix, [&](int b) { return qd_span(a, b).n; });
  __syncthreads();
  griddep_launch();
  // sequences without a token: zeros and -inf
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) {
      T* o = static_cast<T*>(p.out) + (size_t)b * a.Hq * D;
      for (int e = threadIdx.x; e < a.Hq * D; e += kQdThreads) o[e] = Num<T>::from_float(0.f);
      if (p.lse)
        for (int e = threadIdx.x; e < a.Hq; e += kQdThreads) p.lse[(size_t)b * a.Hq + e] = -INFINITY;
    }
  const int total = prefix[a.B] * a.Hkv, nc = min((int)gridDim.x, total), c = blockIdx.x;
  if (c >= nc) return;
  const int x0 = deal_bound(total, nc, c), x1 = deal_bound(total, nc, c + 1);

  if (warp == kQdWarps) {
    // =========================== producer
    const uint32_t el = elect_one();
    const uint64_t policy = policy_evict_first();  // a cache is read once a step
    const int rows = min(a.page_mask + 1, kQdTile), runs = kQdTile / rows, bpr = rows / kQBlock;  // a copy per run of a page
    bool ok = true;
    int it = 0;
    for (int x = x0; x < x1 && ok;) {
      const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
      const QSpan s = qd_span(a, g.b);
      for (int j = g.j0; j < g.j1; ++j, ++it) {
        const int st = it % kQdStages, first = s.token(j) + lane * rows;
        // lane i < runs: its page, and the run's blocks that hold a visible token
        int page = -1, b0 = bpr, b1 = 0;
        bool bad = false;
        if (lane < runs) {
          for (int i = 0; i < bpr; ++i) {
            const int t = first + i * kQBlock;
            if (t < s.len && (t + kQBlock > s.lo || t < a.sinks)) {
              b0 = min(b0, i);
              b1 = i + 1;
            }
          }
          if (b0 < b1) {
            page = paged_page(a, g.b, first);
            bad = page >= a.n_pages;
          }
        }
        const uint32_t none = __ballot_sync(0xffffffffu, bad);
        const bool copies = b0 < b1 && !bad;
        const uint32_t bytes = copies ? (uint32_t)(b1 - b0) * BB : 0u;
        uint32_t sum = bytes;
#pragma unroll
        for (int o = 1; o < kQdBlocks; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        const uint64_t src = reinterpret_cast<uint64_t>(p.cache) +
                             (copies ? page * a.stride_page + g.h * a.stride_head + (int64_t)((first & a.page_mask) / kQBlock + b0) * BB : 0);
        const uint32_t dst = sb + st * S::kStage + (uint32_t)(lane * bpr + b0) * BB;
        if (it >= kQdStages) ok = mbar_wait(&empty[st], (uint32_t)((it / kQdStages - 1) & 1), a.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        if (el) {
          uint32_t m = 0;  // bad runs as a mask of blocks
          for (int i = 0; i < kQdBlocks; ++i) m |= (none >> (i / bpr) & 1u) << i;
          bad_blocks[st] = m;
          mbar_arrive_expect_tx(&full[st], sum);
        }
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < runs; ++i) {
          const uint32_t n = __shfl_sync(0xffffffffu, bytes, i), to = __shfl_sync(0xffffffffu, dst, i);
          const uint64_t from = __shfl_sync(0xffffffffu, src, i);
          if (n && el)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(to),
                "l"(from), "r"(n), "r"(smem_u32(&full[st])), "l"(policy)
                : "memory");
        }
      }
      x += g.j1 - g.j0;
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    for (int i = max(0, it - kQdStages); i < it; ++i) mbar_wait(&full[i % kQdStages], (uint32_t)((i / kQdStages) & 1), a.err);
    return;
  }

  // =========================== consumers
  constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
  const int t = lane & 3, gq = lane >> 2;
  // the tokens of this lane's rows gq and gq + 8 of a block: in this order a lane's words of V lie four tokens apart
  const int r0 = (gq >> 1) + 4 * (gq & 1), r1 = r0 + 8;
  bool ok = true;
  int it = 0;
  for (int x = x0; x < x1;) {
    const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x, x1);
    const QSpan s = qd_span(a, g.b);
    // q as B fragments: lane (gq, t) holds channels 16 t .. 16 t + 15 of each group of head gq
    uint32_t qb[G][2][2][2];      // [group][word][even, odd nibbles][b0, b1]
    float kf[2], qs[G][2];        // per head 2t, 2t + 1: factor of the products, sums of q times scale
    {
      const bool live = gq < a.G;
      const T* row = static_cast<const T*>(p.q) + g.b * p.q_batch + (int64_t)(g.h * a.G + (live ? gq : 0)) * p.q_head + 16 * t;
      float f[G][16], top = 0.f, sum[G];
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        sum[gg] = 0.f;
        const uint4 v[2] = {__ldg(reinterpret_cast<const uint4*>(row + 64 * gg)), __ldg(reinterpret_cast<const uint4*>(row + 64 * gg + 8))};
        const T* h = reinterpret_cast<const T*>(v);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[gg][e] = live ? Num<T>::to_float(h[e]) : 0.f;
          top = fmaxf(top, fabsf(f[gg][e]));
          sum[gg] += f[gg][e];
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], o);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int ex = max((int)(__float_as_uint(top) >> 23), 15);   // top < 2^(ex - 126)
      const float up = __uint_as_float((uint32_t)(268 - ex) << 23);  // 2^(141 - ex): top up < 2^15
      const float down = __uint_as_float((uint32_t)(ex - 14) << 23) * 0x1p24f * a.scale_log2;  // 2^(ex - 141), the codes' 2^24
#pragma unroll
      for (int gg = 0; gg < G; ++gg)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float* y = f[gg] + 8 * w;
          qb[gg][w][0][0] = pack_half2(y[0] * up, y[4] * up);
          qb[gg][w][0][1] = pack_half2(y[2] * up, y[6] * up);
          qb[gg][w][1][0] = pack_half2(y[1] * up * 0.0625f, y[5] * up * 0.0625f);
          qb[gg][w][1][1] = pack_half2(y[3] * up * 0.0625f, y[7] * up * 0.0625f);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kf[e] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * e);
#pragma unroll
        for (int gg = 0; gg < G; ++gg) qs[gg][e] = __shfl_sync(0xffffffffu, sum[gg], 8 * t + 4 * e) * a.scale_log2;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[G][4][4], ob[G][2];  // products with the codes; sums of p b
    int E[G];                    // exponent over the scales seen (as of fp32 bits)
#pragma unroll
    for (int gg = 0; gg < G; ++gg) {
      E[gg] = 0;
      ob[gg][0] = ob[gg][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[gg][i][0] = o[gg][i][1] = o[gg][i][2] = o[gg][i][3] = 0.f;
    }

    for (int j = g.j0; j < g.j1; ++j, ++it) {
      if (it % kQdWarps != warp) continue;
      const int st = it % kQdStages, tok0 = s.token(j);
      if (ok) ok = mbar_wait(&full[st], (uint32_t)((it / kQdStages) & 1), a.err);
      const uint32_t tb = sb + st * S::kStage, bad = bad_blocks[st];
      const bool edge = !((tok0 >= s.lo && tok0 + kQdTile <= s.len) || tok0 + kQdTile <= min(a.sinks, s.len));
      // ---- scores
      float sc[kQdBlocks][4];
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k) {
        const uint32_t kb = tb + k * BB;
        float ac[G][4] = {};
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          const uint2 y0 = lds64(kb + qcode_off(D, 0, gg, 0) + r0 * 32 + 8 * t), y1 = lds64(kb + qcode_off(D, 0, gg, 0) + r1 * 32 + 8 * t);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t u0 = w ? y0.y : y0.x, u1 = w ? y1.y : y1.x, v0 = u0 >> 8, v1 = u1 >> 8;
            mma16816(ac[gg], u0 & M0, u1 & M0, v0 & M0, v1 & M0, qb[gg][w][0][0], qb[gg][w][0][1]);
            mma16816(ac[gg], u0 & M1, u1 & M1, v0 & M1, v1 & M1, qb[gg][w][1][0], qb[gg][w][1][1]);
          }
        }
        uint32_t sb0[G], sb1[G];  // scale and bias of the rows' tokens
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          sb0[gg] = lds32(kb + qparam_off(D, 0, gg, 0) + r0 * 4 * G);
          sb1[gg] = lds32(kb + qparam_off(D, 0, gg, 0) + r1 * 4 * G);
          if (bad >> k & 1u) sb0[gg] = sb1[gg] = 0u;  // a page of zeros
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = 0.f, z = 0.f;
#pragma unroll
          for (int gg = 0; gg < G; ++gg) {
            const uint32_t sbx = e < 2 ? sb0[gg] : sb1[gg];
            y = fmaf(half_lo(sbx), ac[gg][e], y);
            z = fmaf(half_hi(sbx), qs[gg][e & 1], z);
          }
          sc[k][e] = fmaf(y, kf[e & 1], z);
        }
        if (edge) {
          auto seen = [&](int y) { return y < s.len && (y >= s.lo || y < a.sinks); };
          const int at = tok0 + k * kQBlock;
          if (!seen(at + r0)) sc[k][0] = sc[k][1] = -INFINITY;
          if (!seen(at + r1)) sc[k][2] = sc[k][3] = -INFINITY;
        }
      }
      // ---- online softmax over the tile's tokens (columns 2t, 2t + 1)
      float al[2], ms[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = fmaxf(sc[0][e], sc[0][e + 2]);
#pragma unroll
        for (int k = 1; k < kQdBlocks; ++k) y = fmaxf(y, fmaxf(sc[k][e], sc[k][e + 2]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
        const float n = fmaxf(m[e], y);
        ms[e] = n == -INFINITY ? 0.f : n;
        al[e] = fast_exp2(m[e] - ms[e]);
        m[e] = n;
        l[e] *= al[e];
      }
      // ---- scales of V
      uint32_t sv[kQdBlocks][2][G];
      uint32_t most[G];
#pragma unroll
      for (int gg = 0; gg < G; ++gg) most[gg] = 0;
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k)
#pragma unroll
        for (int gg = 0; gg < G; ++gg)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t y = lds32(tb + k * BB + qparam_off(D, 1, gg, 0) + (e ? r1 : r0) * 4 * G);
            // nothing of a token that is not seen (its weight is 0, its scale may be anything), zeros of a bad page
            if (bad >> k & 1u) y = 0u;
            if (edge) {
              const int at = tok0 + k * kQBlock + (e ? r1 : r0);
              if (!(at < s.len && (at >= s.lo || at < a.sinks))) y = 0u;
            }
            sv[k][e][gg] = y;
            most[gg] = max(most[gg], y & 0x7fffu);
          }
      float inv[G];
      bool grown = al[0] != 1.f || al[1] != 1.f;
      float fo[G][2];
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, most[gg]);
        const int ex = (int)(__float_as_uint(half_lo(top)) >> 23) + 1;  // scales < 2^(ex - 127)
        float f = 1.f;
        if (ex > E[gg]) {
          f = E[gg] == 0 ? 0.f : __uint_as_float((uint32_t)max(127 + E[gg] - ex, 0) << 23);
          E[gg] = ex;
          grown = true;
        }
        inv[gg] = __uint_as_float((uint32_t)(254 - E[gg]) << 23);  // 2^(127 - E)
        fo[gg][0] = al[0] * f;
        fo[gg][1] = al[1] * f;
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          ob[gg][0] *= al[0];
          ob[gg][1] *= al[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[gg][i][0] *= fo[gg][0];
            o[gg][i][1] *= fo[gg][1];
            o[gg][i][2] *= fo[gg][0];
            o[gg][i][3] *= fo[gg][1];
          }
        }
      }
      // ---- weights and the product with V's codes
#pragma unroll
      for (int k = 0; k < kQdBlocks; ++k) {
        const uint32_t vb = tb + k * BB;
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (the shift behind the difference: in front of it a large maximum would round it away)
          pr[e] = fast_exp2((sc[k][e] - ms[e & 1]) + kQdShift);
          l[e & 1] += pr[e];
        }
#pragma unroll
        for (int gg = 0; gg < G; ++gg) {
          const float s0 = half_lo(sv[k][0][gg]) * inv[gg], s1 = half_lo(sv[k][1][gg]) * inv[gg];
          const float b0 = half_hi(sv[k][0][gg]), b1 = half_hi(sv[k][1][gg]);
          ob[gg][0] += fmaf(pr[0], b0, pr[2] * b1);
          ob[gg][1] += fmaf(pr[1], b0, pr[3] * b1);
          uint32_t h0, h1, e0, e1;
          split_half2(pr[0] * s0, pr[1] * s0, h0, e0);
          split_half2(pr[2] * s1, pr[3] * s1, h1, e1);
          const uint32_t bh0 = movtrans(h0), bh1 = movtrans(h1), bl0 = movtrans(e0), bl1 = movtrans(e1);
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
            mma16816(o[gg][i], f[0], f[1], f[2], f[3], bh0, bh1);
            mma16816(o[gg][i], f[0], f[1], f[2], f[3], bl0, bl1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    x += g.j1 - g.j0;

    // ---- merge the warps
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
#pragma unroll
        for (int gg = 0; gg < G; ++gg) ob[gg][e] += __shfl_xor_sync(0xffffffffu, ob[gg][e], off);
      }
    if (lane < 4) {
      *reinterpret_cast<float2*>(stats + warp * 16 + 2 * t) = make_float2(m[0], m[1]);
      *reinterpret_cast<float2*>(stats + warp * 16 + 8 + 2 * t) = make_float2(l[0], l[1]);
    }
    // o[gg][i]: channels 64 gg + 8 gq + i and + 4, stored as [gg][i, i + 4][gq][8 heads]
#pragma unroll
    for (int gg = 0; gg < G; ++gg)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = E[gg] == 0 ? 0.f : __uint_as_float((uint32_t)E[gg] << 23) * (i & 1 ? 0x1p20f : 0x1p24f);
        float* ow = merge + warp * D * 8 + ((gg * 8 + i) * 8 + gq) * 8 + 2 * t;
        *reinterpret_cast<float2*>(ow) = make_float2(fmaf(o[gg][i][0], f, ob[gg][0]), fmaf(o[gg][i][1], f, ob[gg][1]));
        *reinterpret_cast<float2*>(ow + 4 * 64) = make_float2(fmaf(o[gg][i][2], f, ob[gg][0]), fmaf(o[gg][i][3], f, ob[gg][1]));
      }
    named_bar_sync(1, 32 * kQdWarps);
    {
      const int gg = threadIdx.x & 7;
      float M = -INFINITY, L = 0.f, f[kQdWarps];
#pragma unroll
      for (int w = 0; w < kQdWarps; ++w) M = fmaxf(M, stats[w * 16 + gg]);
      const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kQdWarps; ++w) {
        f[w] = fast_exp2(stats[w * 16 + gg] - Ms);
        L += f[w] * stats[w * 16 + 8 + gg];
      }
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const float il = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no weight at all: zeros; a NaN stays one
      float* rec = p.records + (size_t)(2 * c + (g.j0 == 0 ? 1 : 0)) * qrec_floats<D>();
      const size_t head = (size_t)g.b * a.Hq + g.h * a.G + gg;
#pragma unroll
      for (int dd = threadIdx.x >> 3; dd < D; dd += 4 * kQdWarps) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kQdWarps; ++w) v += f[w] * merge[(w * D + dd) * 8 + gg];
        const int ch = (dd & ~63) + 8 * (dd & 7) + (dd >> 3 & 7);
        if (!whole) rec[16 + ch * 8 + gg] = v;
        else if (gg < a.G) static_cast<T*>(p.out)[head * D + ch] = Num<T>::from_float(v * il);
      }
      if (threadIdx.x < 8) {
        if (!whole) {
          rec[gg] = M;
          rec[8 + gg] = L;
        } else if (gg < a.G && p.lse) {
          p.lse[head] = (M - kQdShift + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    named_bar_sync(1, 32 * kQdWarps);
  }
}

// Merge of the units that lie in several runs.  CTA (c, y) looks at the run of decode CTA c: where its last unit
// begins in it and goes on in the next runs, it merges that unit's records (slot 1 of c, slot 0 of the following
// CTAs) for 32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(kQdCombThreads) qpaged_combine_kernel(QdArgs p, int ncta) {
  const PagedArgs& a = p.a;
  extern __shared__ float csm[];
  constexpr int kGroups = kQdCombThreads / (8 * kQdCombCols);  // records taken side by side
  __shared__ float part[kQdCombThreads];
  int* prefix = reinterpret_cast<int*>(csm);
  float* fac = csm + a.B + 1;  // [record][8]
  float* red = fac + 8 * ncta;  // M, L [8] each
  deal_prefix(a.B, prefix, [&](int b) { return qd_span(a, b).n; });
  __syncthreads();
  griddep_wait();
  const int total = prefix[a.B] * a.Hkv, nc = min(ncta, total), c = blockIdx.x;
  if (c >= nc) return;
  const int x0 = deal_bound(total, nc, c), x1 = deal_bound(total, nc, c + 1);
  const DealSeg g = deal_seg(prefix, a.B, a.Hkv, x1 - 1, x1);  // the last tile's unit
  const int begin = x1 - 1 - g.j0;                        // its first tile
  if (begin < x0 || g.j0 + 1 == g.n) return;
  const int nrec = deal_owner(total, nc, begin + g.n - 1) - c + 1;
  auto rec = [&](int i) { return p.records + (size_t)(2 * (c + i) + (i == 0 ? 1 : 0)) * qrec_floats<D>(); };
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
  const int e = threadIdx.x % (8 * kQdCombCols), grp = threadIdx.x / (8 * kQdCombCols), gg = e & 7;
  const int dd = blockIdx.y * kQdCombCols + (e >> 3);
  float v = 0.f;
#pragma unroll 8
  for (int i = grp; i < nrec; i += kGroups) v += fac[i * 8 + gg] * __ldcg(rec(i) + 16 + dd * 8 + gg);
  part[threadIdx.x] = v;
  __syncthreads();
  if (grp == 0 && gg < a.G) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) v += part[i * 8 * kQdCombCols + e];
    const float L = red[8 + gg], inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const size_t head = (size_t)g.b * a.Hq + g.h * a.G + gg;
    static_cast<T*>(p.out)[head * D + dd] = Num<T>::from_float(v * inv);
    if (p.lse && dd == 0) p.lse[head] = (red[gg] - kQdShift + log2f(L)) * 0.6931471805599453f;
  }
}

template <typename T, int D>
cudaError_t launch_qdecode_td(const QdArgs& p, cudaStream_t s) {
  const int ncta = sm_count();
  const size_t smem = QdSmem<D>::kOffPrefix + ((size_t)p.a.B + 1) * 4;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(qpaged_decode_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  qpaged_decode_kernel<T, D><<<ncta, kQdThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(qpaged_combine_kernel<T, D>, dim3(ncta, D / kQdCombCols), kQdCombThreads,
                          ((size_t)p.a.B + 1 + 8 * ncta + 16) * 4, s, p, ncta);
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
