// dkv_qpaged_prefill: causal attention of the last tokens of each sequence over a cache held in 4 bits, with an
// optional sliding window and sinks, on the tcgen05 tensor cores.  The sequences' queries lie one behind the other.
//
// A CTA owns two groups of 128 query rows that share every K and V tile: two heads of one KV head at the same
// tokens where the group size is even, else 256 tokens of one head; up to 64 queries stand in rows of 8, 16, 32 or
// 64 a head, so that a group holds several heads.  A grid that would leave half of the multiprocessors idle is
// multiplied by cutting the key tiles of each CTA into parts, which a second grid joins by their references and sums.
// Per 64-key tile j and group g
//   S_g = Q_g K_j^T   M = 128 queries, N = 64 keys   (64 TMEM columns, two buffers a group)
//   O_g += P_g V_j    M = 128, N = d, P from TMEM (fp16, over the first 32 columns of its S)
//
// Warps 0-7 hold a query row per thread: they bring Q to shared memory, and turn S into P.  Warp 8 streams the
// tiles' bytes (bulk copies, one per page and tile) into a ring, warps 12-15 make fp16 values of them:
// a group's values scale * code + bias are fp16 numbers exactly, so the tensor cores see the very values of the cache.
// Warps 9 and 10 issue the products.  All operands are fp16; bf16 queries are brought into its range by a power of
// two for each row, which goes into that row's factor of the scores (exact for values above 2^-24 of the largest).
// Codes come out of a word in the order 0 4 1 5 2 6 3 7; Q stands in the same order, and O leaves it at the end.
//
// P = 2^(score - ref) is rounded once to fp16.  A row's reference lies kQpShift below a maximum and moves, with O
// rescaled in tensor memory, only when weights leave fp16's range: when a tile's sum of them exceeds 2^15, which is
// found without a maximum.  So P is at most 2^15, weights down to e^-14 of the largest keep 11 bits and smaller ones
// are off by 2^-32 of it at most.  One fp16 value is a choice: an operand has 16 bits, and a second P V product for what
// the first leaves would be 512 more of a tile's 1312 cycles of products; fp16 outputs are 2.3e-4 from the definition (root
// mean square, the prompt under a window below), a plain form's with fp32 weights 2.1e-4, bf16 ones both 1.7e-3.
//
// Values in the cache are finite.  What lies in slots that no row of the CTA sees may be anything and counts as
// zeros; a weight of 0 takes care of what only some rows see.
//
// Bound: a 128 x 64 tile at d 128 takes 8 x 50 cycles for S (6 KB of shared memory a product) and 4 x 64 for P V, 1312
// for the two groups, and making its values 300 more of shared memory's time.  A tile takes 1800.  The rest is the way
// from one warp to the next (a wait that is ready costs 100 cycles or more) and the instructions' own arrival: what
// the warps run between two tiles does not stay in the innermost instruction cache, so short code counts (edge tiles
// in a function of their own: 548 to 516 us on an 8k causal prompt; K's and V's values in one rolled loop).  Also
// measured there: 576 us with a maximum in the loop and separate barriers for K, V and slots, 468 with one barrier for
// a tile and one commit for both uses of a product's end; a second warpgroup for the values (fewer registers for the
// rows) 523.  A CTA costs 11 us beside its tiles (barriers 1.3, queries 3.6, first tile 2.5, output 2.1, launch).
//
// So in a large grid a CTA that comes to its end takes over the place of one that has not begun (cluster launch
// control): warp 11 asks for it, works out its rows and tiles for all warps, and the next tiles' bytes and values are
// made while the last rows leave.  That leaves 6.6 us from a unit's last tile to the next one's first (product's end
// 0.7, output 2.3, next unit 0.4, queries sent for 1.1, there 0.65, converted 0.8 to 1.4, first scores 0.65): the 8k
// causal prompt 446 us in a graph (465 without), 16k under a window of 1024 141 (147), 8 prompts of 700 to 4096 507
// (537).  A place is taken when the loading warp has sent off the unit's last tile: taken at a unit's start, places
// wait for busy CTAs while others run out (8k causal 465).  The second group's start put off by three tiles, to have
// the groups' ends apart, cost 2 us.  A group that falls idle in the next unit waits for its rows there; a
// wait in every unit cost the windowed prompt 6 us.  Edge tiles without a new maximum in a third function: 498 for the 8 prompts, and 142
// under the window.
//
// Measured (d 128): a prompt of 8191, 32 query and 8 KV heads, pages of 16: 451 us, 1.22 PFLOP/s.  One of 16384
// under a window of 1024, 12 heads: 144 us.  32 queries over 300 to 2000 keys, d 64: 16.4 us in a graph.
#include "paged_tc.cuh"
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kQpThreads = 512, kQpM = 128, kQpN = 64;
constexpr float kQpShift = 7.f;
constexpr float kQpLarge = 0x1p20f;  // scores (in base 2) whose rounding would show in the range
constexpr float kQpMost = 0x1p15f;   // of a weight

template <int D>
struct QpSmem {
  static constexpr int kR = 4;     // slots for K, and for V
  static constexpr int kRaw = 3;   // tiles of bytes on their way
  static constexpr uint32_t kQ = kQpM * D * 2;          // one group's Q
  static constexpr uint32_t kTile = kQpN * D * 2;       // one K or V tile
  static constexpr uint32_t kRawTile = kQpN / kQBlock * qblock_bytes(D);
  static constexpr uint32_t kOffK = 2 * kQ;
  static constexpr uint32_t kOffV = kOffK + kR * kTile;
  static constexpr uint32_t kOffRaw = kOffV + kR * kTile;
  static constexpr uint32_t kOffBar = kOffRaw + kRaw * kRawTile;
  static constexpr uint32_t kBytes = kOffBar + 768;
};

struct QpArgs {
  PagedArgs a;
  PackedQuery q;
  const uint8_t* cache;
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
  float2* part_stat; // [CTA][part][256 rows] reference and sum, when parts > 1
};

// Parts of `tiles` key tiles: as many as take the least time by the model, with kQpJoin us for the join, one
// where that takes no longer.  The grid and its join have to agree, so the roundings are spelled out.
constexpr float kQpJoin = 2.5f;
__device__ inline int qp_parts(const QpArgs& p, int tiles) {
  if (p.parts < 2) return 1;
  const int parts = min(min((int)rintf(__fsqrt_rn(__fmul_rn(p.ratio, (float)tiles))), p.parts), tiles);
  if (parts < 2) return 1;
  const float whole = __fmul_rn(p.tile_us, (float)tiles), cut = __fadd_rn(__fmul_rn(p.tile_us, (float)((tiles + parts - 1) / parts)), __fadd_rn(__fmul_rn(p.part_us, (float)parts), kQpJoin));
  return cut < whole ? parts : 1;
}

// The queries of a sequence: its span, and the row of its first one.
struct QpSpan {
  QuerySpan s;
  int start;
};
__device__ inline QpSpan qp_span(const QpArgs& p, int b) {
  QpSpan r;
  const int s0 = __ldg(p.q.starts + b), s1 = __ldg(p.q.starts + b + 1);
  r.s.len = paged_len(p.a, b);
  r.start = s0;
  r.s.n = s1 - s0;
  if (s0 < 0 || s1 < s0 || s1 > p.q.rows || r.s.n > p.q.max_q) {
    raise_error(p.a.err, DKV_DEVERR_INDEX);
    r.s.n = 0;
  }
  r.s.off = r.s.len - r.s.n;
  return r;
}

// Row `row` of group g of a CTA's 256: its head and token.
struct QpRow {
  int head, token;
  bool live;
};
__device__ inline QpRow qp_row(const QpArgs& p, int kvh, int h0, int row0, int n, int g, int row) {
  QpRow r;
  const int h = h0 + (p.by_heads ? (g * kQpM + row) >> p.rows_shift : 0);  // within the KV head's group
  r.head = kvh * p.a.G + h;
  r.token = row0 + (p.by_heads ? row & (p.rows - 1) : g * kQpM + row);
  r.live = h < p.a.G && r.token < n;
  return r;
}

// natural log-sum-exp of a row's reference and sum (-inf for a row that sees no key)
__device__ inline float qp_lse(float ref, float l) { return (ref + log2f(l)) * 0.6931471805599453f; }

// bit c: the query at position pos sees key k0 + c
__device__ inline unsigned long long qp_sees(const PagedArgs& a, int pos, int k0) {
  const int hi = pos - k0, lo = a.window ? pos - a.window + 1 - k0 : 0, sk = a.sinks - k0;
  auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
  return below(hi + 1) & (~below(lo) | below(sk));
}

// The tiles that are not all seen, and those that move a row's reference: scores once more, the reference, and with it
// O and the sum, moved to kQpShift below the maximum where that is higher, and P from there.  Returns reference and
// sum.  In rolled loops, apart from the plain tiles' code: with this in it that loop does not stay in the
// instruction cache, beside the other warps' (8k causal prompt 548 us, 470 without).  A score is rounded by its
// factor before the reference is taken off, as the maximum was: an fma would leave the rounding of the maximum in
// the exponent, 2^-4 at kQpLarge but hundreds at 2^32.
template <int D>
__device__ __noinline__ float2 other_tile(unsigned long long sees, uint32_t ts, uint32_t to, float slog2, float ref, float l, bool some) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kQpN; c += 32) {
    const uint32_t bits = (uint32_t)(sees >> c);
    uint32_t s[32];
    tc_ld32(ts + c, s);
    tc_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) top = fmaxf(top, bits >> e & 1u ? __uint_as_float(s[e]) : -INFINITY);
  }
  top = __fmul_rn(top, slog2);
  const bool up = top > ref + kQpShift;
  const float al = up ? fast_exp2(ref - (top - kQpShift)) : 1.f;
  if (up) ref = top - kQpShift;
  if (some && __any_sync(0xffffffffu, up)) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      tc_ld32(to + c, o);
      tc_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
      tc_st32(to + c, o);
    }
  }
  const float off = ref == -INFINITY ? 0.f : -ref;
  l *= al;
#pragma unroll 1
  for (int c = 0; c < kQpN; c += 32) {  // (P's columns c / 2 .. c / 2 + 15 lie over scores that have been read)
    const uint32_t bits = (uint32_t)(sees >> c);
    uint32_t s[32], w[16];
    tc_ld32(ts + c, s);
    tc_ld_wait();
    float2 lp = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 x = add2(mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(slog2, slog2)), make_float2(off, off));
      const float2 y = make_float2(bits >> e & 1u ? fast_exp2(x.x) : 0.f, bits >> (e + 1) & 1u ? fast_exp2(x.y) : 0.f);
      lp = add2(lp, y);
      w[e / 2] = pack_half2(y.x, y.y);
    }
    tc_st16(ts + c / 2, w);
    l += lp.x + lp.y;
  }
  return make_float2(ref, l);
}

// an arrival without a branch around it
__device__ inline void mbar_arrive_if(uint64_t* bar, bool x) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)), "r"((uint32_t)x)
               : "memory");
}

template <int N>
__device__ inline void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ inline void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// 128 registers for each of 512 threads at the start, and 2 x 168 + 80 + 96 = 4 x 128.  (Two warpgroups for the values
// leave 144 to the rows, whose loop then takes 1.15 times as long.)
constexpr int kQpRegsRows = 168, kQpRegsIssue = 80, kQpRegsValues = 96;

// What a CTA works at: two groups of rows and the key tiles of a part.
struct QpUnit {
  int b, start, row0, tile, part, parts, hg, kvh, h0;  // h0: first head, within the KV head's group
  QuerySpan qs;
  int tokA, tokB, p_lo;  // tokens of the groups; position of the first
  KeySpan<kQpN> ks;
  int t0, nA, nB, nt;    // the part's first key tile, and tiles of the groups (A's may end a tile or two before B's)
  bool rows, some;       // there are any; there is a unit
  __device__ int key(int j) const { return ks.key(t0 + j); }  // first key of tile j
};
__device__ inline QpUnit qp_unit(const QpArgs& p, int x, int y, int z) {
  const PagedArgs& a = p.a;
  QpUnit u;
  const QpSpan span = qp_span(p, y);
  u.some = true;
  u.b = y;
  u.start = span.start;
  u.qs = span.s;
  // head and first query row of the groups (of all heads the later rows, with more keys, first)
  u.tile = (int)gridDim.z - 1 - z;
  u.row0 = u.tile * (p.by_heads ? p.rows : 2 * kQpM);
  u.part = x % p.parts;
  u.hg = x / p.parts;
  u.kvh = u.hg / p.per_kv;
  u.h0 = u.hg % p.per_kv * p.heads;
  u.rows = u.row0 < u.qs.n;
  u.nA = u.nB = u.nt = u.t0 = u.parts = u.tokA = u.tokB = u.p_lo = 0;
  u.ks = {};
  if (!u.rows) return u;
  u.tokA = min(p.by_heads ? p.rows : kQpM, u.qs.n - u.row0);
  u.tokB = p.by_heads ? u.tokA : max(0, min(kQpM, u.qs.n - u.row0 - kQpM));
  // heads of the second group (0: an empty one)
  const int hdB = p.by_heads ? max(0, min(kQpM / p.rows, a.G - u.h0 - kQpM / p.rows)) : (u.tokB > 0 ? 1 : 0);
  u.p_lo = u.qs.off + u.row0;
  u.ks = key_span<kQpN>(a, u.p_lo, u.p_lo + (p.by_heads ? u.tokA : u.tokA + u.tokB) - 1);
  u.parts = qp_parts(p, u.ks.n);
  u.rows = u.part < u.parts;  // (fewer than a sequence of the table's length would take)
  if (!u.rows) return u;
  u.t0 = (int)((int64_t)u.ks.n * u.part / u.parts);
  const int t1 = (int)((int64_t)u.ks.n * (u.part + 1) / u.parts);
  const int endA = p.by_heads ? u.ks.n : min(u.ks.n, max(0, u.ks.st + (max(0, u.p_lo + u.tokA) + kQpN - 1) / kQpN - u.ks.wt0));
  u.nA = max(0, min(endA, t1) - u.t0);
  u.nB = hdB > 0 ? t1 - u.t0 : 0;
  u.nt = max(u.nA, u.nB);
  return u;
}

// A CTA that has not begun yet is taken off the grid, and its place in the grid written to `to`; or none is left.
__device__ inline void take_cta(void* to, uint64_t* full) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(to)), "r"(smem_u32(full))
               : "memory");
}
__device__ inline bool taken_cta(const void* from, int& x, int& y, int& z) {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred q;\n\tld.shared.b128 h, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 q, h;\n\tselp.u32 %3, 1, 0, q;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@q clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, h;\n\t}"
      : "=&r"(x), "=&r"(y), "=&r"(z), "=&r"(is)
      : "r"(smem_u32(from))
      : "memory");
  return is != 0;
}

// kOn: CTAs take over others' places.
template <typename T, int D, bool kOn>
__global__ void __launch_bounds__(kQpThreads, 1) qpaged_prefill_kernel(QpArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = QpSmem<D>;
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!kOn && p.parts > 1) griddep_launch();  // the join; without it the next grid on the stream may be anyone's

  const uint32_t sb = smem_u32(smem);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);  // [slot]
  uint64_t* o_done = kv_full + S::kR;    // [group][slot] O_j, and so S_j, is done
  uint64_t* raw_full = o_done + 2 * S::kR;  // [stage]
  uint64_t* raw_empty = raw_full + S::kRaw;
  uint64_t* q_full = raw_empty + S::kRaw;  // [group]
  uint64_t* s_full = q_full + 2;         // [group][buffer]
  uint64_t* p_full = s_full + 4;         // [group][buffer]
  uint64_t* drain = p_full + 4;          // [group] after a wait that gave up
  uint64_t* rows_through = drain + 2;    // [group] the rows of a group that falls idle have seen the end of its last product
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rows_through + 2);
  volatile uint32_t* bad_blocks = tmem_slot + 1;  // [stage] blocks on bad pages
  uint64_t* unit_full = reinterpret_cast<uint64_t*>(tmem_slot + 4);  // [2]
  uint64_t* unit_empty = unit_full + 2;                              // [2]
  uint64_t* taken_full = unit_empty + 2;
  uint64_t* unit_sent = taken_full + 1;  // a unit's copies are on their way
  void* taken = taken_full + 2;                                      // 16 bytes
  QpUnit* units = reinterpret_cast<QpUnit*>(taken_full + 4);         // [2]
  static_assert(336 + 2 * sizeof(QpUnit) <= 768, "the units fit");

  bool ok = true;
  const QpUnit first = qp_unit(p, blockIdx.x, blockIdx.y, blockIdx.z);
  // After unit i a warp goes on with the one that warp 11 has found, if any.
  auto next = [&](int i) -> bool {
    ok = __all_sync(0xffffffffu, ok);
    if (!kOn || !ok) return false;
    ++i;
    ok = __all_sync(0xffffffffu, mbar_wait(&unit_full[i & 1], (uint32_t)((i - 1) >> 1) & 1u, a.err));
    return ok && units[i & 1].some;
  };
  // (its place is free again)
  auto left = [&](int i) {
    if (!kOn) return;
    __syncwarp();
    mbar_arrive_if(&unit_empty[i & 1], lane == 0);
  };

  // the rows of a warp of 0-7: their queries
  auto ask = [&](const QpUnit& u) {
    constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes of a row, rows at once
    const int g = warp >> 2, c = lane % kLanes, step = min(p.rows, 32);
    if ((g ? u.nB : u.nA) == 0) return;
    for (int r0 = 32 * (warp & 3); r0 < 32 * (warp & 3) + 32; r0 += step) {  // rows of one head
      const QpRow r = qp_row(p, u.kvh, u.h0, u.row0, u.qs.n, g, r0);
      const int n = r.live ? u.qs.n - r.token : 0;
      const T* from = static_cast<const T*>(p.q.q) + 8 * c;
      if (r.live) from += (int64_t)(u.start + r.token) * p.q.qs.token + (int64_t)r.head * p.q.qs.head;
#pragma unroll 4
      for (int i = lane / kLanes; i < step; i += kAt)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sb + g * S::kQ + sw128(kQpM, r0 + i, c)), 
                     "l"(i < n ? from + i * p.q.qs.token : from), "r"(i < n ? 16 : 0)
                     : "memory");
    }
  };
  // the pages of a unit's tiles from j on, in warp 8: a lane looks after one run of slots of a page (a tile has 64 / rows
  // of them), one look for a batch of tiles
  const int rows = min(a.page_mask + 1, kQpN), runs = kQpN / rows, bpr = rows / kQBlock, batch = 32 / runs;
  uint64_t src = 0;
  uint32_t bytes = 0, dst = 0, sum = 0, none = 0;
  auto look = [&](const QpUnit& u, int j) {
    const int k = j + lane / runs, r = lane % runs, first = u.key(k) + r * rows;
    int b0 = bpr, b1 = 0;  // blocks with a visible token
    for (int i = 0; i < bpr; ++i) {
      const int t = first + i * kQBlock;
      if (k < u.nt && t < u.ks.hi && (t + kQBlock > u.ks.lo || t < a.sinks)) {
        b0 = min(b0, i);
        b1 = i + 1;
      }
    }
    const int page = b0 < b1 ? paged_page(a, u.b, first) : 0;
    const bool bad = page >= a.n_pages;
    bytes = b0 < b1 && !bad ? (uint32_t)(b1 - b0) * qblock_bytes(D) : 0u;
    if (bytes)
      src = reinterpret_cast<uint64_t>(p.cache) + page * a.stride_page + u.kvh * a.stride_head +
            (int64_t)((first & a.page_mask) / kQBlock + b0) * qblock_bytes(D);
    dst = (uint32_t)(r * bpr + b0) * qblock_bytes(D);
    none = __ballot_sync(0xffffffffu, bad);
    sum = bytes;
    for (int o = 1; o < runs; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  };

  // Warps 8-15 set up what all wait on, and look up the first pages; meanwhile the others send for their queries.
  if (warp >= 8) {
    if (threadIdx.x == 9 * 32) {
      for (int i = 0; i < S::kR; ++i) {
        mbar_init(&kv_full[i], 4);  // a lane of each warp that makes values
        mbar_init(&o_done[i], 1);
        mbar_init(&o_done[S::kR + i], 1);
      }
      for (int i = 0; i < S::kRaw; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], 4);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 4);  // a lane of each warp
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 4);
        mbar_init(&drain[i], 1);
        mbar_init(&rows_through[i], 4);
        mbar_init(&unit_full[i], 1);
        mbar_init(&unit_empty[i], 15);  // all warps but the one that fills them
      }
      mbar_init(taken_full, 1);
      mbar_init(unit_sent, 1);
      fence_mbar_init();
    }
    if (warp == 11) tc_alloc<512>(tmem_slot);
    if (kOn && threadIdx.x == 12 * 32) units[0] = first;
    if (warp == 8) look(first, 0);
    tc_fence_before();
    named_bar_sync(1, kQpThreads / 2);
    asm volatile("barrier.cta.arrive 2, %0;" ::"n"(kQpThreads) : "memory");
  } else {
    ask(first);
    named_bar_sync(2, kQpThreads);
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 12) {
    // =========================== values: a thread makes half of a token's channels, of K and then of V
    regs_dec<kQpRegsValues>();
    const int tid = threadIdx.x - 12 * 32, tok = tid & 63, half = tid >> 6;
    constexpr int kWords = D / 16;  // of eight codes
    // bytes of this thread's parameters and codes (of K) in a tile's bytes
    const int g = D == 128 ? half : 0;
    const uint32_t block = sb + S::kOffRaw + (uint32_t)(tok / kQBlock) * qblock_bytes(D);
    const uint32_t param = block + (uint32_t)qparam_off(D, 0, g, tok % kQBlock);
    const uint32_t codes = block + (uint32_t)qcode_off(D, 0, g, tok % kQBlock) + (D == 128 ? 0 : 16 * half);
    const uint32_t row = sb + S::kOffK + sw128(kQpN, tok, half * kWords);  // 16-byte piece c of it is at row ^ 16 c
    int sl = 0, rs = 0, un = 0, before = 0;  // (tiles so far, up to kR)
    uint32_t ph = 0, rph = 0;
    do {
      const QpUnit u = kOn ? units[un & 1] : first;
      left(un);
      const KeySpan<kQpN>& ks = u.ks;
      for (int j = 0; j < u.nt; ++j) {
        if (ok) ok = mbar_wait(&raw_full[rs], rph, a.err);
        const int t = u.key(j) + tok;
        const bool zero = !(t < ks.hi && (t >= ks.lo || t < a.sinks)) || (bad_blocks[rs] >> (tok / kQBlock) & 1u);
        // (rolled: K's and V's code is the same, and short code stays in the instruction cache)
        if (before < S::kR) {
          ++before;
        } else if (ok) {
          ok = mbar_wait(&o_done[sl], ph ^ 1u, a.err);
          if (ok) ok = mbar_wait(&o_done[S::kR + sl], ph ^ 1u, a.err);
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          uint32_t sbits = lds32(param + rs * S::kRawTile + kv * D);
          uint4 c[kWords / 4];
#pragma unroll
          for (int x = 0; x < kWords / 4; ++x) c[x] = lds128(codes + rs * S::kRawTile + kv * 8 * D + 16 * x);
          if (zero) sbits = 0u;
          const __half2 sbh = *reinterpret_cast<__half2*>(&sbits), s2 = __low2half2(sbh), b2 = __high2half2(sbh);
          const uint32_t to = row + kv * (S::kOffV - S::kOffK) + sl * S::kTile;
#pragma unroll
          for (int x = 0; x < kWords / 4; ++x) {
            const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) sts128(to ^ (16 * (4 * x + y)), qvalues8(w[y], s2, b2));
          }
        }
        fence_proxy_async();
        __syncwarp();
        mbar_arrive_if(&kv_full[sl], lane == 0);
        mbar_arrive_if(&raw_empty[rs], lane == 0);
        if (++sl == S::kR) { sl = 0; ph ^= 1u; }
        if (++rs == S::kRaw) { rs = 0; rph ^= 1u; }
      }
    } while (next(un++));
  } else if (warp >= 8) {
    regs_dec<kQpRegsIssue>();
    if (warp == 8) {
      // =========================== the tiles' bytes
      const uint32_t el = elect_one();
      int st = 0, un = 0, sent = 0;  // (sent: stages in use at the end)
      uint32_t ph = 0;
      do {
        const QpUnit u = kOn ? units[un & 1] : first;
        left(un);
        if (un > 0) look(u, 0);
        for (int j = 0, in = 0; j < u.nt; ++j, ++in) {
          if (in == batch) {
            look(u, j);
            in = 0;
          }
          if (sent == S::kRaw) ok = mbar_wait(&raw_empty[st], ph ^ 1u, a.err);
          else ++sent;
          if (!__all_sync(0xffffffffu, ok)) break;
          const uint32_t all = __shfl_sync(0xffffffffu, sum, in * runs);
          if (el) {
            uint32_t m = 0;  // bad runs as a mask of blocks
            if (none)
              for (int i = 0; i < kQpN / kQBlock; ++i) m |= (none >> (in * runs + i / bpr) & 1u) << i;
            bad_blocks[st] = m;
            mbar_arrive_expect_tx(&raw_full[st], all);
          }
          __syncwarp();
          if (lane / runs == in && bytes)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             sb + S::kOffRaw + st * S::kRawTile + dst),
                         "l"(src), "r"(bytes), "r"(smem_u32(&raw_full[st]))
                         : "memory");
          if (++st == S::kRaw) { st = 0; ph ^= 1u; }
        }
        if (kOn) mbar_arrive_if(unit_sent, el);
      } while (next(un++));
      // every copy has landed before the CTA may end (also after a wait that gave up): the last one of each stage
      for (int i = 0; i < sent; ++i) {
        if (--st < 0) { st = S::kRaw - 1; ph ^= 1u; }
        mbar_wait(&raw_full[st], ph, a.err);
      }
    } else if (warp < 11) {
      // =========================== products of group g
      // The whole warp walks through here and one elected lane issues: in code that one lane runs alone the
      // operands are not known to be uniform, and an issue took 75 to 150 cycles.
      constexpr uint32_t id_s = tc_idesc(Num<__half>::kUmma, false, kQpN), id_o = tc_idesc(Num<__half>::kUmma, true, D);
      const uint32_t el = elect_one();
      const int g = warp - 9;
      const uint32_t tg = tmem + 256u * g;
      const uint64_t qd = tc_desc(sb + g * S::kQ, 16, 1024);
      uint64_t* const sf = s_full + 2 * g;
      uint64_t* const pf = p_full + 2 * g;
      uint64_t* const od = o_done + S::kR * g;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = mbar_wait(bar, parity, a.err);
        __syncwarp();
      };
      uint32_t it = 0, c = 0, qph = 0, tph = 0;  // tiles so far, and those of this group: slots go by the first, buffers by the second
      int un = 0;
      bool busy = false;  // the group's last unit with tiles had rows
      do {
        const QpUnit u = kOn ? units[un & 1] : first;
        left(un);
        const int n = g ? u.nB : u.nA;
        auto scores = [&](int j) {
          const uint32_t buf = (c + j) & 1, sl = (it + j) % S::kR;
          wait(&kv_full[sl], ((it + j) / S::kR) & 1u);
          if (j >= 2) wait(&od[(it + j - 2) % S::kR], ((it + j - 2) / S::kR) & 1u);  // the buffer holds P_{j-2}
          tc_fence_after();
          const uint64_t kd = tc_desc(sb + S::kOffK + sl * S::kTile, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)  // 16 channels: 32 bytes of a 128-byte row, then the next 64 channels
            tc_mma(tg + kQpN * buf, qd + (uint64_t)(((k >> 2) * kQpM * 128 + (k & 3) * 32) >> 4),
                   kd + (uint64_t)(((k >> 2) * kQpN * 128 + (k & 3) * 32) >> 4), id_s, k > 0, el);
          tc_commit(&sf[buf], el);
        };
        // In a unit where the group is empty nothing holds this warp, and its arrivals would take the barrier that the rows
        // wait on for the last product, four tiles earlier, through another phase: not before all of them have seen that one.
        if (kOn && n == 0 && u.nt > 0 && busy) {
          wait(&rows_through[g], tph);
          tph ^= 1u;
          busy = false;
        }
        if (n > 0) {
          busy = true;
          wait(&q_full[g], qph);  // (the rows have read the last unit's O by then)
          qph ^= 1u;
          scores(0);
          for (int j = 0; j < n; ++j) {
            if (j + 1 < n) scores(j + 1);
            const uint32_t buf = (c + j) & 1, sl = (it + j) % S::kR;
            wait(&pf[buf], ((c + j) >> 1) & 1u);
            tc_fence_after();
            const uint64_t vd = tc_desc(sb + S::kOffV + sl * S::kTile, kQpN * 128, 1024);
            const uint32_t ts = tg + kQpN * buf;
#pragma unroll
            for (int k = 0; k < kQpN / 16; ++k)  // 16 keys: 16 rows of 128 bytes
              tc_mma_ta(tg + 128u, ts + 8u * k, vd + (uint64_t)(k * 16 * 128 >> 4), id_o, k > 0 ? 1u : (j > 0 ? 1u : 0u), el);
            tc_commit(&od[sl], el);
          }
        }
        for (int j = n; j < u.nt; ++j) {  // the other group's alone: this one is done with the slot
          const uint32_t sl = (it + j) % S::kR;
          wait(&kv_full[sl], ((it + j) / S::kR) & 1u);
          mbar_arrive_if(&od[sl], lane == 0);
        }
        it += u.nt;
        c += n;
      } while (next(un++));
      if (!__all_sync(0xffffffffu, ok)) {  // a wait gave up, and the rows may have too: no product outlives the CTA
        tc_commit(&drain[g], el);
        mbar_wait(&drain[g], 0, a.err);
      }
    } else if (kOn) {
      // =========================== the units: places of CTAs that have not begun, taken off the grid
      const uint32_t el = elect_one();
      for (int i = 1;; ++i) {
        if (i >= 2) ok = mbar_wait(&unit_empty[i & 1], (uint32_t)((i - 2) >> 1) & 1u, a.err);
        // (not before this CTA comes to its end: who takes early leaves others idle)
        // This wait is as long as a unit (1e6 tokens 15 ms): 20 s at most.  The loading warp arrives if its waits give up, too.
        if (ok) ok = mbar_wait(unit_sent, (uint32_t)(i - 1) & 1u, a.err, 16 * kWaitLimit);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (el) {
          mbar_arrive_expect_tx(taken_full, 16);
          take_cta(taken, taken_full);
        }
        __syncwarp();
        int x, y, z;
        ok = mbar_wait(taken_full, (uint32_t)(i - 1) & 1u, a.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        const bool some = taken_cta(taken, x, y, z);
        fence_proxy_async();
        QpUnit u = {};
        if (some) u = qp_unit(p, x, y, z);
        if (lane == 0) units[i & 1] = u;
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_full[i & 1]);
        if (!some) break;
      }
    }
  } else {
    // =========================== one query row per thread
    regs_inc<kQpRegsRows>();
    const int g = warp >> 2, rw = warp & 3, row = 32 * rw + lane;
    uint32_t it = 0, cc = 0;  // tiles so far, and those of this group
    int un = 0;
    bool busy = false;  // as the products'
    do {
      const QpUnit u = kOn ? units[un & 1] : first;
      left(un);
      if (!u.rows) continue;
      if (un > 0) ask(u);
      const QuerySpan& qs = u.qs;
      const KeySpan<kQpN>& ks = u.ks;
      const int n = g ? u.nB : u.nA, parts = u.parts, p_lo = u.p_lo, t0 = u.t0;
      if (kOn) {  // (the warp is together here: all of it has seen the last unit's end)
        mbar_arrive_if(&rows_through[g], lane == 0 && n == 0 && u.nt > 0 && busy);
        busy = n > 0 || (busy && u.nt == 0);
      }
      const QpRow me = qp_row(p, u.kvh, u.h0, u.row0, qs.n, g, row);
      const int pos = qs.off + me.token;
      float slog2 = a.scale_log2;
      if (n > 0) {
        // Each thread brings its row of Q into the order of the codes, and into fp16's range.  (Not unrolled further:
        // straight code that runs once for a CTA waits for its instructions.)
        constexpr int L = D / 8;
        const uint32_t to = sb + g * S::kQ;
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        float up = 1.f;
        if (Num<T>::kUmma == 1) {
          uint32_t top = 0;  // the row's largest magnitudes, by their bits
#pragma unroll 4
          for (int c = 0; c < L; ++c) {
            const uint4 v = lds128(to + sw128(kQpM, row, c));
            top = __vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
            top = __vmaxu2(__vmaxu2(top, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
          }
          const int ex = max((int)(max(top & 0xffffu, top >> 16) >> 7), 15);  // all < 2^(ex - 126)
          up = __uint_as_float((uint32_t)(268 - ex) << 23);                    // 2^(141 - ex): below 2^15 then
          slog2 *= __uint_as_float((uint32_t)(ex - 14) << 23);                 // 2^(ex - 141)
        }
#pragma unroll 4
        for (int c = 0; c < L; ++c) {
          const uint32_t at = to + sw128(kQpM, row, c);
          const uint4 v = lds128(at);
          uint32_t w[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
          if (Num<T>::kUmma == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = mul2(make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)), make_float2(up, up));
              w[e] = pack_half2(f.x, f.y);
            }
          sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[g]);
      }
      // tiles [plain, edges) are seen whole by all of the group's rows
      const int g_lo = p.by_heads ? p_lo : p_lo + g * kQpM, g_hi = g_lo + (g ? u.tokB : u.tokA) - 1;
      const int first_tile = ks.wt0 - ks.st + t0;  // of the window's tiles, tile j holds keys from 64 (first_tile + j) on
      const int plain = max(a.window ? ((max(0, g_hi - a.window + 1) + kQpN - 1) / kQpN) - first_tile : -first_tile, ks.st - t0);
      const int edges = ((g_lo + 1) >> 6) - first_tile;
      static_assert(kQpN == 64, "a shift by 6");
      const uint32_t tg = tmem + ((uint32_t)(32 * rw) << 16) + 256u * g, to = tg + 128u;
      float ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const uint32_t buf = (cc + j) & 1, ts = tg + kQpN * buf;
        if (ok) ok = mbar_wait(&s_full[2 * g + buf], ((cc + j) >> 1) & 1u, a.err);
        tc_fence_after();
        bool other = j < plain || j >= edges;
        if (!other) {
          uint32_t s[kQpN];
#pragma unroll
          for (int c = 0; c < kQpN / 32; ++c) tc_ld32(ts + 32 * c, s + 32 * c);
          tc_ld_wait();
          const float2 scale2 = make_float2(slog2, slog2), minus2 = make_float2(-ref, -ref);
          float2 lp[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t w[kQpN / 2];
#pragma unroll
          for (int e = 0; e < kQpN / 2; ++e) {
            const float2 x = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, minus2);
            const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            lp[e & 1] = add2(lp[e & 1], y);
            w[e] = pack_half2(y.x, y.y);
          }
          const float sum = (lp[0].x + lp[1].x) + (lp[0].y + lp[1].y);
          // no weight is above 2^15 where their sum is not (without a reference x, and so the sum, is infinite or NaN)
          other = __any_sync(0xffffffffu, !(sum <= kQpMost) || !(fabsf(ref) < kQpLarge));
          if (!other) {
            tc_st32(ts, w);
            l += sum;
          }
        }
        if (other) {
          if (j > 0 && ok) ok = mbar_wait(&o_done[S::kR * g + (it + j - 1) % S::kR], ((it + j - 1) / S::kR) & 1u, a.err);
          tc_fence_after();
          const float2 rl = other_tile<D>(qp_sees(a, pos, u.key(j)), ts, to, slog2, ref, l, j > 0);
          ref = rl.x;
          l = rl.y;
        }
        tc_st_wait();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&p_full[2 * g + buf], lane == 0);
      }
      if (n > 0 && ok) ok = mbar_wait(&o_done[S::kR * g + (it + n - 1) % S::kR], ((it + n - 1) / S::kR) & 1u, a.err);
      tc_fence_after();
      const bool live = u.rows && me.live;
      const float il = n == 0 || l == 0.f ? 0.f : 1.f / l;  // a row that sees no key: zeros
      // The rows go through the group's Q, which no product reads any more, so that a warp then writes
      // whole rows of the output.
      const uint32_t stage = sb + g * S::kQ;
      const int64_t rec = (((int64_t)u.b * gridDim.z + u.tile) * (gridDim.x / p.parts) + u.hg) * p.parts + u.part;
#pragma unroll 2  // (short code, as above: all four at once, with the next load on its way, 150 us under the window)
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tc_ld32(to + 32 * c, o);
          tc_ld_wait();
        }
        float f[32];  // channels in their own order
#pragma unroll
        for (int e = 0; e < 32; ++e) f[(e & ~7) + (e & 7) / 2 + 4 * (e & 1)] = n > 0 && l != 0.f ? __uint_as_float(o[e]) * il : 0.f;
        if (parts > 1) {
          if (live) {
            float* o32 = p.part_o + (rec * 2 * kQpM + g * kQpM + row) * D + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(o32 + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          }
          continue;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          sts128(stage + sw128(kQpM, row, (32 * c + e) / 8),
                 make_uint4(Num<T>::pack(f[e], f[e + 1]), Num<T>::pack(f[e + 2], f[e + 3]), Num<T>::pack(f[e + 4], f[e + 5]),
                            Num<T>::pack(f[e + 6], f[e + 7])));
      }
      if (parts > 1) {
        if (live) p.part_stat[rec * 2 * kQpM + g * kQpM + row] = make_float2(ref, l);
      } else if (u.rows) {
        __syncwarp();
        const int ch = lane % (D / 8);  // a row's piece; D / 8 lanes a row
        T* out = static_cast<T*>(p.out) + 8 * ch;
        auto store = [&](const QpRow& first, int r0, int n_rows) {  // rows r0 .. r0 + n_rows - 1, of one head
          if (!first.live) return;
          T* at = out + (int64_t)first.head * p.os.head + (int64_t)(u.start + first.token) * p.os.token;
          const int live_rows = min(n_rows, qs.n - first.token);
#pragma unroll 4
          for (int r = lane / (D / 8); r < live_rows; r += 256 / D)
            *reinterpret_cast<uint4*>(at + (int64_t)r * p.os.token) = lds128(stage + sw128(kQpM, r0 + r, ch));
        };
        const int step = min(p.rows, 32);
        for (int r = 32 * rw; r < 32 * rw + 32; r += step) store(qp_row(p, u.kvh, u.h0, u.row0, qs.n, g, r), r, step);
        if (live && p.lse) p.lse[(int64_t)me.head * p.q.rows + u.start + me.token] = qp_lse(ref, l);
      }
      it += u.nt;
      cc += n;
    } while (next(un++));  // (the rows of the output are read by then)
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 11) tc_free<512>(tmem);
}

// The parts of a row joined: weights l_part 2^(ref_part - M), in part order.  A warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) qpaged_prefill_join_kernel(QpArgs p, int tiles, int hgs) {
  constexpr int V = D / 32;  // channels of a lane
  const PagedArgs& a = p.a;
  griddep_wait();
  const int b = blockIdx.z, tile = (int)blockIdx.y / hgs, hg = (int)blockIdx.y % hgs, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const QpSpan span = qp_span(p, b);
  const QuerySpan& qs = span.s;
  const int row0 = tile * (p.by_heads ? p.rows : 2 * kQpM), p_lo = qs.off + row0;
  const QpRow me = qp_row(p, hg / p.per_kv, hg % p.per_kv * p.heads, row0, qs.n, row / kQpM, row % kQpM);
  if (!me.live) return;
  const int parts = qp_parts(p, key_span<kQpN>(a, p_lo, p_lo + min(p.by_heads ? p.rows : 2 * kQpM, qs.n - row0) - 1).n);
  if (parts < 2) return;  // written by its one part
  const int64_t rec = (((int64_t)b * tiles + tile) * hgs + hg) * p.parts;
  auto at = [&](int i) { return (rec + i) * 2 * kQpM + row; };
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
  T* out = static_cast<T*>(p.out) + (int64_t)me.head * p.os.head + (int64_t)(span.start + me.token) * p.os.token + V * lane;
#pragma unroll
  for (int e = 0; e < V; e += 2) *reinterpret_cast<uint32_t*>(out + e) = Num<T>::pack(f[e] * il, f[e + 1] * il);
  if (p.lse && lane == 0) p.lse[(int64_t)me.head * p.q.rows + span.start + me.token] = qp_lse(M, L);
}

template <typename T, int D, bool kOn>
cudaError_t launch_qprefill_kernel(const QpArgs& p, dim3 grid, cudaStream_t s) {
  constexpr uint32_t smem = QpSmem<D>::kBytes;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(qpaged_prefill_kernel<T, D, kOn>), smem);
  if (e != cudaSuccess) return e;
  qpaged_prefill_kernel<T, D, kOn><<<grid, kQpThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_qprefill_td(const QpArgs& p, cudaStream_t s) {
  const int tiles = (p.q.max_q + (p.by_heads ? p.rows : 2 * kQpM) - 1) / (p.by_heads ? p.rows : 2 * kQpM);
  const int hgs = p.a.Hkv * p.per_kv;
  const dim3 grid(hgs * p.parts, p.a.B, tiles);
  // Taking places over pays from about two CTAs a multiprocessor on: 160 CTAs of up to 80 tiles (d 64) 68.5 us with it
  // and 67.4 without, 512 of 48 tiles 122.4 and 123.2, 768 of 19 tiles 139 and 147.
  const bool on = (int64_t)grid.x * grid.y * grid.z > 2 * sm_count();
  const cudaError_t e = on ? launch_qprefill_kernel<T, D, true>(p, grid, s) : launch_qprefill_kernel<T, D, false>(p, grid, s);
  if (e != cudaSuccess || p.parts == 1) return e;
  return launch_dependent(qpaged_prefill_join_kernel<T, D>, dim3(2 * kQpM / 8, tiles * hgs, p.a.B), 256, 0, s, p, tiles, hgs);
}

}  // namespace

size_t qpaged_prefill_ws_bytes(int d) { return kWsHeader + (size_t)sm_count() * 2 * kQpM * (d + 2) * 4; }

cudaError_t launch_qpaged_prefill(const PagedArgs& a, int d, int dtype, const PackedQuery& q, const uint8_t* cache,
                                  void* out, const dkv_strides& os, float* lse, uint8_t* ws, cudaStream_t s) {
  QpArgs p;
  p.a = a;
  p.q = q;
  p.cache = cache;
  p.out = out;
  p.os = os;
  p.lse = lse;
  // Rows of a head in a group.  Up to 64 queries: a power of two, so that a group holds several heads.
  p.rows = 8;
  while (p.rows < q.max_q && p.rows < kQpM) p.rows *= 2;
  p.rows_shift = 0;
  while ((1 << p.rows_shift) < p.rows) ++p.rows_shift;
  p.by_heads = a.G % 2 == 0 || p.rows < kQpM;
  p.heads = p.by_heads ? 2 * kQpM / p.rows : 1;
  p.per_kv = (a.G + p.heads - 1) / p.heads;
  // Parts of the key tiles, when the grid would fill at most half of the multiprocessors (records for one grid of
  // them are what the workspace holds).
  const int tokens = p.by_heads ? p.rows : 2 * kQpM;
  const int64_t ctas = (int64_t)a.Hkv * p.per_kv * a.B * ((q.max_q + tokens - 1) / tokens);
  const int64_t keys = a.window > 0 && (int64_t)a.window + a.sinks + tokens < a.cap ? (int64_t)a.window + a.sinks + tokens : a.cap;
  const int64_t fit = sm_count() / ctas;
  p.tile_us = 0.85f;
  p.part_us = 0.65f + 2e-6f * (float)d * (float)a.B * (float)a.Hq * (float)q.max_q;
  p.ratio = p.tile_us / p.part_us;
  p.parts = 1;
  if (fit > 1) {
    const float tiles = (float)((keys + kQpN - 1) / kQpN);
    float parts = rintf(sqrtf(p.ratio * tiles));
    parts = fminf(fmaxf(parts, 1.f), fminf((float)fit, tiles));
    if (p.tile_us * ceilf(tiles / parts) + kQpJoin + p.part_us * parts < p.tile_us * tiles) p.parts = (int)parts;
  }
  p.part_o = reinterpret_cast<float*>(ws + kWsHeader);
  p.part_stat = reinterpret_cast<float2*>(p.part_o + (size_t)sm_count() * 2 * kQpM * d);
  if (dtype == DKV_BF16) return d == 128 ? launch_qprefill_td<__nv_bfloat16, 128>(p, s) : launch_qprefill_td<__nv_bfloat16, 64>(p, s);
  return d == 128 ? launch_qprefill_td<__half, 128>(p, s) : launch_qprefill_td<__half, 64>(p, s);
}

}  // namespace dkv
