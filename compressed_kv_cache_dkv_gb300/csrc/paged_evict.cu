// dkv_paged_evict: keep the heaviest tokens of every (sequence, KV head) and move them
// together.
//
// select: a unit's tokens are split over a cluster of CTAs (kSelCluster where the table has room for
// more than kSelStage, of which one does the work of a shorter sequence; else a CTA alone).  They bring the weights' order-preserving integer images into
// shared memory, find the smallest image that stays by radix selection (three passes of 11, 11
// and 10 bits over histograms that every CTA adds up from all of them through distributed shared
// memory), then write the kept positions, ascending, from one scan that counts certain and equal
// images side by side.  Bound by the latency of its passes.
//
// move: a gather of budget rows of K and V per unit, bound by memory (each kept row read and
// written once).  A CTA moves one chunk of kMoveBytes of K and as much of V, whole rows, all of
// it in flight at once.  Position j is filled from a position >= j, so that a sequence compacted
// in place needs an order only between a chunk's write and the reads of the chunks before it:
// CTAs take their chunks from a counter, unit by unit and upwards, read, raise the chunk's flag,
// wait for the flags of those earlier chunks of the unit whose rows come from where this one
// writes, and write.  A page that is compacted in place may hold tokens of other sequences, which
// move to pages of their own: the sequences that move come first in the counter's order, and
// where a batch has both kinds a sequence in place writes once all rows that move have been read.
// A CTA waits only for CTAs that started before it and that read without waiting, so every wait ends.
//
// Measured (d 128): 32 sequences of 2500 to 8192 tokens, 8 KV heads, cut to 4096 (1.03 GB): 179 us,
// of which 17 the selection; 5.8 TB/s.  30000 tokens to 15000, 8 heads: 43 us; 300 to 256: 8.3 us (graphs).
#include "paged.cuh"

namespace dkv {
namespace {

constexpr int kSelThreads = 1024, kSelBins = 2048;
constexpr int kSelPer = 8;                        // consecutive tokens of a thread in the ordered pass
constexpr int kSelStage = 24 * 1024;              // images a CTA holds in shared memory (two CTAs fit a multiprocessor)
constexpr int kSelCluster = 8;
constexpr int kMoveThreads = 256, kMoveVec = 2;   // 16-byte pieces of K, and as many of V, per thread
constexpr int kMoveBytes = kMoveThreads * kMoveVec * 16;
constexpr int kZeroChunk = 8192;                  // weights zeroed by one CTA
constexpr int kPollLimit = 1 << 22;               // polls of a flag before a wait gives up

// a < b as floats iff image(a) < image(b); -0 is 0, NaN is -infinity
__device__ inline uint32_t weight_image(float w) {
  if (isnan(w)) w = -INFINITY;
  if (w == 0.f) w = 0.f;
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Workspace: [header][order EvictSeq [B]][EvictState][flags [unit][chunk]]
struct EvictSeq {  // in the order in which the sequences are moved
  int32_t b, n;    // sequence, tokens that stay
  int32_t in_place, mixed;  // mixed: the batch has sequences in place and others
};
struct EvictState {
  uint32_t ticket;   // chunks taken
  uint32_t moved;    // of a mixed batch: chunks read of the sequences that are not in place
  uint32_t to_move;  // and how many there are
  uint32_t pad;
};
struct EvictPlan {
  int rows, chunks, zeros;  // rows of a chunk, chunks of a unit's rows, chunks of its weights' tail
  size_t off_state, off_flags, bytes;
};
__host__ __device__ inline EvictPlan evict_plan(int B, int Hkv, int cap, int d, int budget) {
  EvictPlan p;
  p.rows = kMoveBytes / (2 * d);
  p.chunks = (budget + p.rows - 1) / p.rows;
  p.zeros = (cap + kZeroChunk - 1) / kZeroChunk;
  p.off_state = kWsHeader + (size_t)B * sizeof(EvictSeq);
  p.off_flags = p.off_state + sizeof(EvictState);
  p.bytes = p.off_flags + (size_t)B * Hkv * p.chunks * 4;
  return p;
}

__device__ inline int ld_cluster_s32(const void* local, uint32_t rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// What the move kernel starts from, written by one CTA: the sequences that move to other pages, then
// those compacted in place (their first page stays), each kind in the batch's order.
__device__ inline void evict_order(const PagedArgs& a, const PagedEvict& e, const EvictPlan& plan, uint8_t* ws, int* wsum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto stays = [&](int b) { return __ldg(a.table + (size_t)b * a.max_pages) == __ldg(e.new_table + (size_t)b * e.new_max_pages); };
  int moving = 0;
  for (int b0 = 0; b0 < a.B; b0 += kSelThreads) moving += __syncthreads_count(b0 + tid < a.B && !stays(b0 + tid));
  const bool mixed = moving > 0 && moving < a.B;
  EvictSeq* order = reinterpret_cast<EvictSeq*>(ws + kWsHeader);
  int before = 0, to_move = 0;  // sequences that move in front of these; this thread's chunks
  for (int b0 = 0; b0 < a.B; b0 += kSelThreads) {
    const int b = b0 + tid;
    const bool in = b < a.B, move = in && !stays(b);
    const uint32_t bits = __ballot_sync(0xffffffffu, move);
    if (lane == 0) wsum[warp] = __popc(bits);
    __syncthreads();
    const int count = wsum[lane];
    const int at = before + __reduce_add_sync(0xffffffffu, lane < warp ? count : 0) + __popc(bits & ((1u << lane) - 1));
    before += __reduce_add_sync(0xffffffffu, count);
    if (in) {
      const int n = min(paged_len(a, b), e.budget);
      order[move ? at : moving + b - at] = {b, n, !move, mixed};
      if (move) to_move += (n + plan.rows - 1) / plan.rows;
    }
    __syncthreads();
  }
  to_move = __reduce_add_sync(0xffffffffu, to_move);
  if (lane == 0) wsum[warp] = to_move;
  __syncthreads();
  if (warp == 0) {
    to_move = __reduce_add_sync(0xffffffffu, wsum[lane]);
    if (lane == 0) *reinterpret_cast<EvictState*>(ws + plan.off_state) = {0u, 0u, (uint32_t)to_move * a.Hkv, 0u};
  }
}

template <int CL>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(PagedArgs a, PagedEvict e, EvictPlan plan,
                                                                  uint8_t* __restrict__ ws) {
  extern __shared__ __align__(16) uint32_t img[];  // images of this CTA's weights (when they fit)
  __shared__ int hist[kSelBins];
  __shared__ int wsum[32];
  __shared__ int sh_digit, sh_above;
  const int rank = CL > 1 ? (int)cluster_ctarank() : 0;
  const int u = (int)(blockIdx.x / CL) - 1, b = u / a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch();
  if (u < 0) {  // beside the units' CTAs
    if (rank == 0) evict_order(a, e, plan, ws, wsum);
    return;
  }
  const int len = paged_len(a, b), n = min(len, e.budget);
  int32_t* kept = e.kept + (size_t)u * e.budget;
  uint32_t* flags = reinterpret_cast<uint32_t*>(ws + plan.off_flags) + (size_t)u * plan.chunks;
  const int all = CL * kSelThreads, me = rank * kSelThreads + tid;
  for (int i = me; i < plan.chunks; i += all) flags[i] = 0;
  for (int j = n + me; j < e.budget; j += all) kept[j] = -1;
  if (len <= e.budget) {  // the same answer in every CTA of a cluster
    for (int j = me; j < n; j += all) kept[j] = j;
    return;
  }
  const bool alone = CL == 1 || len <= kSelStage;
  if (alone && rank > 0) return;
  auto sync = [&]() {
    if (alone) __syncthreads();
    else cluster_sync();
  };
  // candidates [c0, c1); the tokens around them stay whatever they weigh
  const int c0 = e.first, c1 = len - e.recent;
  // this CTA's tokens
  const int share = alone ? len : (len + CL - 1) / CL, t0 = min(rank * share, len), t1 = min(t0 + share, len);
  const float* w = e.weights + (size_t)u * a.cap;
  const bool staged = share <= kSelStage;
  if (staged) {
    for (int t = t0 + tid; t < t1; t += kSelThreads) img[t - t0] = weight_image(__ldg(w + t));
    __syncthreads();
  }
  auto image = [&](int t) { return staged ? img[t - t0] : weight_image(__ldg(w + t)); };
  int k = e.budget - e.first - e.recent;  // candidates to keep: 0 <= k < c1 - c0
  uint32_t thr = 0xffffffffu, mask = 0;   // the smallest image that stays (none above it when k is 0)
  if (k > 0) {
    thr = 0;
    const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const int bins = 1 << bits[p];
      for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = max(c0, t0) + tid; t < min(c1, t1); t += kSelThreads) {
        const uint32_t x = image(t);
        if ((x & mask) == thr) atomicAdd(&hist[(x >> shift[p]) & (bins - 1)], 1);
      }
      sync();
      // the digit with fewer than k images above it and at least k down to it: thread i takes the
      // i-th group of bins from the top
      const int per = bins / kSelThreads, top = bins - 1 - tid * per;
      int cnt[2] = {0, 0};
      for (int i = 0; i < per; ++i) {
        if (alone) cnt[i] = hist[top - i];
        else {
#pragma unroll
          for (int r = 0; r < CL; ++r) cnt[i] += ld_cluster_s32(&hist[top - i], r);
        }
      }
      const int sum = cnt[0] + cnt[1];
      int scan = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      if (lane == 31) wsum[warp] = scan;
      sync();  // (the histograms are read)
      const int before = lane < warp ? wsum[lane] : 0;
      const int above = scan - sum + __reduce_add_sync(0xffffffffu, before);
      if (above < k && above + sum >= k) {
        const int second = above + cnt[0] < k;
        sh_digit = top - second;
        sh_above = above + (second ? cnt[0] : 0);
      }
      __syncthreads();
      thr |= (uint32_t)sh_digit << shift[p];
      mask |= (uint32_t)(bins - 1) << shift[p];
      k -= sh_above;  // still to find among the images that share thr's high bits
      __syncthreads();
    }
  }
  // every image above thr stays, and the first k that equal it.  Tokens of this thread: bits of the
  // certain ones and of the equal ones among t .. t + kSelPer - 1
  auto look = [&](int t, uint32_t& keep, uint32_t& tie) {
    keep = tie = 0;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      if (t + i >= t1) continue;
      if (t + i < c0 || t + i >= c1) keep |= 1u << i;
      else {
        const uint32_t x = image(t + i);
        keep |= (x > thr ? 1u : 0u) << i;
        tie |= (x == thr ? 1u : 0u) << i;
      }
    }
  };
  int out = 0, ties = 0;  // certain and equal images before this CTA's tokens, then before the chunk
  if (!alone) {
    int mk = 0, mt = 0;
    for (int base = t0; base < t1; base += kSelThreads * kSelPer) {
      uint32_t keep, tie;
      look(base + tid * kSelPer, keep, tie);
      mk += __popc(keep);
      mt += __popc(tie);
    }
    mk = __reduce_add_sync(0xffffffffu, mk);
    mt = __reduce_add_sync(0xffffffffu, mt);
    if (tid < 2) hist[tid] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&hist[0], mk);
      atomicAdd(&hist[1], mt);
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      out += ld_cluster_s32(&hist[0], r);
      ties += ld_cluster_s32(&hist[1], r);
    }
  }
  for (int base = t0; base < t1; base += kSelThreads * kSelPer) {
    const int t = base + tid * kSelPer;
    uint32_t keep, tie;
    look(t, keep, tie);
    // both counts in one scan (a chunk has kSelThreads * kSelPer = 2^13 tokens at most)
    const int v = __popc(keep) | __popc(tie) << 16;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    const int part = wsum[lane];
    const int chunk = __reduce_add_sync(0xffffffffu, part);
    const int before = s - v + __reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
    int nk = out + (before & 0xffff), nt = ties + (before >> 16);
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const bool kp = keep >> i & 1u, te = tie >> i & 1u;
      if (kp || (te && nt < k)) kept[nk + min(nt, k)] = t + i;
      nk += kp;
      nt += te;
    }
    out += chunk & 0xffff;
    ties += chunk >> 16;
    __syncthreads();
  }
  if (!alone) cluster_sync();  // nobody leaves while another reads its counts
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads, 8) evict_move_kernel(PagedArgs a, PagedEvict e, EvictPlan plan,
                                                                 uint4* __restrict__ kp, uint4* __restrict__ vp,
                                                                 uint8_t* __restrict__ ws) {
  constexpr int R = D / 8, kRows = kMoveThreads / R;  // pieces of a row, rows of one access
  __shared__ uint32_t sh_ticket;
  const int tid = threadIdx.x;
  griddep_wait();
  EvictState* state = reinterpret_cast<EvictState*>(ws + plan.off_state);
  if (tid == 0) sh_ticket = atomicAdd(&state->ticket, 1u);
  __syncthreads();
  const int per = plan.chunks + plan.zeros;
  const int ou = (int)(sh_ticket / (uint32_t)per), c = (int)(sh_ticket % (uint32_t)per), h = ou % a.Hkv;
  const int4 seq = __ldg(reinterpret_cast<const int4*>(ws + kWsHeader) + ou / a.Hkv);  // EvictSeq
  const int b = seq.x, n = seq.y, u = b * a.Hkv + h;
  const bool in_place = seq.z != 0, mixed = seq.w != 0;
  const int32_t* kept = e.kept + (size_t)u * e.budget;
  const float* w = e.weights + (size_t)u * a.cap;
  float* nw = e.new_weights + (size_t)u * a.cap;
  uint32_t* flags = reinterpret_cast<uint32_t*>(ws + plan.off_flags) + (size_t)u * plan.chunks;
  auto poll = [&](auto over) {  // false after kPollLimit polls
    for (int x = 0; x < kPollLimit; ++x) {
      if (over()) return true;
      __nanosleep(100);
    }
    raise_error(a.err, DKV_DEVERR_TIMEOUT);
    return false;
  };
  // the chunks of the unit before chunk `to` with a row from position j0 or behind (a run of chunks, since
  // kept is ascending) have read their rows; false when a wait gave up
  auto wait_for = [&](int to, int j0) {
    bool ok = true;
    for (int i = to - 1 - tid; i >= 0 && ok; i -= kMoveThreads) {
      if (__ldg(kept + min((i + 1) * plan.rows, n) - 1) < j0) break;
      ok = poll([&]() {
        uint32_t f;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(f) : "l"(flags + i) : "memory");
        return f != 0;
      });
    }
    return __syncthreads_and(ok);
  };
  if (c >= plan.chunks) {  // zeros behind the kept tokens' weights
    const int z0 = max(n, (c - plan.chunks) * kZeroChunk), z1 = min(a.cap, (c - plan.chunks + 1) * kZeroChunk);
    if (z0 >= z1) return;
    if (nw == w && !wait_for((n + plan.rows - 1) / plan.rows, z0)) return;
    for (int j = z0 + tid; j < z1; j += kMoveThreads) nw[j] = 0.f;
    return;
  }
  const int j0 = c * plan.rows;
  if (c == 0 && h == 0 && tid == 0) e.new_lens[b] = n;
  if (j0 >= n) return;
  uint4 v[2 * kMoveVec];
  int64_t to[kMoveVec];
#pragma unroll
  for (int x = 0; x < kMoveVec; ++x) {
    const int j = j0 + x * kRows + tid / R;
    to[x] = -1;
    if (j >= n) continue;
    const int t = __ldg(kept + j), sp = paged_page(a, b, t);
    const int dp = __ldg(e.new_table + (size_t)b * e.new_max_pages + (j >> a.page_shift));
    if (dp < 0 || dp >= a.n_pages) {
      raise_error(a.err, DKV_DEVERR_INDEX);
      continue;
    }
    if (t == j && sp == dp) continue;  // it lies there already
    v[x] = v[x + kMoveVec] = make_uint4(0, 0, 0, 0);
    if (sp < a.n_pages) {
      const int64_t from = (sp * a.stride_page + h * a.stride_head + (t & a.page_mask) * a.stride_token) / 8 + tid % R;
      v[x] = __ldcg(kp + from);
      v[x + kMoveVec] = __ldcg(vp + from);
    }
    to[x] = (dp * a.stride_page + h * a.stride_head + (j & a.page_mask) * a.stride_token) / 8 + tid % R;
  }
  const int jw = j0 + tid;
  const bool weighs = tid < plan.rows && jw < n;
  float wt = 0.f;
  if (weighs) wt = __ldcg(w + __ldg(kept + jw));
  if (in_place || nw == w || mixed) {
    __threadfence();  // this thread's reads are done
    __syncthreads();
    if (tid == 0) {
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(flags + c), "r"(1u) : "memory");
      if (mixed && !in_place) atomicAdd(&state->moved, 1u);
    }
    if ((in_place || nw == w) && !wait_for(c, j0)) return;
    if (in_place && mixed) {  // other sequences' rows may lie where this one writes
      bool ok = true;
      if (tid == 0) ok = poll([&]() {
        uint32_t moved;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(moved) : "l"(&state->moved) : "memory");
        return moved >= state->to_move;
      });
      if (!__syncthreads_and(ok)) return;
    }
  }
#pragma unroll
  for (int x = 0; x < kMoveVec; ++x)
    if (to[x] >= 0) {
      kp[to[x]] = v[x];
      vp[to[x]] = v[x + kMoveVec];
    }
  if (weighs) nw[jw] = wt;
}

}  // namespace

size_t paged_evict_ws_bytes(const PagedArgs& a, int d) { return evict_plan(a.B, a.Hkv, a.cap, d, a.cap).bytes; }

cudaError_t launch_paged_evict(const PagedArgs& a, int d, const PagedEvict& e, void* k_pool, void* v_pool, uint8_t* ws,
                               cudaStream_t s) {
  const int units = a.B * a.Hkv;
  const EvictPlan plan = evict_plan(a.B, a.Hkv, a.cap, d, e.budget);
  const size_t smem = (size_t)(a.cap < kSelStage ? a.cap : kSelStage) * 4;
  const bool wide = a.cap > kSelStage;
  const auto select = wide ? evict_select_kernel<kSelCluster> : evict_select_kernel<1>;
  cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(select), smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((units + 1) * (wide ? kSelCluster : 1));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSelCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = wide ? 1 : 0;
  if ((err = cudaLaunchKernelEx(&cfg, select, a, e, plan, ws)) != cudaSuccess) return err;
  return launch_dependent(d == 128 ? evict_move_kernel<128> : evict_move_kernel<64>,
                          dim3((unsigned)units * (plan.chunks + plan.zeros)), kMoveThreads, 0, s, a, e, plan,
                          static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), ws);
}

}  // namespace dkv
