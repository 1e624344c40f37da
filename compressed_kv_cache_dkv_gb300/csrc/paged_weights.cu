// dkv_paged_weights: softmax weights summed by key, weights[t] += sum over queries of
// 2^(c q.k_t - lse), on the tcgen05 tensor cores.
//
// A CTA owns 128 keys of one (sequence, KV head) and goes through every query row that can see
// them, head by head: S^T = K Q^T puts one key into each TMEM lane, so a thread sums its key's
// weights over the columns in registers and every key has one owner (no atomics, a fixed order).
// Two warpgroups take query tiles in turn, each with its own 128 TMEM columns; warp 8 streams
// the query tiles with TMA through two slots, one lane of warp 9 issues the products.  Two CTAs
// share a multiprocessor.  Bound by the exponentials (one per visible pair: twice the cycles of
// its product at d 128) for whole prompts, by the read of K for a few queries; the query tile is
// cut to 32 or 64 rows when there are no more queries, since a product's time goes with its rows.
#include "paged_tc.cuh"

namespace dkv {
namespace {

constexpr int kWtThreads = 320, kWtM = 128, kWtN = 128;  // keys, query rows of a tile at most

template <int D>
struct WtSmem {
  static constexpr uint32_t kTile = 128 * D * 2;  // K tile, or a slot of query rows
  static constexpr uint32_t kOffQ = kTile;
  static constexpr uint32_t kOffLse = kOffQ + 2 * kTile;  // [warpgroup][128] base-2 lse
  static constexpr uint32_t kOffBar = kOffLse + 2 * kWtN * 4;
  static constexpr uint32_t kBytes = kOffBar + 128;
};

template <typename T, int D>
__global__ void __launch_bounds__(kWtThreads, 2)
    paged_weights_kernel(PagedArgs a, PagedQuery q, const float* __restrict__ lse, float* __restrict__ weights, int qn,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using S = WtSmem<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // of all units the earlier keys, which more queries see, first
  const int u = blockIdx.x, b = u / a.Hkv, h = u % a.Hkv, k0 = blockIdx.y * kWtM;
  const QuerySpan qs = query_span(a, q.q_lens, q.Tq, b);
  // query rows that see a key of the tile
  const int r_lo = max(0, k0 - qs.off);
  int r_hi = qs.n - 1;
  if (a.window > 0 && k0 >= a.sinks) r_hi = (int)min((int64_t)r_hi, (int64_t)k0 + kWtM - 2 + a.window - qs.off);
  if (k0 >= qs.len || r_lo > r_hi) return;
  const int t_lo = r_lo / qn, per = r_hi / qn - t_lo + 1, nq = per * a.G;  // query tiles, those of a head side by side

  const uint32_t sb = smem_u32(smem);
  float* lse2 = reinterpret_cast<float*>(smem + S::kOffLse);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* q_full = k_full + 1;   // [slot]
  uint64_t* q_empty = q_full + 2;  // [slot]
  uint64_t* s_full = q_empty + 2;  // [warpgroup]
  uint64_t* s_empty = s_full + 2;  // [warpgroup]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_empty + 2);
  if (threadIdx.x == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&qmap);
    mbar_init(k_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 128);
    }
    fence_mbar_init();
  }
  if (warp == 0) tc_alloc<256>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 8) {
    // =========================== loads
    const int rows = min(a.page_mask + 1, 64), pk = kWtM / rows, nbox = pk * (D / 64);
    const int pi = lane % pk, hf = lane / pk, first = k0 + pi * rows;
    const int lo = paged_window_lo(a, max(qs.off, 0));
    const bool need = first < qs.len && (first + rows > lo || first < a.sinks);  // else zeros, wherever the table points
    if (lane == 0) mbar_arrive_expect_tx(k_full, S::kTile);
    __syncwarp();
    if (lane < nbox)
      tma_load_4d(sb + hf * kWtM * 128 + pi * rows * 128, &kmap, hf * 64, first & a.page_mask, h,
                  need ? paged_page(a, b, first) : a.n_pages, k_full);
    int i = 0;
    for (; i < nq && ok; ++i) {
      const int sl = i & 1;
      if (i >= 2) ok = mbar_wait(&q_empty[sl], (uint32_t)((i / 2 - 1) & 1), a.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[sl], (uint32_t)qn * D * 2);
        for (int x = 0; x < D / 64; ++x)
          tma_load_4d(sb + S::kOffQ + sl * S::kTile + x * qn * 128, &qmap, x * 64, (t_lo + i % per) * qn, h * a.G + i / per, b,
                      &q_full[sl]);
      }
      __syncwarp();
    }
    // every copy has landed before the CTA may end (also after a wait that gave up)
    mbar_wait(k_full, 0, a.err);
    for (int x = max(0, i - 2); x < i; ++x) mbar_wait(&q_full[x & 1], (uint32_t)((x / 2) & 1), a.err);
  } else if (warp == 9) {
    // =========================== products
    // (the whole warp, one elected lane issuing: see the prefill kernel)
    const uint32_t el = elect_one(), id = tc_idesc(Num<T>::kUmma, false, (uint32_t)qn);
    const uint64_t kd = tc_desc(sb, 16, 1024);
    ok = mbar_wait(k_full, 0, a.err);
    for (int i = 0; i < nq; ++i) {
      const int w = i & 1;
      ok = ok && mbar_wait(&q_full[w], (uint32_t)((i / 2) & 1), a.err);
      if (i >= 2) ok = ok && mbar_wait(&s_empty[w], (uint32_t)((i / 2 - 1) & 1), a.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t qd = tc_desc(sb + S::kOffQ + w * S::kTile, 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc_mma(tmem + 128u * w, kd + (uint64_t)(((k >> 2) * kWtM * 128 + (k & 3) * 32) >> 4),
               qd + (uint64_t)(((k >> 2) * qn * 128 + (k & 3) * 32) >> 4), id, k > 0, el);
      tc_commit(&q_empty[w], el);
      tc_commit(&s_full[w], el);
    }
  } else {
    // =========================== sums: one key per thread and warpgroup
    const int w = warp >> 2, row = threadIdx.x & 127, t = k0 + row;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128u * w;
    float* l2 = lse2 + kWtN * w;
    const float slog2 = a.scale_log2;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = w; i < nq; i += 2) {
      const int r0 = (t_lo + i % per) * qn, head = h * a.G + i / per;
      if (row < qn) {
        const float v = r0 + row < qs.n ? __ldg(lse + ((int64_t)b * a.Hq + head) * q.Tq + r0 + row) : -INFINITY;
        l2[row] = v == -INFINITY ? INFINITY : v * 1.4426950408889634f;
      }
      named_bar_sync(1 + w, 128);
      if (ok) ok = mbar_wait(&s_full[w], (uint32_t)((i / 2) & 1), a.err);
      tc_fence_after();
      // columns [c_lo, c_hi] see this key; the warp's keys bound the columns worth loading
      const int c_lo = t - qs.off - r0;
      const int c_end = min(qn, qs.n - r0);
      const int64_t c_win = a.window > 0 && t >= a.sinks ? (int64_t)t + a.window - 1 - qs.off - r0 : c_end - 1;
      const int c_hi = (int)min((int64_t)c_end - 1, c_win);
      const int w_lo = __reduce_min_sync(0xffffffffu, c_lo), w_hi = __reduce_max_sync(0xffffffffu, c_hi);
      const bool whole = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= c_end - 1);
#pragma unroll
      for (int c = 0; c < kWtN / 32; ++c) {
        if (32 * c + 31 < w_lo || 32 * c > w_hi) continue;
        uint32_t s[32];
        tc_ld32(ts + 32 * c, s);
        tc_ld_wait();
        if (whole && 32 * c + 31 < c_end) {
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[e & 3] += fast_exp2(fmaf(__uint_as_float(s[e]), slog2, -l2[32 * c + e]));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = fast_exp2(fmaf(__uint_as_float(s[e]), slog2, -l2[32 * c + e]));
            acc[e & 3] += 32 * c + e >= c_lo && 32 * c + e <= c_hi ? x : 0.f;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&s_empty[w]);
      named_bar_sync(1 + w, 128);  // l2 is read
    }
    const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    if (w == 1) lse2[kWtN + row] = sum;
    named_bar_sync(3, 256);
    if (w == 0 && t < qs.len) weights[(size_t)u * a.cap + t] += sum + lse2[kWtN + row];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tc_free<256>(tmem);
}

template <typename T, int D>
cudaError_t launch_td(const PagedArgs& a, const CUtensorMap& kmap, const CUtensorMap& qmap, const PagedQuery& q,
                      const float* lse, float* weights, cudaStream_t s) {
  constexpr uint32_t smem = WtSmem<D>::kBytes;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(paged_weights_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.B * a.Hkv, (a.cap + kWtM - 1) / kWtM);
  paged_weights_kernel<T, D><<<grid, kWtThreads, smem, s>>>(a, q, lse, weights, paged_weights_rows(q.Tq), kmap, qmap);
  return cudaGetLastError();
}

}  // namespace

int paged_weights_rows(int Tq) { return Tq <= 32 ? 32 : Tq <= 64 ? 64 : 128; }

cudaError_t launch_paged_weights(const PagedArgs& a, int d, int dtype, const CUtensorMap& kmap, const CUtensorMap& qmap,
                                 const PagedQuery& q, const float* lse, float* weights, cudaStream_t s) {
  if (dtype == DKV_BF16)
    return d == 128 ? launch_td<__nv_bfloat16, 128>(a, kmap, qmap, q, lse, weights, s)
                    : launch_td<__nv_bfloat16, 64>(a, kmap, qmap, q, lse, weights, s);
  return d == 128 ? launch_td<__half, 128>(a, kmap, qmap, q, lse, weights, s)
                  : launch_td<__half, 64>(a, kmap, qmap, q, lse, weights, s);
}

}  // namespace dkv
