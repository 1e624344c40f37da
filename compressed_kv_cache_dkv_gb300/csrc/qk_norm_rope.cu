// dkv_qk_norm_rope: the norm of each query and key head, their rotation to the token's position, and keys and
// values into 16-bit pages, in one pass over a projection's output.
//
//   y = x / sqrt(mean(x^2) + eps) * gain        over the d channels of a head, in fp32
//   (y_j, y_{j+h}) turned by position * f_j     for j < h, rounded once, at the end
//
// A turn is taken as a 64-bit fraction of the circle: position * turn_j modulo 2^64 is exact however far the position
// is.  turn_j is not: it comes of a double, off by 2^-54 of a circle for a frequency up to 1 (three roundings, of the
// power, of 1 / 2 pi and of their product, of 2^-53 each, and those of the exponent: (3 + ln 1 / f) f / 2 pi of 2^-53), so
// that position 2^31 is off by 2^-23.  The upper 32 bits go to sincospif as fp32: 2^-26 of a circle more.
//
// d / 8 lanes share a row, eight channels (16 bytes) each; the partner channels of the rotation are a fixed number of
// lanes away, and come over as they were loaded.  Gains are folded into the cosines and sines, the norm's factor
// into the last product.  A warp keeps these of its token and walks the heads in rounds of kRotDepth rows for each of
// its row groups, the next round's rows on their way meanwhile.  Bound by memory: 4 d bytes a head, 6 d for a key that
// also goes into a page.
//
// Measured: 16384 tokens of 32 query and 8 KV heads, d 128, bf16, keys and values into pages too (436 MB): 82 us, 5.3
// TB/s, 0.79 of the measured copy rate (146 without the next round on its way, gains and norm as products of their
// own).  16 tokens of 12 and 2 heads: 4.3 us in a graph.
#include "paged_tc.cuh"
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kRotThreads = 256, kRotDepth = 4;

// channels 2 i, 2 i + 1 of a piece
template <typename T>
__device__ inline float2 pair_of(const uint4& v, int i) {
  const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  const T* h = reinterpret_cast<const T*>(&w);
  return make_float2(Num<T>::to_float(h[0]), Num<T>::to_float(h[1]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads) qk_norm_rope_kernel(const __grid_constant__ RotateArgs a, int parts) {
  constexpr int L = D / 8, RPW = 32 / L, kStep = RPW * kRotDepth;  // lanes of a row, rows at once, rows of a round
  const int lane = threadIdx.x & 31, li = lane % L, sub = lane / L;
  const int64_t w = (int64_t)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5);
  const int64_t tok = w / parts;
  if (tok >= a.rows) return;
  const int pos = __ldg(a.positions + tok);
  if (pos < 0) return;  // a row of padding
  // where the token's key and value go
  int64_t page_at = -1;
  if (a.slots) {
    const int64_t slot = __ldg(a.slots + tok);
    if (slot >= 0 && slot < a.n_slots) page_at = (slot >> a.page_shift) * a.stride_page + (slot & a.page_mask) * a.stride_token;
    else if (slot != -1 && lane == 0) raise_error(a.err, DKV_DEVERR_INDEX);
  }
  // rounds of queries, of keys and of values to copy; this warp takes every parts-th
  const int nq = (a.hq + kStep - 1) / kStep, nk = (a.hkv + kStep - 1) / kStep, rounds = nq + nk + (page_at >= 0 ? nk : 0);
  struct Round {
    uint4 v[kRotDepth];
  };
  auto fetch = [&](int r) {
    Round x;
    const int kind = r < nq ? 0 : r < nq + nk ? 1 : 2, heads = kind ? a.hkv : a.hq;
    const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
    const int64_t* st = kind == 0 ? a.qs : kind == 1 ? a.ks : a.vs;
    const int h0 = (r - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kStep + sub;
    const T* at = src + tok * st[0] + h0 * st[1] + 8 * li;
#pragma unroll
    for (int i = 0; i < kRotDepth; ++i) {
      x.v[i] = make_uint4(0, 0, 0, 0);
      if (r < rounds && h0 + i * RPW < heads) x.v[i] = *reinterpret_cast<const uint4*>(at + (int64_t)(i * RPW) * st[1]);
    }
    return x;
  };
  int r = (int)(w % parts);
  Round next = fetch(r);

  const int hl = a.half / 8;  // lanes of the first half
  const bool turns = li < 2 * hl;
  const int other = li < hl ? li + hl : turns ? li - hl : li, partner = lane - li + other;
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (!turns) continue;
    const uint64_t f = (uint64_t)pos * a.turn[(li < hl ? 8 * li : 8 * (li - hl)) + e];
    sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &sn[e], &cs[e]);
    if (li < hl) sn[e] = -sn[e];
  }
  float2 A[4], B[4];  // of a row's channels, and of their partners
  int have = -1;
  for (; r < rounds; r += parts) {
    const Round cur = next;
    next = fetch(r + parts);
    const int kind = r < nq ? 0 : r < nq + nk ? 1 : 2, heads = kind ? a.hkv : a.hq;
    const int h0 = (r - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kStep + sub;
    if (kind == 2) {
#pragma unroll
      for (int i = 0; i < kRotDepth; ++i)
        if (h0 + i * RPW < heads)
          *reinterpret_cast<uint4*>(static_cast<T*>(a.v_pool) + page_at + (h0 + i * RPW) * a.stride_head + 8 * li) = cur.v[i];
      continue;
    }
    if (have != kind) {
      have = kind;
      const uint4* gain = static_cast<const uint4*>(kind ? a.k_gain : a.q_gain);
      uint4 g = make_uint4(0, 0, 0, 0), go = g;
      if (gain) {
        g = __ldg(gain + li);
        go = __ldg(gain + other);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        A[e] = make_float2(cs[2 * e], cs[2 * e + 1]);
        B[e] = make_float2(sn[2 * e], sn[2 * e + 1]);
        if (gain) {
          A[e] = mul2(A[e], pair_of<T>(g, e));
          B[e] = mul2(B[e], pair_of<T>(go, e));
        }
      }
    }
    T* const out = static_cast<T*>(kind ? a.k_out : a.q_out);
    const int64_t* st = kind ? a.kos : a.qos;
    T* const at = out + tok * st[0] + h0 * st[1] + 8 * li;
#pragma unroll
    for (int i = 0; i < kRotDepth; ++i) {
      float2 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = pair_of<T>(cur.v[i], e);
      float inv = 1.f;
      if (a.norm) {
        float2 s2 = mul2(y[0], y[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(y[e], y[e], s2);
        float s = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        inv = rsqrtf(fmaf(s, 1.f / D, a.eps));
      }
      uint4 z = cur.v[i];
      if (a.half) {
        z.x = __shfl_sync(0xffffffffu, z.x, partner);
        z.y = __shfl_sync(0xffffffffu, z.y, partner);
        z.z = __shfl_sync(0xffffffffu, z.z, partner);
        z.w = __shfl_sync(0xffffffffu, z.w, partner);
      }
      if (h0 + i * RPW >= heads) continue;
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 x = mul2(y[e], A[e]);
        if (turns) x = fma2(pair_of<T>(z, e), B[e], x);  // (a channel that does not turn takes nothing of an infinite one)
        x = mul2(x, make_float2(inv, inv));
        o[e] = Num<T>::pack(x.x, x.y);
      }
      const uint4 res = make_uint4(o[0], o[1], o[2], o[3]);
      if (out) *reinterpret_cast<uint4*>(at + (int64_t)(i * RPW) * st[1]) = res;
      if (kind && page_at >= 0)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.k_pool) + page_at + (h0 + i * RPW) * a.stride_head + 8 * li) = res;
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RotateArgs& a, int d, int dtype, cudaStream_t s) {
  // Warps of a token: each makes the token's cosines again, so one where the tokens alone fill the GPU.
  const int step = 32 / (d / 8) * kRotDepth, nk = (a.hkv + step - 1) / step, rounds = (a.hq + step - 1) / step + (a.v ? 2 : 1) * nk;
  const int64_t want = (int64_t)sm_count() * 32;
  int parts = (int)(a.rows >= want ? 1 : (want + a.rows - 1) / a.rows);
  if (parts > rounds) parts = rounds;
  const int64_t warps = (int64_t)a.rows * parts;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)((warps + kRotThreads / 32 - 1) / (kRotThreads / 32)), kRotThreads, 0, s>>>(a, parts);
  };
  if (dtype == DKV_BF16) d == 128 ? go(qk_norm_rope_kernel<__nv_bfloat16, 128>) : go(qk_norm_rope_kernel<__nv_bfloat16, 64>);
  else d == 128 ? go(qk_norm_rope_kernel<__half, 128>) : go(qk_norm_rope_kernel<__half, 64>);
  return cudaGetLastError();
}

}  // namespace dkv
