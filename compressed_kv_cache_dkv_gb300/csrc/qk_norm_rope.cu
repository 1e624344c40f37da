// dkv_qk_norm_rope: the norm of each query and key head, their rotation to the token's position, and keys and
// values into 16-bit pages, in one pass over a projection's output.
//
//   y = x / sqrt(mean(x^2) + eps) * gain        over the d channels of a head, in fp32
//   (y_j, y_{j+h}) turned by position * f_j     for j < h, rounded once, at the end
//
// A turn is taken as a 64-bit fraction of the circle: position * turn_j modulo 2^64 is exact however far the
// position is, its upper 32 bits are the angle to 2^-32 of a circle, and sincospif takes it from there.
//
// d / 8 lanes share a row, eight channels (16 bytes) each; the partner channels of the rotation are a fixed
// number of lanes away.  A warp keeps the cosines and sines of its token and walks the heads, kRotDepth
// loads in flight.  Bound by memory: 4 d bytes a head, 6 d for a key that also goes into a page.
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kRotThreads = 256, kRotDepth = 4;

template <typename T>
__device__ inline void load8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T* h = reinterpret_cast<const T*>(&w[i]);
    x[2 * i] = Num<T>::to_float(h[0]);
    x[2 * i + 1] = Num<T>::to_float(h[1]);
  }
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
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);  // queries, keys, values to copy
  // where the token's key and value go
  int64_t page_at = -1;
  if (a.slots) {
    const int64_t slot = __ldg(a.slots + tok);
    if (slot >= 0 && slot < a.n_slots) page_at = (slot >> a.page_shift) * a.stride_page + (slot & a.page_mask) * a.stride_token;
    else if (slot != -1 && lane == 0) raise_error(a.err, DKV_DEVERR_INDEX);
  }
  float cs[8], sn[8];
  const int hl = a.half / 8;  // lanes of the first half
  const bool turns = li < 2 * hl;
  const int partner = lane - li + (li < hl ? li + hl : turns ? li - hl : li);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (!turns) continue;
    const uint64_t f = (uint64_t)pos * a.turn[(8 * li + e) % a.half];
    sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &sn[e], &cs[e]);
    if (li < hl) sn[e] = -sn[e];
  }
  float qg[8], kg[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) qg[e] = kg[e] = 1.f;
  if (a.q_gain) load8<T>(__ldg(static_cast<const uint4*>(a.q_gain) + li), qg);
  if (a.k_gain) load8<T>(__ldg(static_cast<const uint4*>(a.k_gain) + li), kg);

  for (int r0 = (int)(w % parts) * kStep; r0 < heads; r0 += parts * kStep) {
    uint4 in[kRotDepth];
#pragma unroll
    for (int x = 0; x < kRotDepth; ++x) {
      const int r = r0 + x * RPW + sub;
      in[x] = make_uint4(0, 0, 0, 0);
      if (r >= heads) continue;
      const bool isq = r < a.hq, isk = r < a.hq + a.hkv;
      const int h = isq ? r : isk ? r - a.hq : r - a.hq - a.hkv;
      const T* src = static_cast<const T*>(isq ? a.q : isk ? a.k : a.v);
      const int64_t st = isq ? a.qs[0] : isk ? a.ks[0] : a.vs[0], sh = isq ? a.qs[1] : isk ? a.ks[1] : a.vs[1];
      in[x] = *reinterpret_cast<const uint4*>(src + tok * st + h * sh + 8 * li);
    }
#pragma unroll
    for (int x = 0; x < kRotDepth; ++x) {
      const int r = r0 + x * RPW + sub;
      const bool isq = r < a.hq, isk = r < a.hq + a.hkv;
      float y[8];
      load8<T>(in[x], y);
      if (a.norm) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float inv = rsqrtf(s * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= isq ? qg[e] : kg[e];
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = __shfl_sync(0xffffffffu, y[e], partner);
        o[e] = turns ? fmaf(z, sn[e], y[e] * cs[e]) : y[e];
      }
      if (r >= heads) continue;
      const uint4 out = make_uint4(Num<T>::pack(o[0], o[1]), Num<T>::pack(o[2], o[3]), Num<T>::pack(o[4], o[5]), Num<T>::pack(o[6], o[7]));
      if (isq) {
        *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + tok * a.qos[0] + r * a.qos[1] + 8 * li) = out;
      } else {
        const int h = isk ? r - a.hq : r - a.hq - a.hkv;
        if (isk && a.k_out) *reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + tok * a.kos[0] + h * a.kos[1] + 8 * li) = out;
        if (page_at >= 0)
          *reinterpret_cast<uint4*>(static_cast<T*>(isk ? a.k_pool : a.v_pool) + page_at + h * a.stride_head + 8 * li) = isk ? out : in[x];
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RotateArgs& a, int d, int dtype, cudaStream_t s) {
  // Warps of a token: each makes the token's cosines again, so one where the tokens alone fill the GPU.
  const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0), step = 32 / (d / 8) * kRotDepth, rounds = (heads + step - 1) / step;
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
