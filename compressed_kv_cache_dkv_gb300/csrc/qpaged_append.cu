// dkv_qpaged_append: new K and V rows into pages in 4 bits; dkv_qpaged_gather: rows of the cache back in 16 bits.
//
// Eight lanes share a group of 64 channels, eight channels (16 bytes in, a 32-bit word of codes out) each.
// The grid u of a group: fp16 numbers are u = 2^(e - 10) apart below 2^(e + 1), e the exponent of 65/64 of the
// group's largest magnitude L.  With lo = round(min / u), n = round(max / u) - lo, step = ceil(n / 15) every
// value (lo + code * step) u lies on that grid, and below 2^(e + 1): lo + 15 step <= L / u + 1/2 + 15 and
// 15.5 u < L / 64.  So the values are fp16 numbers exactly, whatever reads them in which order.  All of it is
// exact in fp32 (integers below 2^12, powers of two), and a code is round((x / u - lo) / step) without error: the
// quotient only proposes k, and x / u is compared with the border lo + (k + 1/2) step, a multiple of 1/2.
//
// Bound by memory: 4 d bytes in and 9/8 d out a row and head (the gather the other way round).
#include "qpaged.cuh"

namespace dkv {
namespace {

constexpr int kQaThreads = 256, kQaVec = 4;
constexpr float kQaMost = 61440.f;  // above it lo + 15 step could leave fp16

__device__ inline float2 unpack2(uint32_t x, __half) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
__device__ inline float2 unpack2(uint32_t x, __nv_bfloat16) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// A lane's eight channels of a group: the word of codes, and the group's (scale, bias) as two halves.
// `odd`: a value was not finite or too large.
template <typename T>
__device__ inline uint32_t quantise(const uint4& in, uint32_t* param, bool* odd) {
  float x[8];
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(w[i], T());
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad |= !(fabsf(x[i]) <= kQaMost);
    x[i] = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -kQaMost), kQaMost);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  *odd = bad;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float top = fmaxf(fabsf(lo), fabsf(hi)) * 1.015625f;
  const int e = max((int)(__float_as_uint(top) >> 23) - 127 - 10, -24);  // u = 2^e
  const float u = __uint_as_float((uint32_t)(127 + e) << 23), inv = __uint_as_float((uint32_t)(127 - e) << 23);
  const float b = rintf(lo * inv);
  const int n = (int)(rintf(hi * inv) - b), step = (n + 14) / 15;
  const float st = (float)step, r = step > 0 ? __frcp_rn(st) : 0.f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] * inv, k = floorf((t - b) * r), border = fmaf(k + 0.5f, st, b);
    int c = (int)k;
    c += t > border || (t == border && (c & 1));
    codes |= (uint32_t)min(max(c, 0), 15) << (4 * i);
  }
  *param = pack_half2(st * u, b * u);
  return step > 0 ? codes : 0u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kQaThreads) qpaged_append_kernel(PagedArgs a, const uint4* __restrict__ K,
                                                                  const uint4* __restrict__ V, dkv_strides ns,
                                                                  int n_rows, const int64_t* __restrict__ slots,
                                                                  uint8_t* __restrict__ cache) {
  constexpr int R = D / 8;  // lanes of a row
  const int64_t total = (int64_t)n_rows * a.Hkv * 2 * R, n_slots = (int64_t)a.n_pages << a.page_shift;
  const int64_t base = (int64_t)blockIdx.x * (kQaThreads * kQaVec) + threadIdx.x;
  const int c = (int)(base % R), lane8 = threadIdx.x & 7, g = c / 8;
  const int kv = (int)(base / R & 1);  // (a step of kQaThreads is an even number of rows)
  uint4 in[kQaVec];
  uint8_t* block[kQaVec];
  int tok[kQaVec];
  bool live[kQaVec];
#pragma unroll
  for (int x = 0; x < kQaVec; ++x) {
    const int64_t at = (base + x * kQaThreads) / R;  // (row, head, K or V)
    const int h = (int)((at >> 1) % a.Hkv);
    const int64_t row = (at >> 1) / a.Hkv;
    live[x] = base + x * kQaThreads < total;
    const int64_t slot = live[x] ? __ldg(slots + row) : -1;
    if (slot < 0 || slot >= n_slots) {
      if (slot != -1) raise_error(a.err, DKV_DEVERR_INDEX);
      live[x] = false;
    }
    in[x] = make_uint4(0, 0, 0, 0);
    if (!live[x]) continue;
    in[x] = __ldg((kv ? V : K) + (row * ns.token + h * ns.head) / 8 + c);
    const int t = (int)slot & a.page_mask;
    block[x] = cache + (slot >> a.page_shift) * a.stride_page + h * a.stride_head + (t / kQBlock) * qblock_bytes(D);
    tok[x] = t % kQBlock;
  }
#pragma unroll
  for (int x = 0; x < kQaVec; ++x) {
    uint32_t param;
    bool odd;
    const uint32_t codes = quantise<T>(in[x], &param, &odd);
    if (!live[x]) continue;
    if (odd) raise_error(a.err, DKV_DEVERR_RANGE);
    *reinterpret_cast<uint32_t*>(block[x] + qcode_off(D, kv, g, tok[x]) + lane8 * 4) = codes;
    if (lane8 == 0) *reinterpret_cast<uint32_t*>(block[x] + qparam_off(D, kv, g, tok[x])) = param;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQaThreads) qpaged_gather_kernel(PagedArgs a, const uint8_t* __restrict__ cache,
                                                                  const int32_t* __restrict__ first,
                                                                  const int32_t* __restrict__ counts, int n, uint4* K,
                                                                  uint4* V, dkv_strides os) {
  constexpr int R = D / 8;
  const int b = blockIdx.y, hv = (int)(blockIdx.x % (2u * a.Hkv)), h = hv >> 1, kv = hv & 1;
  int cnt = n;
  if (counts) {
    cnt = __ldg(counts + b);
    if (cnt < 0 || cnt > n) {
      if (threadIdx.x == 0) raise_error(a.err, DKV_DEVERR_INDEX);
      cnt = min(max(cnt, 0), n);
    }
  }
  const int64_t p0 = __ldg(first + b);
  uint4* dst = kv ? V : K;
  const int c = threadIdx.x % R;
#pragma unroll
  for (int x = 0; x < kQaVec; ++x) {
    const int i = ((int)(blockIdx.x / (2u * a.Hkv)) * kQaVec + x) * (kQaThreads / R) + threadIdx.x / R;
    if (i >= cnt) return;
    const int64_t t = p0 + i;
    uint32_t w = 0, sb = 0;
    if (t < 0 || t >= a.cap) {
      raise_error(a.err, DKV_DEVERR_INDEX);
    } else {
      const int page = paged_page(a, b, (int)t), tok = (int)t & a.page_mask;
      if (page < a.n_pages) {
        const uint8_t* block = cache + page * a.stride_page + h * a.stride_head + (tok / kQBlock) * qblock_bytes(D);
        w = __ldg(reinterpret_cast<const uint32_t*>(block + qcode_off(D, kv, c / 8, tok % kQBlock) + 4 * (c & 7)));
        sb = __ldg(reinterpret_cast<const uint32_t*>(block + qparam_off(D, kv, c / 8, tok % kQBlock)));
      }
    }
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&sb));
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = Num<T>::pack(fmaf((float)(w >> (8 * e) & 15u), f.x, f.y), fmaf((float)(w >> (8 * e + 4) & 15u), f.x, f.y));
    dst[(b * os.batch + h * os.head + i * os.token) / 8 + c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

cudaError_t launch_qpaged_append(const PagedArgs& a, int d, int dtype, const void* K, const void* V,
                                 const dkv_strides& ns, int n_rows, const int64_t* slots, uint8_t* cache, cudaStream_t s) {
  const int64_t per = kQaThreads * kQaVec, pieces = (int64_t)n_rows * a.Hkv * 2 * (d / 8);
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)((pieces + per - 1) / per), kQaThreads, 0, s>>>(a, static_cast<const uint4*>(K), static_cast<const uint4*>(V),
                                                                       ns, n_rows, slots, cache);
  };
  if (dtype == DKV_BF16) d == 128 ? go(qpaged_append_kernel<__nv_bfloat16, 128>) : go(qpaged_append_kernel<__nv_bfloat16, 64>);
  else d == 128 ? go(qpaged_append_kernel<__half, 128>) : go(qpaged_append_kernel<__half, 64>);
  return cudaGetLastError();
}

cudaError_t launch_qpaged_gather(const PagedArgs& a, int d, int dtype, const uint8_t* cache, const int32_t* first,
                                 const int32_t* counts, int n, void* K, void* V, const dkv_strides& os, cudaStream_t s) {
  const int per = kQaThreads / (d / 8) * kQaVec;
  auto go = [&](auto kernel) {
    kernel<<<dim3((unsigned)((n + per - 1) / per) * (2u * a.Hkv), a.B), kQaThreads, 0, s>>>(a, cache, first, counts, n, static_cast<uint4*>(K),
                                                                          static_cast<uint4*>(V), os);
  };
  if (dtype == DKV_BF16) d == 128 ? go(qpaged_gather_kernel<__nv_bfloat16, 128>) : go(qpaged_gather_kernel<__nv_bfloat16, 64>);
  else d == 128 ? go(qpaged_gather_kernel<__half, 128>) : go(qpaged_gather_kernel<__half, 64>);
  return cudaGetLastError();
}

}  // namespace dkv
