// dkv_qpaged_append: new K and V rows into pages in 4 bits; dkv_qpaged_gather: rows of the cache back in 16 bits.
//
// Four lanes share a group of 64 channels, sixteen channels (32 bytes in, two 32-bit words of codes out) each.
// The grid u of a group: fp16 numbers are u = 2^(e - 10) apart below 2^(e + 1), e the exponent of 65/64 of the
// group's largest magnitude L.  With lo = round(min / u), n = round(max / u) - lo, step = ceil(n / 15) every
// value (lo + code * step) u lies on that grid, and below 2^(e + 1): lo + 15 step <= L / u + 1/2 + 15 and
// 15.5 u < L / 64.  So the values are fp16 numbers exactly, whatever reads them in which order.  All of it is
// exact in fp32 (integers below 2^12, powers of two), and a code is round((x / u - lo) / step) without error: the
// quotient only proposes k, and x / u is compared with the border lo + (k + 1/2) step, a multiple of 1/2.
//
// Bound by instructions, 122 for 256 values (append: 0.66 of the issue slots), at 0.6 of the memory's rate: 4 d bytes in
// and 9/8 d out a row and head, the gather the other way round.  Minima and maxima are taken on pairs, the grid
// without conversions, quotient and border two at a time.
//
// Measured: 8 prompts of 700 to 4096 tokens, 8 KV heads, d 128, bf16: 27 us in (106 MB; 66 with a quotient, a floor
// and conversions for each value, 33 with eight lanes a group), 21 us back.  One token of 64 sequences: 5.4 us for
// both in a graph.
#include "paged_tc.cuh"
#include "qpaged.cuh"

namespace dkv {
namespace {

// Two rows a thread take 39 us instead of 27 to write the prompts above (89 registers).  Read back, two tokens of eight
// channels a thread take 21 us; sixteen channels, whose stores then leave gaps, 26.
constexpr int kQaThreads = 256, kQgVec = 2;
constexpr float kQaMost = 61440.f;  // above it lo + 15 step could leave fp16

__device__ inline float2 unpack2(uint32_t x, __half) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
__device__ inline float2 unpack2(uint32_t x, __nv_bfloat16) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// the smaller of two pairs, a NaN where either is one
__device__ inline uint32_t min2(uint32_t x, uint32_t y, __half) {
  const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ inline uint32_t min2(uint32_t x, uint32_t y, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr float kMagic = 12582912.f;  // 1.5 2^23: x + kMagic - kMagic is x rounded to a whole number, ties to even

__device__ inline uint32_t max2(uint32_t x, uint32_t y, __half) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ inline uint32_t max2(uint32_t x, uint32_t y, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The grid of a group between lo and hi.
struct Grid {
  float u, inv;  // spacing, and one over it
  float b, st;   // bias and step in spacings
};
__device__ inline Grid grid_of(float lo, float hi) {
  const float top = fmaxf(fabsf(lo), fabsf(hi)) * 1.015625f;
  // u = 2^e, e = max(exponent of top - 10, -24), in place
  const uint32_t e = max(__float_as_uint(top) & 0x7f800000u, 113u << 23) - (10u << 23);
  Grid g;
  g.u = __uint_as_float(e);
  g.inv = __uint_as_float((254u << 23) - e);
  g.b = __fadd_rn(__fmaf_rn(lo, g.inv, kMagic), -kMagic);
  const float n = __fadd_rn(__fadd_rn(__fmaf_rn(hi, g.inv, kMagic), -kMagic), -g.b);
  // (n + 14) / 15 without its remainder: that is at most 14/15, in the middle of which it is rounded
  g.st = __fadd_rn(__fadd_rn(__fmaf_rn(n + 14.f, 1.f / 15.f, -7.f / 15.f), kMagic), -kMagic);
  return g;
}

struct Rows16 {
  uint32_t w[8];  // sixteen channels
};
struct Quantised {
  uint32_t codes[2], param;  // of a lane's sixteen channels, and of the group: (scale, bias) as two halves
  bool odd;                  // a value was not finite or too large
};

// A group with values that are not finite or too large, or with a step of at most one spacing: element by element.
template <typename T>
__device__ __noinline__ Quantised quantise_rare(Rows16 in, uint32_t lanes) {
  float lo = INFINITY, hi = -INFINITY;
  bool bad = false;
  auto value = [&](int i) {
    const float2 f = unpack2(in.w[i / 2], T());
    const float y = i & 1 ? f.y : f.x;
    bad |= !(fabsf(y) <= kQaMost);
    return y != y ? 0.f : fminf(fmaxf(y, -kQaMost), kQaMost);
  };
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = value(i);
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(lanes, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, o));
  }
  const Grid g = grid_of(lo, hi);
  const float r = g.st > 0.f ? 1.f / g.st : 0.f;
  Quantised q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    q.codes[w] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = value(8 * w + i) * g.inv, k = floorf((t - g.b) * r), border = fmaf(k + 0.5f, g.st, g.b);
      int c = (int)k;
      c += t > border || (t == border && (c & 1));
      q.codes[w] |= (uint32_t)min(max(c, 0), 15) << (4 * i);
    }
    if (g.st == 0.f) q.codes[w] = 0;
  }
  q.param = pack_half2(g.st * g.u, g.b * g.u);
  q.odd = bad;
  return q;
}

// A lane's sixteen channels of a group.
template <typename T>
__device__ inline Quantised quantise(const Rows16& in) {
  // minimum and minus the maximum, two values a register
  const T t = T();
  uint32_t lo2 = in.w[0], hi2 = in.w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = min2(lo2, in.w[i], t);
    hi2 = max2(hi2, in.w[i], t);
  }
  uint32_t m = min2(__byte_perm(lo2, hi2, 0x5410) ^ 0x80000000u, __byte_perm(lo2, hi2, 0x7632) ^ 0x80000000u, t);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) m = min2(m, __shfl_xor_sync(0xffffffffu, m, o), t);
  const float2 range = unpack2(m, t);
  const float lo = range.x, hi = -range.y;
  const Grid g = grid_of(lo, hi);
  // (a step of one spacing lets the largest value be half of one above code 15)
  const bool rare = !(lo >= -kQaMost && hi <= kQaMost) || g.st <= 1.f;
  const uint32_t lanes = __ballot_sync(0xffffffffu, rare);
  if (rare) return quantise_rare<T>(in, lanes);
  // k = round(q - 1/2) of a quotient q that is off by little, as the low bits of kMagic + k; the code is k or k + 1 by
  // the side of the border (b + (k + 1/2) st) u, which is exact, that x lies on: k + 1 above it, and on it if k is odd
  // (a difference of 0 less one has the sign bit)
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(g.st));
  const float ri = r * g.inv, off = fmaf(-g.b, r, -0.5f), su = g.st * g.u, mid = fmaf(0.5f, g.st, g.b) * g.u;
  Quantised q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t z[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2(in.w[4 * w + i], t);
      const float2 k = add2(fma2(x, make_float2(ri, ri), make_float2(off, off)), make_float2(kMagic, kMagic));
      const float2 border = fma2(add2(k, make_float2(-kMagic, -kMagic)), make_float2(su, su), make_float2(mid, mid));
      const float2 d = add2(border, make_float2(-x.x, -x.y));
      z[2 * i] = __float_as_uint(k.x);
      z[2 * i + 1] = __float_as_uint(k.y);
      z[2 * i] += (__float_as_uint(d.x) - (z[2 * i] & 1u)) >> 31;
      z[2 * i + 1] += (__float_as_uint(d.y) - (z[2 * i + 1] & 1u)) >> 31;
    }
    // the low bytes are codes
    const uint32_t b0 = z[1] * 16 + z[0], b1 = z[3] * 16 + z[2], b2 = z[5] * 16 + z[4], b3 = z[7] * 16 + z[6];
    q.codes[w] = __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
  }
  q.param = pack_half2(su, g.b * g.u);
  q.odd = false;
  return q;
}
__device__ inline Rows16 load16(const uint4* at) {
  const uint4 x = __ldg(at), y = __ldg(at + 1);
  return {{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
}

// A thread takes sixteen channels of a row's key and of its value.
template <typename T, int D>
__global__ void __launch_bounds__(kQaThreads) qpaged_append_kernel(PagedArgs a, const uint4* __restrict__ K,
                                                                  const uint4* __restrict__ V, dkv_strides ns,
                                                                  int n_rows, const int64_t* __restrict__ slots,
                                                                  uint8_t* __restrict__ cache) {
  constexpr int R = D / 16;  // lanes of a row
  const int64_t n_slots = (int64_t)a.n_pages << a.page_shift;
  const int c = threadIdx.x % R, lane4 = threadIdx.x & 3, g = c / 4;
  const uint32_t pair = blockIdx.x * (kQaThreads / R) + threadIdx.x / R, row = pair / (uint32_t)a.Hkv;
  const int h = (int)(pair - row * (uint32_t)a.Hkv);
  Rows16 k = {}, v = {};
  uint8_t* to = nullptr;  // the block; null: nothing to write
  int tok = 0;
  if (row < (uint32_t)n_rows) {
    const int64_t slot = __ldg(slots + row);
    if (slot >= 0 && slot < n_slots) {
      const int64_t at = (row * ns.token + h * ns.head) / 8 + 2 * c;
      k = load16(K + at);
      v = load16(V + at);
      const int t = (int)slot & a.page_mask;
      tok = t % kQBlock;
      to = cache + (slot >> a.page_shift) * a.stride_page + h * a.stride_head + (t / kQBlock) * qblock_bytes(D);
    } else if (slot != -1) {
      raise_error(a.err, DKV_DEVERR_INDEX);
    }
  }
  const Quantised qk = quantise<T>(k), qv = quantise<T>(v);
  if (!to) return;
  if (qk.odd || qv.odd) raise_error(a.err, DKV_DEVERR_RANGE);
  uint8_t* codes = to + qcode_off(D, 0, g, tok) + lane4 * 8;
  *reinterpret_cast<uint2*>(codes) = make_uint2(qk.codes[0], qk.codes[1]);
  *reinterpret_cast<uint2*>(codes + 8 * D) = make_uint2(qv.codes[0], qv.codes[1]);
  if (lane4 < 2) *reinterpret_cast<uint32_t*>(to + qparam_off(D, lane4, g, tok)) = lane4 ? qv.param : qk.param;
}

// Eight codes as values in order: fp16 ones, exactly; bf16 ones are their roundings.
template <typename T>
__device__ inline uint4 values_of(uint32_t w, uint32_t param) {
  const uint4 v = qvalues8(w, __low2half2(*reinterpret_cast<__half2*>(&param)), __high2half2(*reinterpret_cast<__half2*>(&param)));
  uint4 o = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                       __byte_perm(v.z, v.w, 0x7632));
  if (Num<T>::kUmma == 1) {
    uint32_t* p = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(p[i], __half());
      p[i] = Num<T>::pack(f.x, f.y);
    }
  }
  return o;
}

// A thread takes eight channels of a token's key and of its value.
template <typename T, int D>
__global__ void __launch_bounds__(kQaThreads) qpaged_gather_kernel(PagedArgs a, const uint8_t* __restrict__ cache,
                                                                  const int32_t* __restrict__ first,
                                                                  const int32_t* __restrict__ counts, int n, uint4* K,
                                                                  uint4* V, dkv_strides os) {
  constexpr int R = D / 8;
  const int b = blockIdx.y, h = (int)(blockIdx.x % (unsigned)a.Hkv);
  int cnt = n;
  if (counts) {
    cnt = __ldg(counts + b);
    if (cnt < 0 || cnt > n) {
      if (threadIdx.x == 0) raise_error(a.err, DKV_DEVERR_INDEX);
      cnt = min(max(cnt, 0), n);
    }
  }
  const int64_t p0 = __ldg(first + b);
  const int c = threadIdx.x % R, i0 = (int)(blockIdx.x / (unsigned)a.Hkv) * kQgVec * (kQaThreads / R) + threadIdx.x / R;
  if (i0 >= cnt) return;
  uint32_t wk[kQgVec], wv[kQgVec], sk[kQgVec], sv[kQgVec];
#pragma unroll
  for (int x = 0; x < kQgVec; ++x) {
    const int i = i0 + x * (kQaThreads / R);
    const int64_t t = p0 + i;
    wk[x] = wv[x] = sk[x] = sv[x] = 0;
    if (i >= cnt) continue;
    if (t < 0 || t >= a.cap) {
      raise_error(a.err, DKV_DEVERR_INDEX);
      continue;
    }
    const int page = paged_page(a, b, (int)t), tok = (int)t & a.page_mask;
    if (page >= a.n_pages) continue;
    const uint8_t* block = cache + page * a.stride_page + h * a.stride_head + (tok / kQBlock) * qblock_bytes(D);
    const uint32_t* code = reinterpret_cast<const uint32_t*>(block + qcode_off(D, 0, c / 8, tok % kQBlock) + 4 * (c & 7));
    const uint32_t* param = reinterpret_cast<const uint32_t*>(block + qparam_off(D, 0, c / 8, tok % kQBlock));
    wk[x] = __ldg(code);
    wv[x] = __ldg(code + 2 * D);
    sk[x] = __ldg(param);
    sv[x] = __ldg(param + D / 4);
  }
  const int64_t at = (b * os.batch + h * os.head) / 8 + c;
#pragma unroll
  for (int x = 0; x < kQgVec; ++x) {
    const int i = i0 + x * (kQaThreads / R);
    if (i >= cnt) return;
    K[at + i * os.token / 8] = values_of<T>(wk[x], sk[x]);
    V[at + i * os.token / 8] = values_of<T>(wv[x], sv[x]);
  }
}

}  // namespace

cudaError_t launch_qpaged_append(const PagedArgs& a, int d, int dtype, const void* K, const void* V,
                                 const dkv_strides& ns, int n_rows, const int64_t* slots, uint8_t* cache, cudaStream_t s) {
  const int64_t per = kQaThreads, pieces = (int64_t)n_rows * a.Hkv * (d / 16);
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
  const int per = kQaThreads / (d / 8) * kQgVec;
  auto go = [&](auto kernel) {
    kernel<<<dim3((unsigned)((n + per - 1) / per) * (unsigned)a.Hkv, a.B), kQaThreads, 0, s>>>(a, cache, first, counts, n, static_cast<uint4*>(K),
                                                                          static_cast<uint4*>(V), os);
  };
  if (dtype == DKV_BF16) d == 128 ? go(qpaged_gather_kernel<__nv_bfloat16, 128>) : go(qpaged_gather_kernel<__nv_bfloat16, 64>);
  else d == 128 ? go(qpaged_gather_kernel<__half, 128>) : go(qpaged_gather_kernel<__half, 64>);
  return cudaGetLastError();
}

}  // namespace dkv
