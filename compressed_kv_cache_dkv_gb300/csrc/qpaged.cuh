// Shared by the kernels of the paged cache in 4 bits: the layout of a page, and the launchers.
//
// A page of a KV head is a row of blocks of 16 tokens, 18 d bytes each (G = d / 64 groups of 64 channels):
//   [K codes: G x 16 tokens x 32 bytes][V codes: the same]
//   [K scale, bias: 16 tokens x G x 2 fp16][V scale, bias: the same]
// A value is scale * code + bias; append chooses scale and bias so that this is an fp16 number exactly.
#pragma once

#include "paged.cuh"

namespace dkv {

constexpr int kQBlock = 16;  // tokens of a block
__host__ __device__ constexpr int qblock_bytes(int d) { return 18 * d; }
// byte of a block's parts (kv: 0 K, 1 V): the code word of 8 channels, and the (scale, bias) pair
__host__ __device__ constexpr int qcode_off(int d, int kv, int g, int tok) { return kv * 8 * d + (g * kQBlock + tok) * 32; }
__host__ __device__ constexpr int qparam_off(int d, int kv, int g, int tok) {
  return (16 + kv) * d + (tok * (d / 64) + g) * 4;
}

// Eight codes as values, in the order 0 4 1 5 2 6 3 7.  1024 + code and 1024 + 16 code are the halves whose low
// bits are the code's; every step is exact.
__device__ inline uint4 qvalues8(uint32_t x, __half2 s, __half2 b) {
  const uint32_t y = x >> 8;
  auto half2_of = [](uint32_t w) { return *reinterpret_cast<__half2*>(&w); };
  auto bits = [](__half2 h) { return *reinterpret_cast<uint32_t*>(&h); };
  const __half2 base = half2_of(0x64006400u), sixteenth = half2_of(0x2c002c00u), minus64 = half2_of(0xd400d400u);
  const __half2 c0 = __hsub2(half2_of((x & 0x000f000fu) | 0x64006400u), base);
  const __half2 c1 = __hfma2(half2_of((x & 0x00f000f0u) | 0x64006400u), sixteenth, minus64);
  const __half2 c2 = __hsub2(half2_of((y & 0x000f000fu) | 0x64006400u), base);
  const __half2 c3 = __hfma2(half2_of((y & 0x00f000f0u) | 0x64006400u), sixteenth, minus64);
  return make_uint4(bits(__hfma2(c0, s, b)), bits(__hfma2(c1, s, b)), bits(__hfma2(c2, s, b)), bits(__hfma2(c3, s, b)));
}

// In the kernels below PagedArgs holds the strides of a page and of a head in bytes.
cudaError_t launch_qpaged_append(const PagedArgs& a, int d, int dtype, const void* K, const void* V,
                                 const dkv_strides& ns, int n_rows, const int64_t* slots, uint8_t* cache, cudaStream_t s);
cudaError_t launch_qpaged_gather(const PagedArgs& a, int d, int dtype, const uint8_t* cache, const int32_t* first,
                                 const int32_t* counts, int n, void* K, void* V, const dkv_strides& os, cudaStream_t s);
size_t qpaged_decode_ws_bytes(int d);
cudaError_t launch_qpaged_decode(const PagedArgs& a, int d, int dtype, const void* q, const dkv_strides& qs,
                                 const uint8_t* cache, void* out, float* lse, uint8_t* ws, cudaStream_t s);
// queries in a row: those of sequence b are rows starts[b] .. starts[b + 1] - 1
struct PackedQuery {
  const void* q;
  dkv_strides qs;
  int rows, max_q;
  const int32_t* starts;
};
size_t qpaged_prefill_ws_bytes(int d);
cudaError_t launch_qpaged_prefill(const PagedArgs& a, int d, int dtype, const PackedQuery& q, const uint8_t* cache,
                                  void* out, const dkv_strides& os, float* lse, uint8_t* ws, cudaStream_t s);

// paged_plan.cu
struct PlanArgs {
  int B, page_shift, n_pages, max_pages, rows, free_cap;
  const int32_t* lens;
  const int32_t* news;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* table;
  int64_t* slots;
  int32_t* positions;
  int32_t* starts;
  int32_t* granted;
  int32_t* new_lens;
  int32_t* new_n_free;
  uint32_t* err;
};
size_t plan_ws_bytes(int B);
cudaError_t launch_paged_plan(const PlanArgs& a, uint8_t* ws, cudaStream_t s);

// qk_norm_rope.cu
struct RotateArgs {
  int rows, hq, hkv, half;  // half: pairs of channels that turn
  int norm;
  float eps;
  const void* q;
  const void* k;
  const void* v;
  const void* q_gain;
  const void* k_gain;
  const int32_t* positions;
  void* q_out;
  void* k_out;
  void* k_pool;
  void* v_pool;
  const int64_t* slots;
  int64_t n_slots;
  int page_shift, page_mask;
  int64_t stride_page, stride_head, stride_token;
  int64_t qs[2], ks[2], vs[2], qos[2], kos[2];  // token, head
  uint32_t* err;
  uint64_t turn[64];  // pair j turns by turn[j] 2^-64 of a circle a position
};
cudaError_t launch_qk_norm_rope(const RotateArgs& a, int d, int dtype, cudaStream_t s);

}  // namespace dkv
