// Host side of the paged-cache operators: descriptor checks, argument checks, the
// tensor maps of the pools and of the queries, and the extern "C" entry points.
#include <atomic>
#include <mutex>

#include "paged.cuh"

namespace dkv {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 38;  // a tensor map holds byte strides below 2^40

bool stride_ok(int64_t s, int64_t least) { return s >= least && s < kMaxStride && s % 8 == 0; }

// strides of a [batch][head][token][d] tensor; a dimension of one element may have any stride
int check_strides(const dkv_strides* s, int64_t batch, int64_t heads, int64_t tokens, int d) {
  if (!s) return DKV_ERR_ARG;
  if ((batch > 1 && !stride_ok(s->batch, d)) || (heads > 1 && !stride_ok(s->head, d)) ||
      (tokens > 1 && !stride_ok(s->token, d)))
    return DKV_ERR_ALIGN;
  return DKV_OK;
}

// the encoder lives in the driver; it is looked up once
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// 4-D map of 16-bit elements {d, n1, n2, n3} under element strides {1, s1, s2, s3}, boxes of
// 64 channels x `rows` of dimension 1, 128-byte swizzle
bool encode(CUtensorMap* map, int dtype, const void* base, int d, int64_t n1, int64_t n2, int64_t n3, int64_t s1,
            int64_t s2, int64_t s3, int rows) {
  EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
  // the stride of a dimension of one element is never used, but has to be a legal one
  const cuuint64_t strides[3] = {(cuuint64_t)(n1 > 1 ? s1 : d) * 2, (cuuint64_t)(n2 > 1 ? s2 : d) * 2,
                                 (cuuint64_t)(n3 > 1 ? s3 : d) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return f(map, dtype == DKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
           const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_pool(CUtensorMap* map, const dkv_paged* p, const void* pool) {
  return encode(map, p->dtype, pool, p->head_dim, p->page_size, p->n_kv_heads, p->n_pages, p->stride_token,
                p->stride_head, p->stride_page, p->page_size < 64 ? p->page_size : 64);
}

bool encode_query(CUtensorMap* map, const dkv_paged* p, const void* q, const dkv_strides& qs, int Tq, int rows) {
  return encode(map, p->dtype, q, p->head_dim, Tq, p->n_q_heads, p->batch, qs.token, qs.head, qs.batch, rows);
}

PagedArgs make_args(const dkv_paged* p, const int32_t* table, const int32_t* lens, void* ws) {
  PagedArgs a;
  a.B = p->batch;
  a.Hq = p->n_q_heads;
  a.Hkv = p->n_kv_heads;
  a.G = p->n_q_heads / p->n_kv_heads;
  a.page_shift = 0;
  while ((1 << a.page_shift) < p->page_size) ++a.page_shift;
  a.page_mask = p->page_size - 1;
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.cap = p->max_pages * p->page_size;
  a.window = p->window < a.cap ? p->window : 0;  // a window over the whole capacity hides nothing
  a.sinks = p->sinks < a.cap ? p->sinks : a.cap;
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)p->head_dim);
  a.stride_page = p->stride_page;
  a.stride_head = p->stride_head;
  a.stride_token = p->stride_token;
  a.table = table;
  a.lens = lens;
  a.err = static_cast<uint32_t*>(ws);
  return a;
}

// [what one call keeps in it, and behind the largest such part the scores of decode with weights]
size_t ws_base(const dkv_paged* p) {
  const PagedArgs a = make_args(p, nullptr, nullptr, nullptr);
  const size_t dec = paged_decode_ws_bytes(p->head_dim), pre = paged_prefill_ws_bytes(p->head_dim);
  const size_t ev = paged_evict_ws_bytes(a, p->head_dim), most = dec > pre ? dec : pre;
  return round_up(most > ev ? most : ev, 256);
}
size_t ws_need(const dkv_paged* p, bool with_weights) {
  return ws_base(p) + (with_weights ? (size_t)p->batch * p->n_kv_heads * p->max_pages * p->page_size * 32 : 0);
}

// what all calls check alike
int check_call(const dkv_paged* p, const int32_t* table, const void* ws, size_t ws_bytes, bool with_weights) {
  const int st = dkv_paged_check(p);
  if (st != DKV_OK) return st;
  if (!table || !ws) return DKV_ERR_ARG;
  if (!aligned4(table) || !aligned16(ws)) return DKV_ERR_ALIGN;
  if (ws_bytes < ws_need(p, with_weights)) return DKV_ERR_WORKSPACE;
  return DKV_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? DKV_OK : DKV_ERR_CUDA; }

}  // namespace
}  // namespace dkv

using namespace dkv;

extern "C" {

int dkv_paged_check(const dkv_paged* p) {
  if (!p) return DKV_ERR_ARG;
  if (p->batch < 1 || p->n_q_heads < 1 || p->n_kv_heads < 1 || p->head_dim < 1 || p->page_size < 1 || p->n_pages < 1 ||
      p->max_pages < 1 || p->window < 0 || p->sinks < 0 || (p->dtype != DKV_FP16 && p->dtype != DKV_BF16))
    return DKV_ERR_ARG;
  if (p->n_q_heads % p->n_kv_heads != 0) return DKV_ERR_SHAPE;
  if ((p->head_dim != 64 && p->head_dim != 128) || p->n_q_heads / p->n_kv_heads > 8) return DKV_ERR_UNSUPPORTED;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return DKV_ERR_UNSUPPORTED;
  if (p->batch > 4096 || (int64_t)p->batch * p->n_kv_heads > 65535) return DKV_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page_size > (1 << 20)) return DKV_ERR_UNSUPPORTED;
  if ((p->n_pages > 1 && !stride_ok(p->stride_page, p->head_dim)) ||
      (p->n_kv_heads > 1 && !stride_ok(p->stride_head, p->head_dim)) || !stride_ok(p->stride_token, p->head_dim))
    return DKV_ERR_ALIGN;
  return DKV_OK;
}

size_t dkv_paged_workspace_bytes(const dkv_paged* p, int32_t with_weights) {
  return dkv_paged_check(p) == DKV_OK ? ws_need(p, with_weights != 0) : 0;
}

int dkv_paged_append(const dkv_paged* p, const void* K_new, const void* V_new, const dkv_strides* ns, int32_t n_new,
                     const int32_t* pos, const int32_t* counts, void* k_pool, void* v_pool, const int32_t* page_table,
                     void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, page_table, workspace, ws_bytes, false);
  if (st != DKV_OK) return st;
  if (n_new < 0) return DKV_ERR_ARG;
  if (n_new == 0) return DKV_OK;
  if (!K_new || !V_new || !pos || !k_pool || !v_pool) return DKV_ERR_ARG;
  if (n_new > p->max_pages * p->page_size) return DKV_ERR_SHAPE;
  if ((st = check_strides(ns, p->batch, p->n_kv_heads, n_new, p->head_dim)) != DKV_OK) return st;
  if (!aligned16(K_new) || !aligned16(V_new) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned4(pos) ||
      !aligned4(counts))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, nullptr, workspace);
  return done(launch_paged_append(a, p->head_dim, K_new, V_new, *ns, n_new, pos, counts, k_pool, v_pool,
                                  static_cast<cudaStream_t>(stream)));
}

int dkv_paged_decode(const dkv_paged* p, const void* q, const dkv_strides* qs, const void* k_pool, const void* v_pool,
                     const int32_t* page_table, const int32_t* lens, void* out, float* lse, float* weights,
                     void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, page_table, workspace, ws_bytes, weights != nullptr);
  if (st != DKV_OK) return st;
  if (!q || !k_pool || !v_pool || !lens || !out || (weights && !lse)) return DKV_ERR_ARG;
  if ((st = check_strides(qs, p->batch, p->n_q_heads, 1, p->head_dim)) != DKV_OK) return st;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned4(lens) ||
      !aligned4(lse) || !aligned4(weights))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  PagedMaps m;
  if (!encode_pool(&m.k, p, k_pool) || !encode_pool(&m.v, p, v_pool)) return DKV_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return done(launch_paged_decode(a, p->head_dim, p->dtype, m, q, *qs, out, lse, weights,
                                  reinterpret_cast<float*>(ws + ws_base(p)), ws, static_cast<cudaStream_t>(stream)));
}

int dkv_paged_prefill(const dkv_paged* p, const void* q, const dkv_strides* qs, int32_t Tq, const void* k_pool,
                      const void* v_pool, const int32_t* page_table, const int32_t* lens, const int32_t* q_lens,
                      void* out, const dkv_strides* os, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, page_table, workspace, ws_bytes, false);
  if (st != DKV_OK) return st;
  if (Tq < 0) return DKV_ERR_ARG;
  if (Tq == 0) return DKV_OK;
  if (!q || !k_pool || !v_pool || !lens || !out) return DKV_ERR_ARG;
  if (Tq > (1 << 20)) return DKV_ERR_UNSUPPORTED;
  if ((st = check_strides(qs, p->batch, p->n_q_heads, Tq, p->head_dim)) != DKV_OK ||
      (st = check_strides(os, p->batch, p->n_q_heads, Tq, p->head_dim)) != DKV_OK)
    return st;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned4(lens) ||
      !aligned4(q_lens) || !aligned4(lse))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  PagedMaps m;
  CUtensorMap qm;
  if (!encode_pool(&m.k, p, k_pool) || !encode_pool(&m.v, p, v_pool) || !encode_query(&qm, p, q, *qs, Tq, paged_prefill_rows(Tq)))
    return DKV_ERR_CUDA;
  const PagedQuery pq = {q, *qs, Tq, q_lens};
  return done(launch_paged_prefill(a, p->head_dim, p->dtype, m, qm, pq, v_pool, k_pool, out, *os, lse,
                                   static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

int dkv_paged_weights(const dkv_paged* p, const void* q, const dkv_strides* qs, int32_t Tq, const float* lse,
                      const void* k_pool, const int32_t* page_table, const int32_t* lens, const int32_t* q_lens,
                      float* weights, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, page_table, workspace, ws_bytes, false);
  if (st != DKV_OK) return st;
  if (Tq < 0) return DKV_ERR_ARG;
  if (Tq == 0) return DKV_OK;
  if (!q || !lse || !k_pool || !lens || !weights) return DKV_ERR_ARG;
  if (Tq > (1 << 20)) return DKV_ERR_UNSUPPORTED;
  if ((st = check_strides(qs, p->batch, p->n_q_heads, Tq, p->head_dim)) != DKV_OK) return st;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned4(lens) || !aligned4(q_lens) || !aligned4(lse) ||
      !aligned4(weights))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  CUtensorMap km, qm;
  if (!encode_pool(&km, p, k_pool) || !encode_query(&qm, p, q, *qs, Tq, paged_weights_rows(p->n_q_heads / p->n_kv_heads, Tq))) return DKV_ERR_CUDA;
  const PagedQuery pq = {q, *qs, Tq, q_lens};
  return done(launch_paged_weights(a, p->head_dim, p->dtype, km, qm, pq, lse, weights,
                                   static_cast<cudaStream_t>(stream)));
}

int dkv_paged_evict(const dkv_paged* p, void* k_pool, void* v_pool, const int32_t* page_table, const int32_t* lens,
                    const float* weights, int32_t budget, int32_t first, int32_t recent, const int32_t* new_table,
                    int32_t new_max_pages, int32_t* kept, int32_t* new_lens, float* new_weights, void* workspace,
                    size_t ws_bytes, void* stream) {
  const int st = check_call(p, page_table, workspace, ws_bytes, false);
  if (st != DKV_OK) return st;
  if (budget < 1 || first < 0 || recent < 0 || new_max_pages < 1) return DKV_ERR_ARG;
  if (!k_pool || !v_pool || !lens || !weights || !new_table || !kept || !new_lens || !new_weights) return DKV_ERR_ARG;
  if ((int64_t)first + recent > budget || budget > p->max_pages * p->page_size ||
      (int64_t)new_max_pages * p->page_size < budget)
    return DKV_ERR_SHAPE;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned4(lens) || !aligned4(weights) || !aligned4(new_table) ||
      !aligned4(kept) || !aligned4(new_lens) || !aligned4(new_weights))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  PagedEvict e;
  e.budget = budget;
  e.first = first;
  e.recent = recent;
  e.new_max_pages = new_max_pages;
  e.weights = weights;
  e.new_table = new_table;
  e.kept = kept;
  e.new_lens = new_lens;
  e.new_weights = new_weights;
  return done(launch_paged_evict(a, p->head_dim, e, k_pool, v_pool, static_cast<uint8_t*>(workspace),
                                 static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
