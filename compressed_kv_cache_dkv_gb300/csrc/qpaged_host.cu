// Host side of the serving-step operators: argument checks and the extern "C" entry points of dkv_paged_plan,
// dkv_qk_norm_rope and the paged cache in 4 bits.
#include <cmath>

#include "qpaged.cuh"

namespace dkv {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMostStride = int64_t(1) << 38;
bool in_step(int64_t s, int64_t least, int64_t unit) { return s >= least && s < kMostStride && s % unit == 0; }

// strides of rows with adjacent channels; a dimension of one element may have any stride
int check_rows(const dkv_strides* s, int64_t batch, int64_t heads, int64_t tokens, int d) {
  if (!s) return DKV_ERR_ARG;
  if ((batch > 1 && !in_step(s->batch, d, 8)) || (heads > 1 && !in_step(s->head, d, 8)) || (tokens > 1 && !in_step(s->token, d, 8)))
    return DKV_ERR_ALIGN;
  return DKV_OK;
}

int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

PagedArgs make_args(const dkv_qpaged* p, const int32_t* table, const int32_t* lens, void* ws) {
  PagedArgs a;
  a.B = p->batch;
  a.Hq = p->n_q_heads;
  a.Hkv = p->n_kv_heads;
  a.G = p->n_q_heads / p->n_kv_heads;
  a.page_shift = page_shift(p->page_size);
  a.page_mask = p->page_size - 1;
  a.n_pages = p->n_pages;
  a.max_pages = p->max_pages;
  a.cap = p->max_pages * p->page_size;
  a.window = p->window < a.cap ? p->window : 0;  // a window over the whole capacity hides nothing
  a.sinks = p->sinks < a.cap ? p->sinks : a.cap;
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)p->head_dim);
  a.stride_page = p->stride_page;
  a.stride_head = p->stride_head;
  a.stride_token = 0;
  a.table = table;
  a.lens = lens;
  a.err = static_cast<uint32_t*>(ws);
  return a;
}

size_t ws_need(const dkv_qpaged* p) {
  const size_t dec = qpaged_decode_ws_bytes(p->head_dim), pre = qpaged_prefill_ws_bytes(p->head_dim);
  return round_up(dec > pre ? dec : pre, 256);
}

int check_call(const dkv_qpaged* p, const void* ws, size_t ws_bytes) {
  const int st = dkv_qpaged_check(p);
  if (st != DKV_OK) return st;
  if (!ws) return DKV_ERR_ARG;
  if (!aligned(ws, 16)) return DKV_ERR_ALIGN;
  if (ws_bytes < ws_need(p)) return DKV_ERR_WORKSPACE;
  return DKV_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? DKV_OK : DKV_ERR_CUDA; }

}  // namespace
}  // namespace dkv

using namespace dkv;

extern "C" {

size_t dkv_paged_plan_workspace_bytes(int32_t batch) { return batch >= 1 && batch <= 4096 ? plan_ws_bytes(batch) : 0; }

int dkv_paged_plan(int32_t batch, int32_t page_size, int32_t n_pages, int32_t max_pages, const int32_t* lens,
                   const int32_t* news, int32_t* free_pages, int32_t free_cap, const int32_t* n_free, int32_t* page_table,
                   int32_t rows, int64_t* slots, int32_t* positions, int32_t* starts, int32_t* granted, int32_t* new_lens,
                   int32_t* new_n_free, void* workspace, size_t ws_bytes, void* stream) {
  if (batch < 1 || page_size < 1 || n_pages < 1 || max_pages < 1 || free_cap < 0 || rows < 0) return DKV_ERR_ARG;
  if (batch > 4096 || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) ||
      (int64_t)max_pages * page_size > (1 << 20) || rows > (1 << 30))
    return DKV_ERR_UNSUPPORTED;
  if (!lens || !news || !n_free || !page_table || !starts || !granted || !new_lens || !new_n_free || !workspace ||
      (free_cap > 0 && !free_pages) || (rows > 0 && (!slots || !positions)))
    return DKV_ERR_ARG;
  const void* ints[] = {lens, news, free_pages, n_free, page_table, positions, starts, granted, new_lens, new_n_free};
  for (const void* x : ints)
    if (!aligned(x, 4)) return DKV_ERR_ALIGN;
  if (!aligned(slots, 8) || !aligned(workspace, 16)) return DKV_ERR_ALIGN;
  if (ws_bytes < plan_ws_bytes(batch)) return DKV_ERR_WORKSPACE;
  PlanArgs a;
  a.B = batch;
  a.page_shift = page_shift(page_size);
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.rows = rows;
  a.free_cap = free_cap;
  a.lens = lens;
  a.news = news;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.table = page_table;
  a.slots = slots;
  a.positions = positions;
  a.starts = starts;
  a.granted = granted;
  a.new_lens = new_lens;
  a.new_n_free = new_n_free;
  a.err = static_cast<uint32_t*>(workspace);
  return done(launch_paged_plan(a, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

int dkv_qk_norm_rope(const dkv_rotate* r, const void* q, const dkv_strides* qs, const void* k, const dkv_strides* ks,
                     const void* q_gain, const void* k_gain, const int32_t* positions, void* q_out, const dkv_strides* qos,
                     void* k_out, const dkv_strides* kos, const dkv_paged* p, const void* v, const dkv_strides* vs,
                     const int64_t* slots, void* k_pool, void* v_pool, void* workspace, size_t ws_bytes, void* stream) {
  if (!r || r->rows < 0 || r->n_q_heads < 1 || r->n_kv_heads < 1 || r->head_dim < 1 || r->rope_dims < 0 ||
      (r->dtype != DKV_FP16 && r->dtype != DKV_BF16) || (r->norm && !(r->eps >= 0.f && std::isfinite(r->eps))))
    return DKV_ERR_ARG;
  if (r->head_dim != 64 && r->head_dim != 128) return DKV_ERR_UNSUPPORTED;
  if (r->rope_dims > r->head_dim) return DKV_ERR_ARG;
  if (r->rope_dims % 16 || r->n_q_heads > (1 << 16) || r->n_kv_heads > (1 << 16)) return DKV_ERR_UNSUPPORTED;
  const int half = r->rope_dims / 2;
  if (half > 0 && !r->inv_freq && !(r->rope_base > 1.0 && std::isfinite(r->rope_base))) return DKV_ERR_ARG;
  if (r->inv_freq)
    for (int j = 0; j < half; ++j)
      if (!std::isfinite(r->inv_freq[j])) return DKV_ERR_ARG;
  const bool pages = p || v || slots || k_pool || v_pool;
  if (pages) {
    if (!p || !v || !slots || !k_pool || !v_pool) return DKV_ERR_ARG;
    const int st = dkv_paged_check(p);
    if (st != DKV_OK) return st;
    if (p->n_kv_heads != r->n_kv_heads || p->head_dim != r->head_dim || p->dtype != r->dtype) return DKV_ERR_SHAPE;
  }
  if (workspace && !aligned(workspace, 16)) return DKV_ERR_ALIGN;
  if (workspace && ws_bytes < kWsHeader) return DKV_ERR_WORKSPACE;
  if (r->rows == 0) return DKV_OK;
  if (!q || !k || !positions || !q_out || (!k_out && !pages)) return DKV_ERR_ARG;
  int st;
  if ((st = check_rows(qs, 1, r->n_q_heads, r->rows, r->head_dim)) != DKV_OK ||
      (st = check_rows(ks, 1, r->n_kv_heads, r->rows, r->head_dim)) != DKV_OK ||
      (st = check_rows(qos, 1, r->n_q_heads, r->rows, r->head_dim)) != DKV_OK ||
      (k_out && (st = check_rows(kos, 1, r->n_kv_heads, r->rows, r->head_dim)) != DKV_OK) ||
      (pages && (st = check_rows(vs, 1, r->n_kv_heads, r->rows, r->head_dim)) != DKV_OK))
    return st;
  const void* rows16[] = {q, k, q_gain, k_gain, q_out, k_out, v, k_pool, v_pool};
  for (const void* x : rows16)
    if (!aligned(x, 16)) return DKV_ERR_ALIGN;
  if (!aligned(positions, 4) || !aligned(slots, 8)) return DKV_ERR_ALIGN;
  RotateArgs a = {};
  a.rows = r->rows;
  a.hq = r->n_q_heads;
  a.hkv = r->n_kv_heads;
  a.half = half;
  a.norm = r->norm != 0;
  a.eps = r->eps;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.positions = positions;
  a.q_out = q_out;
  a.k_out = k_out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.slots = slots;
  a.qs[0] = qs->token, a.qs[1] = qs->head;
  a.ks[0] = ks->token, a.ks[1] = ks->head;
  a.qos[0] = qos->token, a.qos[1] = qos->head;
  if (k_out) a.kos[0] = kos->token, a.kos[1] = kos->head;
  if (pages) {
    a.vs[0] = vs->token, a.vs[1] = vs->head;
    a.page_shift = page_shift(p->page_size);
    a.page_mask = p->page_size - 1;
    a.n_slots = (int64_t)p->n_pages * p->page_size;
    a.stride_page = p->stride_page;
    a.stride_head = p->stride_head;
    a.stride_token = p->stride_token;
  }
  a.err = static_cast<uint32_t*>(workspace);
  for (int j = 0; j < half; ++j) {
    const double f = r->inv_freq ? r->inv_freq[j] : std::pow(r->rope_base, -2.0 * j / r->rope_dims);
    double turns = f * 0.15915494309189535;  // of the circle, a position
    turns -= std::floor(turns);
    // (the product is below 2^64 but for a fraction that rounds up to 1)
    a.turn[j] = turns >= 1.0 ? 0ull : (uint64_t)(turns * 18446744073709551616.0);
  }
  return done(launch_qk_norm_rope(a, r->head_dim, r->dtype, static_cast<cudaStream_t>(stream)));
}

int dkv_qpaged_check(const dkv_qpaged* p) {
  if (!p) return DKV_ERR_ARG;
  if (p->batch < 1 || p->n_q_heads < 1 || p->n_kv_heads < 1 || p->head_dim < 1 || p->page_size < 1 || p->n_pages < 1 ||
      p->max_pages < 1 || p->window < 0 || p->sinks < 0 || (p->dtype != DKV_FP16 && p->dtype != DKV_BF16))
    return DKV_ERR_ARG;
  if (p->n_q_heads % p->n_kv_heads != 0) return DKV_ERR_SHAPE;
  if ((p->head_dim != 64 && p->head_dim != 128) || p->n_q_heads / p->n_kv_heads > 8) return DKV_ERR_UNSUPPORTED;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return DKV_ERR_UNSUPPORTED;
  if (p->batch > 4096 || (int64_t)p->batch * p->n_kv_heads > 65535) return DKV_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page_size > (1 << 20)) return DKV_ERR_UNSUPPORTED;
  const int64_t page = (int64_t)p->page_size / kQBlock * qblock_bytes(p->head_dim);
  if ((p->n_pages > 1 && !in_step(p->stride_page, page, 16)) || (p->n_kv_heads > 1 && !in_step(p->stride_head, page, 16)))
    return DKV_ERR_ALIGN;
  return DKV_OK;
}

size_t dkv_qpaged_workspace_bytes(const dkv_qpaged* p) { return dkv_qpaged_check(p) == DKV_OK ? ws_need(p) : 0; }

int dkv_qpaged_append(const dkv_qpaged* p, const void* K, const void* V, const dkv_strides* ns, int32_t rows,
                      const int64_t* slots, void* cache, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, workspace, ws_bytes);
  if (st != DKV_OK) return st;
  if (rows < 0) return DKV_ERR_ARG;
  if (rows == 0) return DKV_OK;
  if (!K || !V || !slots || !cache) return DKV_ERR_ARG;
  if (rows > (1 << 30) || (int64_t)rows * p->n_kv_heads > (int64_t(1) << 31)) return DKV_ERR_UNSUPPORTED;
  if ((st = check_rows(ns, 1, p->n_kv_heads, rows, p->head_dim)) != DKV_OK) return st;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, nullptr, nullptr, workspace);
  return done(launch_qpaged_append(a, p->head_dim, p->dtype, K, V, *ns, rows, slots, static_cast<uint8_t*>(cache),
                                   static_cast<cudaStream_t>(stream)));
}

int dkv_qpaged_gather(const dkv_qpaged* p, const void* cache, const int32_t* page_table, const int32_t* first,
                      const int32_t* counts, int32_t n, void* K, void* V, const dkv_strides* os, void* workspace,
                      size_t ws_bytes, void* stream) {
  int st = check_call(p, workspace, ws_bytes);
  if (st != DKV_OK) return st;
  if (n < 0) return DKV_ERR_ARG;
  if (n == 0) return DKV_OK;
  if (!cache || !page_table || !first || !K || !V) return DKV_ERR_ARG;
  if (n > p->max_pages * p->page_size) return DKV_ERR_SHAPE;
  if ((st = check_rows(os, p->batch, p->n_kv_heads, n, p->head_dim)) != DKV_OK) return st;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(cache, 16) || !aligned(page_table, 4) || !aligned(first, 4) || !aligned(counts, 4))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, nullptr, workspace);
  return done(launch_qpaged_gather(a, p->head_dim, p->dtype, static_cast<const uint8_t*>(cache), first, counts, n, K, V, *os,
                                   static_cast<cudaStream_t>(stream)));
}

int dkv_qpaged_decode(const dkv_qpaged* p, const void* q, const dkv_strides* qs, const void* cache, const int32_t* page_table,
                      const int32_t* lens, void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, workspace, ws_bytes);
  if (st != DKV_OK) return st;
  if (!q || !cache || !page_table || !lens || !out) return DKV_ERR_ARG;
  if ((st = check_rows(qs, p->batch, p->n_q_heads, 1, p->head_dim)) != DKV_OK) return st;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  return done(launch_qpaged_decode(a, p->head_dim, p->dtype, q, *qs, static_cast<const uint8_t*>(cache), out, lse,
                                   static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

int dkv_qpaged_prefill(const dkv_qpaged* p, const void* q, const dkv_strides* qs, int32_t rows, int32_t max_q,
                       const int32_t* starts, const void* cache, const int32_t* page_table, const int32_t* lens, void* out,
                       const dkv_strides* os, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_call(p, workspace, ws_bytes);
  if (st != DKV_OK) return st;
  if (rows < 0 || max_q < 0) return DKV_ERR_ARG;
  if (rows == 0 || max_q == 0) return DKV_OK;
  if (!q || !starts || !cache || !page_table || !lens || !out) return DKV_ERR_ARG;
  if (rows > (1 << 30)) return DKV_ERR_UNSUPPORTED;
  if (max_q > rows) max_q = rows;
  if (max_q > (1 << 20)) return DKV_ERR_UNSUPPORTED;
  if ((st = check_rows(qs, 1, p->n_q_heads, rows, p->head_dim)) != DKV_OK ||
      (st = check_rows(os, 1, p->n_q_heads, rows, p->head_dim)) != DKV_OK)
    return st;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(starts, 4) || !aligned(page_table, 4) ||
      !aligned(lens, 4) || !aligned(lse, 4))
    return DKV_ERR_ALIGN;
  const PagedArgs a = make_args(p, page_table, lens, workspace);
  const PackedQuery pq = {q, *qs, rows, max_q, starts};
  return done(launch_qpaged_prefill(a, p->head_dim, p->dtype, pq, static_cast<const uint8_t*>(cache), out, *os, lse,
                                    static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
