// Host side of the attention calls declared in include/lora.h: argument
// validation and launches.
#include <cmath>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace {

using ra::clear_stale_error;
using ra::cuda_status;

bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
int64_t elem(const lora_seqs *s) { return s->dtype == LORA_BF16 ? 2 : 4; }

// The geometry and the counts; what the plan's size depends on.
int check_shape(const lora_seqs *s) {
  if (s == nullptr) return LORA_EINVAL;
  if (s->dtype != LORA_BF16 && s->dtype != LORA_F32) return LORA_EINVAL;
  if (s->num_heads < 1 || s->num_heads > LORA_MAX_HEADS || s->num_kv_heads < 1 || s->num_kv_heads > s->num_heads)
    return LORA_ERANGE;
  if (s->head_dim < 8 || s->head_dim > LORA_MAX_HEAD_DIM) return LORA_ERANGE;
  if (s->num_heads % s->num_kv_heads != 0 || s->head_dim % 8 != 0) return LORA_EINVAL;
  if (!(s->scale > 0.f) || !std::isfinite(s->scale)) return LORA_EINVAL;
  if (s->num_seqs < 0 || s->num_seqs > LORA_MAX_SEQS || s->num_tokens < 0 || s->num_tokens > LORA_MAX_TOKENS)
    return LORA_ERANGE;
  return LORA_OK;
}

bool has_cache(const lora_seqs *s) { return s->page_size != 0; }

int check_seqs(const lora_seqs *s) {
  const int st = check_shape(s);
  if (st != LORA_OK) return st;
  if (has_cache(s)) {
    if (s->page_size < 8 || s->page_size > 1024 || (s->page_size & (s->page_size - 1)) != 0) return LORA_EINVAL;
    if (s->max_pages < 1 || (int64_t)s->max_pages * s->page_size > LORA_MAX_KV_LEN) return LORA_ERANGE;
  }
  if (s->plan == nullptr || s->plan_bytes < lora_seqs_plan_bytes(s)) return LORA_EINVAL;
  if (!aligned(s->plan, 16)) return LORA_EALIGN;
  return LORA_OK;
}

// A matrix of the batch's rows, `width` wide.
int check_rows(const lora_seqs *s, const void *p, int64_t ld, int64_t width) {
  if (p == nullptr || ld < width) return LORA_EINVAL;
  if (!aligned(p, 16) || ld * elem(s) % 16 != 0) return LORA_EALIGN;
  return LORA_OK;
}

int check_cache(const lora_seqs *s, const lora_kv_cache *c) {
  if (!has_cache(s) || c == nullptr) return LORA_EINVAL;
  if (c->k == nullptr || c->v == nullptr || s->block_table == nullptr || s->ld_table < s->max_pages) return LORA_EINVAL;
  if (c->num_pages < 1) return LORA_ERANGE;
  if (!aligned(s->block_table, 4) || !aligned(c->k, 16) || !aligned(c->v, 16)) return LORA_EALIGN;
  for (const int64_t d : {c->k_page, c->k_row, c->k_head, c->v_page, c->v_row, c->v_head}) {
    if (d < 1) return LORA_EINVAL;
    if (d * elem(s) % 16 != 0) return LORA_EALIGN;
  }
  return LORA_OK;
}

// Whether two column ranges of rows (strides in bytes) share memory. Ranges of one matrix lie beside each other.
bool overlap(const void *p, int64_t ldp, int64_t wp, const void *q, int64_t ldq, int64_t wq, int64_t rows) {
  const intptr_t a = reinterpret_cast<intptr_t>(p), b = reinterpret_cast<intptr_t>(q);
  if (a + (rows - 1) * ldp + wp <= b || b + (rows - 1) * ldq + wq <= a) return false;
  if (ldp != ldq) return true;
  const int64_t d = ((b - a) % ldp + ldp) % ldp;  // q's first column in p's rows
  return d < wp || ldp - d < wq;
}

int run(const lora_seqs *s, ra::AttnArgs &a, const void *q, int64_t ldq, void *out, int64_t ldo, float *lse, void *ws,
        size_t ws_bytes, lora_stream_t stream) {
  const int64_t width = (int64_t)s->num_heads * s->head_dim;
  int st = check_rows(s, q, ldq, width);
  if (st == LORA_OK) st = check_rows(s, out, ldo, width);
  if (st != LORA_OK) return st;
  const int64_t es = elem(s);
  if (overlap(out, ldo * es, width * es, q, ldq * es, width * es, s->num_tokens)) return LORA_EINVAL;
  if (!aligned(lse, 4)) return LORA_EALIGN;
  if (ws == nullptr || ws_bytes < lora_attn_workspace_bytes(s)) return LORA_EINVAL;
  if (!aligned(ws, 16)) return LORA_EALIGN;
  a.s = ra::attn_shape(*s);
  a.p = ra::attn_plan(a.s, s->num_seqs, s->num_tokens);
  a.plan = static_cast<const int32_t *>(s->plan);
  a.err = static_cast<int32_t *>(s->plan) + ra::AttnPlan::kErr;
  a.q = q;
  a.ldq = ldq;
  a.out = out;
  a.ldo = ldo;
  a.lse = lse;
  a.ws = static_cast<float *>(ws);
  a.num_tokens = s->num_tokens;
  const int64_t max_kv = has_cache(s) ? (int64_t)s->page_size * s->max_pages : s->num_tokens;
  const cudaStream_t st_ = (cudaStream_t)stream;
  cudaError_t e = a.s.few > 0 ? ra::launch_attn_few(a, st_)
                  : a.s.tc                          ? ra::launch_attn_tc(a, st_)
                                                    : ra::launch_attn_rows(a, st_);
  if (e == cudaSuccess && ra::attn_may_split(a.s, max_kv)) e = ra::launch_attn_combine(a, (cudaStream_t)stream);
  return cuda_status(e);
}

}  // namespace

extern "C" {

size_t lora_seqs_plan_bytes(const lora_seqs *seqs) {
  if (check_shape(seqs) != LORA_OK) return 0;
  return ra::attn_plan_bytes(*seqs);
}

size_t lora_attn_workspace_bytes(const lora_seqs *seqs) {
  if (check_shape(seqs) != LORA_OK) return 0;
  const ra::AttnShape s = ra::attn_shape(*seqs);
  return (size_t)(ra::attn_slot_rows(*seqs) * s.Hkv * (s.D + 2)) * sizeof(float);
}

int lora_prepare_seqs(const lora_seqs *seqs, lora_stream_t stream) {
  clear_stale_error();
  const int st = check_seqs(seqs);
  if (st != LORA_OK) return st;
  if (seqs->num_seqs > 0 && seqs->q_start == nullptr) return LORA_EINVAL;
  if (!aligned(seqs->q_start, 4) || !aligned(seqs->kv_len, 4)) return LORA_EALIGN;
  return cuda_status(ra::launch_prepare_seqs(*seqs, (cudaStream_t)stream));
}

int lora_kv_write(const lora_seqs *seqs, const lora_kv_cache *cache, const void *k, int64_t ldk, const void *v,
                  int64_t ldv, lora_stream_t stream) {
  clear_stale_error();
  int st = check_seqs(seqs);
  if (st == LORA_OK) st = check_cache(seqs, cache);
  if (st != LORA_OK) return st;
  if (seqs->num_seqs == 0 || seqs->num_tokens == 0) return LORA_OK;
  const int64_t width = (int64_t)seqs->num_kv_heads * seqs->head_dim;
  st = check_rows(seqs, k, ldk, width);
  if (st == LORA_OK) st = check_rows(seqs, v, ldv, width);
  if (st != LORA_OK) return st;
  return cuda_status(ra::launch_kv_write(*seqs, *cache, k, ldk, v, ldv, (cudaStream_t)stream));
}

int lora_attn_prompt(const lora_seqs *seqs, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                     int64_t ldv, void *out, int64_t ldo, float *lse, void *ws, size_t ws_bytes, lora_stream_t stream) {
  clear_stale_error();
  int st = check_seqs(seqs);
  if (st != LORA_OK) return st;
  if (seqs->kv_len != nullptr) return LORA_EINVAL;
  if (seqs->num_seqs == 0 || seqs->num_tokens == 0) return LORA_OK;
  const int64_t width = (int64_t)seqs->num_kv_heads * seqs->head_dim;
  st = check_rows(seqs, k, ldk, width);
  if (st == LORA_OK) st = check_rows(seqs, v, ldv, width);
  if (st != LORA_OK) return st;
  const int64_t es = elem(seqs), wide = (int64_t)seqs->num_heads * seqs->head_dim;
  if (out == nullptr || ldo < wide) return LORA_EINVAL;
  if (overlap(out, ldo * es, wide * es, k, ldk * es, width * es, seqs->num_tokens) ||
      overlap(out, ldo * es, wide * es, v, ldv * es, width * es, seqs->num_tokens))
    return LORA_EINVAL;
  ra::AttnArgs a{};
  a.kv.k = k;
  a.kv.v = v;
  a.kv.k_row = ldk;
  a.kv.v_row = ldv;
  a.kv.k_head = a.kv.v_head = seqs->head_dim;
  return run(seqs, a, q, ldq, out, ldo, lse, ws, ws_bytes, stream);
}

int lora_attn_paged(const lora_seqs *seqs, const lora_kv_cache *cache, const void *q, int64_t ldq, void *out,
                    int64_t ldo, float *lse, void *ws, size_t ws_bytes, lora_stream_t stream) {
  clear_stale_error();
  int st = check_seqs(seqs);
  if (st == LORA_OK) st = check_cache(seqs, cache);
  if (st != LORA_OK) return st;
  if (seqs->num_seqs == 0 || seqs->num_tokens == 0) return LORA_OK;
  ra::AttnArgs a{};
  a.kv.k = cache->k;
  a.kv.v = cache->v;
  a.kv.k_page = cache->k_page;
  a.kv.k_row = cache->k_row;
  a.kv.k_head = cache->k_head;
  a.kv.v_page = cache->v_page;
  a.kv.v_row = cache->v_row;
  a.kv.v_head = cache->v_head;
  a.kv.page_size = seqs->page_size;
  while ((1 << a.kv.log2_page) < seqs->page_size) ++a.kv.log2_page;
  a.kv.num_pages = cache->num_pages;
  a.kv.max_pages = seqs->max_pages;
  a.kv.table = seqs->block_table;
  a.kv.ld_table = seqs->ld_table;
  return run(seqs, a, q, ldq, out, ldo, lse, ws, ws_bytes, stream);
}

int lora_query_seqs(const lora_seqs *seqs, int32_t *out, lora_stream_t stream) {
  if (seqs == nullptr || seqs->plan == nullptr || out == nullptr) return LORA_EINVAL;
  clear_stale_error();
  int32_t v[2] = {0, 0};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(v, static_cast<const int32_t *>(seqs->plan) + ra::AttnPlan::kErr, sizeof(v),
                                  cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e);
  *out = v[1];
  if ((v[0] & ra::kErrAttn) != 0) return LORA_EDEVICE;
  return v[0] == 0 && v[1] == 0 ? LORA_OK : LORA_EBADSEQ;
}

}  // extern "C"
