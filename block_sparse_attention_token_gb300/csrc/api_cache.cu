// extern "C" entry points of the cache of keys and values in 8 bits: argument
// validation (before any CUDA call, so host errors leave outputs untouched) and dispatch.
#include <math.h>

#include "api.cuh"
#include "cache.cuh"

using namespace sparsp;

namespace {

sparsp_status_t check_cache(const sparsp_cache_t* c, CacheDims* s) {
  if (c == nullptr) return SPARSP_ERR_INVALID_ARG;
  if (c->blocks <= 0 || c->heads <= 0 || c->d <= 0 || c->bt <= 0) return SPARSP_ERR_SHAPE;
  if ((c->d != 64 && c->d != 128) || (c->bt != 64 && c->bt != 128) || c->heads > 65535) return SPARSP_ERR_UNSUPPORTED;
  if ((int64_t)c->blocks * c->bt > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;   // int32 slots
  *s = CacheDims{c->blocks, c->heads, c->d, c->bt};
  return SPARSP_OK;
}

sparsp_status_t check_requests(const CacheDims& c, int32_t B, int32_t max_blocks, int64_t tokens) {
  if (B <= 0 || max_blocks <= 0 || tokens < 0) return SPARSP_ERR_SHAPE;
  if (B > kCacheMaxRequests || (int64_t)max_blocks * c.bt > INT32_MAX || tokens > INT32_MAX)
    return SPARSP_ERR_UNSUPPORTED;
  return SPARSP_OK;
}

// Elements between tokens and between heads of new keys or values (0: heads * d and d).
sparsp_status_t check_strides(const CacheDims& c, int elem, int64_t tokens, int64_t* token, int64_t* head) {
  if (*token == 0) *token = (int64_t)c.heads * c.d;
  if (*head == 0) *head = c.d;
  if (*token < c.d || *head < c.d || *token > (int64_t)1 << 40 || *head > (int64_t)1 << 40) return SPARSP_ERR_SHAPE;
  if (tokens > 0 && *token > ((int64_t)1 << 60) / tokens) return SPARSP_ERR_SHAPE;   // (heads below 2^16)
  if (*token * elem % 16 != 0 || *head * elem % 16 != 0) return SPARSP_ERR_ALIGN;
  return SPARSP_OK;
}

// Words of 32 bits that an argument takes up.
struct Words {
  const void* p;
  int64_t n;
  bool meets(const Words& o) const {
    return n > 0 && o.n > 0 && (const uint8_t*)p < (const uint8_t*)o.p + 4 * o.n && (const uint8_t*)o.p < (const uint8_t*)p + 4 * n;
  }
};
bool apart(const Words* out, int n_out, const Words* in, int n_in) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (out[o].meets(in[i])) return false;
    for (int other = 0; other < o; ++other)
      if (out[o].meets(out[other])) return false;
  }
  return true;
}

// The pools' pointers, and what they take up: codes and scales of K, of V.
sparsp_status_t check_pools(const CacheDims& c, const void* kc, const float* ks, const void* vc, const float* vs, Words* pools) {
  CHECK_PTR(kc);
  CHECK_PTR(ks);
  CHECK_PTR(vc);
  CHECK_PTR(vs);
  const int64_t scales = (int64_t)c.blocks * c.heads, codes = scales * c.bt * c.d / 4;
  pools[0] = {kc, codes};
  pools[1] = {ks, scales};
  pools[2] = {vc, codes};
  pools[3] = {vs, scales};
  return SPARSP_OK;
}

sparsp_status_t check_attn(const sparsp_cache_t* cache, int32_t B, int32_t H, int64_t tokens, int32_t max_add,
                           int32_t max_blocks, CacheDims* c) {
  sparsp_status_t r = check_cache(cache, c);
  if (r == SPARSP_OK) r = check_requests(*c, B, max_blocks, tokens);
  if (r != SPARSP_OK) return r;
  if (H <= 0 || H % c->heads != 0 || max_add < 1) return SPARSP_ERR_SHAPE;
  if (tokens * H > INT32_MAX || (int64_t)max_add * (H / c->heads) > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;
  return SPARSP_OK;
}

}  // namespace

extern "C" {

sparsp_status_t sparsp_cache_extend(const sparsp_cache_t* cache, int32_t B, int32_t max_blocks, const int32_t* len,
                                    const int32_t* add, const int32_t* free_blocks, int32_t n_free,
                                    const int32_t* used, int32_t* table, int32_t* len_out, int32_t* start,
                                    int32_t* slots, int64_t tokens, int32_t* used_out, int32_t* d_status,
                                    sparsp_stream_t stream) {
  CacheDims c;
  sparsp_status_t r = check_cache(cache, &c);
  if (r == SPARSP_OK) r = check_requests(c, B, max_blocks, tokens);
  if (r != SPARSP_OK) return r;
  if (n_free < 0) return SPARSP_ERR_SHAPE;
  CHECK_PTR(len);
  CHECK_PTR(add);
  if (n_free > 0) {   // may start anywhere in a longer list
    if (free_blocks == nullptr) return SPARSP_ERR_INVALID_ARG;
    if ((uintptr_t)free_blocks % 4 != 0) return SPARSP_ERR_ALIGN;
  }
  CHECK_OPT_PTR(used);
  CHECK_PTR(table);
  CHECK_PTR(len_out);
  CHECK_PTR(start);
  if (tokens > 0) CHECK_PTR(slots);
  CHECK_OPT_PTR(used_out);
  CHECK_OPT_PTR(d_status);
  // len_out may be len and used_out used; nothing else that is written may be read or written elsewhere
  const Words in[] = {{len, B}, {add, B}, {free_blocks, n_free}, {used, used != nullptr}};
  const Words out[] = {{len_out, B}, {used_out, used_out != nullptr}, {start, (int64_t)B + 1}, {slots, tokens},
                       {table, (int64_t)B * max_blocks}};
  for (int o = 0; o < 5; ++o) {
    for (const Words& i : in)
      if (out[o].meets(i) && !(out[o].p == i.p && (out[o].p == len_out ? i.p == len : out[o].p == used_out && i.p == used)))
        return SPARSP_ERR_INVALID_ARG;
    for (int other = 0; other < o; ++other)
      if (out[o].meets(out[other])) return SPARSP_ERR_INVALID_ARG;
  }
  CacheExtend a{B, max_blocks, n_free, (int)tokens, len, add, free_blocks, used, table, len_out, start, slots, used_out};
  return launch_cache_extend(c, a, d_status, (cudaStream_t)stream);
}

sparsp_status_t sparsp_cache_write(const sparsp_cache_t* cache, int32_t dtype, const void* k, int64_t k_stride,
                                   int64_t k_head, const void* v, int64_t v_stride, int64_t v_head,
                                   const int32_t* slots, int64_t tokens, void* kc, float* ks, void* vc, float* vs,
                                   int32_t* d_status, sparsp_stream_t stream) {
  CacheDims c;
  sparsp_status_t r = check_cache(cache, &c);
  if (r != SPARSP_OK) return r;
  if (tokens < 0) return SPARSP_ERR_SHAPE;
  if (tokens > INT32_MAX || (dtype != SPARSP_F32 && dtype != SPARSP_BF16)) return SPARSP_ERR_UNSUPPORTED;
  if (tokens > 0) {
    CHECK_PTR(k);
    CHECK_PTR(v);
    CHECK_PTR(slots);
  }
  const int elem = dtype == SPARSP_F32 ? 4 : 2;
  Words pools[4];
  r = check_strides(c, elem, tokens, &k_stride, &k_head);
  if (r == SPARSP_OK) r = check_strides(c, elem, tokens, &v_stride, &v_head);
  if (r == SPARSP_OK) r = check_pools(c, kc, ks, vc, vs, pools);
  if (r != SPARSP_OK) return r;
  CHECK_OPT_PTR(d_status);
  auto rows = [&](const void* p, int64_t token, int64_t head) {
    return Words{p, tokens == 0 ? 0 : ((tokens - 1) * token + (c.heads - 1) * head + c.d) * elem / 4};
  };
  const Words in[] = {rows(k, k_stride, k_head), rows(v, v_stride, v_head), {slots, tokens}};
  if (!apart(pools, 4, in, 3)) return SPARSP_ERR_INVALID_ARG;
  CacheWrite a{k, v, k_stride, k_head, v_stride, v_head, slots, (int)tokens, (uint8_t*)kc, (uint8_t*)vc, ks, vs};
  return launch_cache_write(c, dtype, a, d_status, (cudaStream_t)stream);
}

size_t sparsp_attn_cache_workspace_size(const sparsp_cache_t* cache, int32_t B, int32_t H, int64_t tokens,
                                        int32_t max_add, int32_t max_blocks) {
  CacheDims c;
  if (check_attn(cache, B, H, tokens, max_add, max_blocks, &c) != SPARSP_OK) return 0;
  return attn_cache_ws(c, H / c.heads, max_add);
}

sparsp_status_t sparsp_attn_cache_fwd(const sparsp_cache_t* cache, int32_t B, int32_t H, const void* q,
                                      int64_t q_stride, const int32_t* start, int64_t tokens, int32_t max_add,
                                      const int32_t* len, const int32_t* table, int32_t max_blocks, const void* kc,
                                      const float* ks, const void* vc, const float* vs, const int32_t* row_ptr,
                                      const int32_t* col_idx, int64_t col_cap, float scale, uint32_t flags, void* o,
                                      float* lse, void* ws, size_t ws_bytes, int32_t* d_status,
                                      sparsp_stream_t stream) {
  CacheAttn a{};
  sparsp_status_t r = check_attn(cache, B, H, tokens, max_add, max_blocks, &a.c);
  if (r != SPARSP_OK) return r;
  if ((flags & ~SPARSP_CACHE_CAUSAL) || isnan(scale) || isinf(scale)) return SPARSP_ERR_INVALID_ARG;
  const int64_t row = (int64_t)H * a.c.d;
  if (q_stride == 0) q_stride = row;
  if (q_stride < row || q_stride > (int64_t)1 << 31) return SPARSP_ERR_SHAPE;
  if (q_stride % 8 != 0) return SPARSP_ERR_ALIGN;
  if (tokens > 0) {
    CHECK_PTR(q);
    CHECK_PTR(o);
    CHECK_PTR(lse);
  }
  CHECK_PTR(start);
  CHECK_PTR(len);
  CHECK_PTR(table);
  Words in[10];   // what is read
  r = check_pools(a.c, kc, ks, vc, vs, in);
  if (r != SPARSP_OK) return r;
  if ((row_ptr == nullptr) != (col_idx == nullptr) || col_cap < 0) return SPARSP_ERR_INVALID_ARG;
  CHECK_OPT_PTR(row_ptr);
  CHECK_OPT_PTR(col_idx);
  CHECK_OPT_PTR(d_status);
  CHECK_PTR(ws);
  if (ws_bytes < attn_cache_ws(a.c, H / a.c.heads, max_add)) return SPARSP_ERR_WORKSPACE;
  if (tokens == 0) return SPARSP_OK;
  in[4] = {q, ((tokens - 1) * q_stride + row) / 2};   // (row is even)
  in[5] = {start, (int64_t)B + 1};
  in[6] = {len, B};
  in[7] = {table, (int64_t)B * max_blocks};
  in[8] = {row_ptr, row_ptr != nullptr ? (int64_t)B * a.c.heads + 1 : 0};
  in[9] = {col_idx, col_idx != nullptr ? (col_cap < (int64_t)1 << 60 ? col_cap : (int64_t)1 << 60) : 0};
  const Words out[] = {{o, tokens * row / 2}, {lse, tokens * H}};
  if (!apart(out, 2, in, 10)) return SPARSP_ERR_INVALID_ARG;
  a.B = B;
  a.H = H;
  a.group = H / a.c.heads;
  a.max_blocks = max_blocks;
  a.tokens = (int)tokens;
  a.max_add = max_add;
  a.q = (const __nv_bfloat16*)q;
  a.q_token = q_stride;
  a.start = start;
  a.len = len;
  a.table = table;
  a.kc = (const uint8_t*)kc;
  a.vc = (const uint8_t*)vc;
  a.ks = ks;
  a.vs = vs;
  a.row_ptr = row_ptr;
  a.col_idx = col_idx;
  a.col_cap = col_cap;
  a.scale_log2 = (scale <= 0.f ? 1.0f / sqrtf((float)a.c.d) : scale) * 1.4426950408889634f;
  a.causal = (flags & SPARSP_CACHE_CAUSAL) != 0;
  a.o = (__nv_bfloat16*)o;
  a.lse = lse;
  a.d_status = d_status;
  return launch_attn_cache(a, ws, (cudaStream_t)stream);
}

}  // extern "C"
