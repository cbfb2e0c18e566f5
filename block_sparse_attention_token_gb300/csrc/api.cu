// extern "C" entry points of libsparsp: argument validation (before any CUDA
// call, so host errors leave outputs untouched) and dispatch to launchers.
#include <math.h>

#include "common.cuh"
#include "mask.cuh"

using namespace sparsp;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Validates the shape and fills Dims. Accepts d in {64,128}, Bt in {64,128},
// nb <= kMaxBlocks, B*H <= 65535.
sparsp_status_t check_shape(const sparsp_shape_t* sh, Dims* s) {
  if (sh == nullptr) return SPARSP_ERR_INVALID_ARG;
  if (sh->B <= 0 || sh->H <= 0 || sh->T <= 0 || sh->Y <= 0 || sh->X <= 0 || sh->d <= 0 ||
      sh->ta <= 0 || sh->tb <= 0 || sh->tc <= 0)
    return SPARSP_ERR_SHAPE;
  if (sh->dtype != SPARSP_F32 && sh->dtype != SPARSP_BF16) return SPARSP_ERR_UNSUPPORTED;
  if (sh->T % sh->ta || sh->Y % sh->tb || sh->X % sh->tc) return SPARSP_ERR_SHAPE;
  if (sh->d != 64 && sh->d != 128) return SPARSP_ERR_UNSUPPORTED;
  const int64_t Bt = (int64_t)sh->ta * sh->tb * sh->tc;
  if (Bt != 64 && Bt != 128) return SPARSP_ERR_UNSUPPORTED;
  const int64_t nT = sh->T / sh->ta, nY = sh->Y / sh->tb, nX = sh->X / sh->tc;
  const int64_t nb = nT * nY * nX;
  if (nb > kMaxBlocks) return SPARSP_ERR_UNSUPPORTED;
  if ((int64_t)sh->B * sh->H > 65535) return SPARSP_ERR_UNSUPPORTED;
  // int32 CSR offsets must hold B*H*nb*nb entries
  if ((int64_t)sh->B * sh->H * nb * nb > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;
  s->B = sh->B; s->H = sh->H; s->T = sh->T; s->Y = sh->Y; s->X = sh->X; s->d = sh->d;
  s->ta = sh->ta; s->tb = sh->tb; s->tc = sh->tc; s->dtype = sh->dtype;
  s->N = (int64_t)sh->T * sh->Y * sh->X;
  s->Bt = (int)Bt;
  s->nb = (int)nb;
  s->nT = (int)nT; s->nY = (int)nY; s->nX = (int)nX;
  s->elem = sh->dtype == SPARSP_F32 ? 4 : 2;
  return SPARSP_OK;
}

#define CHECK_PTR(p)                                   \
  do {                                                 \
    if ((p) == nullptr) return SPARSP_ERR_INVALID_ARG; \
    if (!aligned16(p)) return SPARSP_ERR_ALIGN;        \
  } while (0)

#define CHECK_OPT_PTR(p)                                        \
  do {                                                          \
    if ((p) != nullptr && !aligned16(p)) return SPARSP_ERR_ALIGN; \
  } while (0)

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Every attention option bit; a call ignores the ones that do not concern it.
constexpr uint32_t kKnownFlags = SPARSP_SCHED_FLAT | SPARSP_KERNEL_PORTABLE | SPARSP_BWD_SPLIT_KV |
                                 SPARSP_OUT_RASTER | SPARSP_IN_RASTER | SPARSP_LISTS_SEEN | SPARSP_GRID_CAP_MASK;

// Attention workspace layout: items, counter(s), then backward extras.
struct AttnWs {
  int32_t* items;      // [rows]
  int32_t* counter;    // [4]
  int32_t* hist;       // [B*H*(2nb+1)] flat-order scratch
  int32_t* pair_ptr;   // [B*H*ceil(nb/2)+1] row offsets of query-block pairs (64-token blocks)
  // backward only
  int32_t* col_ptr;    // [rows+1]
  int32_t* row_idx;    // [B*H*nb*nb]
  int32_t* items2;     // [rows] order over CSC columns
  float* delta;        // [B*H*N]
  float* lse2;         // [B*H*N] LSE * log2(e)
  // token masks only: the CSR of the block pairs that see something
  int32_t* seen_ptr;   // [rows+1]
  int32_t* seen_idx;   // [B*H*nb*nb]
  // masked forward only: items for the general kernel, [rows] and [rows + 2]
  int32_t* fix_items;
  int32_t* fix_mark;   // marks, then count and pull counter
  size_t bytes;
};

AttnWs attn_ws_layout(const Dims& s, bool backward, void* base, bool masked = false) {
  AttnWs w{};
  uint8_t* p = (uint8_t*)base;
  size_t off = 0;
  auto take = [&](size_t n) {
    uint8_t* r = p ? p + off : nullptr;
    off += align256(n);
    return r;
  };
  const size_t rows = (size_t)s.rows();
  w.items = (int32_t*)take(rows * 4);
  w.counter = (int32_t*)take(16);
  w.hist = (int32_t*)take(lpt_ws(s));
  w.pair_ptr = (int32_t*)take(((size_t)s.B * s.H * ((s.nb + 1) / 2) + 1) * 4);
  if (backward) {
    w.col_ptr = (int32_t*)take((rows + 1) * 4);
    w.row_idx = (int32_t*)take(rows * (size_t)s.nb * 4);
    w.items2 = (int32_t*)take(rows * 4);
    w.delta = (float*)take((size_t)s.B * s.H * s.N * 4);
    w.lse2 = (float*)take((size_t)s.B * s.H * s.N * 4);
  }
  if (masked) {
    w.seen_ptr = (int32_t*)take((rows + 1) * 4);
    w.seen_idx = (int32_t*)take(rows * (size_t)s.nb * 4);
    w.fix_items = (int32_t*)take(rows * 4);
    w.fix_mark = (int32_t*)take((rows + 2) * 4);
  }
  w.bytes = off;
  return w;
}

// A raster tensor's token stride: 0 means contiguous; else at least H*d
// elements and a multiple of 16 bytes.
sparsp_status_t check_stride(const Dims& s, int64_t* stride) {
  const int64_t hd = (int64_t)s.H * s.d;
  if (*stride == 0) *stride = hd;
  if (*stride < hd || *stride > INT64_MAX / 8 / (s.B * s.N)) return SPARSP_ERR_SHAPE;
  if (*stride * s.elem % 16 != 0) return SPARSP_ERR_ALIGN;
  return SPARSP_OK;
}

// Do the byte ranges of two raster tensors with these token strides overlap?
bool overlap(const Dims& s, const void* a, int64_t a_stride, const void* b, int64_t b_stride) {
  const int64_t last = (int64_t)s.B * s.N - 1, hd = (int64_t)s.H * s.d;
  const uint8_t *pa = (const uint8_t*)a, *pb = (const uint8_t*)b;
  return pa < pb + (last * b_stride + hd) * s.elem && pb < pa + (last * a_stride + hd) * s.elem;
}

constexpr int kNormMaxCols = 16384;

sparsp_status_t check_norm(const sparsp_shape_t* shape, uint32_t flags, Dims* s) {
  const sparsp_status_t r = check_shape(shape, s);
  if (r != SPARSP_OK) return r;
  if (flags & ~(SPARSP_NORM_RMS | SPARSP_NORM_HEAD)) return SPARSP_ERR_INVALID_ARG;
  if (!(flags & SPARSP_NORM_HEAD) && (int64_t)s->H * s->d > kNormMaxCols) return SPARSP_ERR_UNSUPPORTED;
  return SPARSP_OK;
}

// Axes of a rotary table: even column counts, at least one position per axis.
sparsp_status_t check_rope(const sparsp_rope_t* r) {
  if (r == nullptr) return SPARSP_ERR_INVALID_ARG;
  for (int ax = 0; ax < 3; ++ax)
    if (r->cols[ax] < 0 || r->cols[ax] % 2 || r->cols[ax] > 128 || r->extent[ax] < 1) return SPARSP_ERR_SHAPE;
  if (rope_table_entries(*r) > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;
  return SPARSP_OK;
}

// A score cap: none, or one whose ratio to the scale fp32 holds well.
bool cap_ok(float cap, float scale, int d) {
  if (cap == 0.f) return true;
  if (!(cap >= 9.5367431640625e-7f && cap <= 1048576.f)) return false;   // 2^-20 .. 2^20
  const float x = (scale <= 0.f ? 1.0f / sqrtf((float)d) : scale) / cap;
  return isnormal(x) && isfinite(x * 4.f);
}

// Is it worth dropping the block pairs that see nothing of each other before the
// work is ordered? The three launches cost 12 us; a stage of the attention kernel that turns
// out empty costs it little. By the stages of the busiest SM, if every block were
// selected: up to 128 of them lists without regard to the mask (60% of all blocks, three
// documents) take the forward 5 to 14 us longer with the launches (1 to 16 heads, 1,024 to
// 4,096 tokens: 27 -> 40 us ... 98 -> 111; backward 64 -> 76 ... 306 -> 318, but 182 -> 155 with
// 128-token blocks and 64 stages), from 384 on such lists gain (8,192 tokens, 12 heads: forward
// 212 -> 183 and 186 -> 129 us, backward 708 -> 575 and 774 -> 466) and lists selected by masked
// scores lose the 12 us (145 -> 157).
bool drops_unseen(const Dims& s, int items_per_head) {
  const int sms = device_sm_count();
  const int64_t items = (int64_t)s.B * s.H * items_per_head, per_sm = (items + sms - 1) / (sms > 0 ? sms : 1);
  return sms <= 0 || per_sm * items_per_head > 128;
}

// What an attention call launches, decided in one place for the call and for
// sparsp_attn_launches.
struct AttnSteps {
  bool tc;          // the tcgen05 kernels
  bool masked;      // a token mask or a cap
  bool compacts;    // three launches that drop the pairs that see nothing of each other
  bool one_order;   // the work is ordered by one launch (order_items)
  bool pairs;       // items are pairs of 64-token blocks, whose costs take a launch first
  bool flat;        // SPARSP_SCHED_FLAT
  bool twice;       // forward: the general kernel follows over the items passed on to it
  int per_head;     // items per head
  int order_launches() const { return one_order ? 1 : (pairs ? 1 : 0) + (flat ? 2 : 1); }
};
AttnSteps attn_steps(const Dims& s, uint32_t flags, bool plan, float cap, bool backward) {
  AttnSteps a{};
  a.tc = s.dtype == SPARSP_BF16 && !(flags & SPARSP_KERNEL_PORTABLE) &&
         (backward ? attn_bwd_tc_supported(s) : attn_fwd_tc_supported(s));
  a.masked = plan || cap > 0.f;
  a.per_head = !a.tc ? s.nb : backward ? attn_bwd_tc_items_per_head(s) : attn_fwd_tc_items_per_head(s);
  a.compacts = plan && !(flags & SPARSP_LISTS_SEEN) && drops_unseen(s, a.per_head);
  a.one_order = a.masked && order_items_fits(s, a.per_head, plan);
  a.pairs = a.per_head != s.nb;
  a.flat = (flags & SPARSP_SCHED_FLAT) != 0;
  a.twice = a.masked && !(cap > 0.f && cap <= kFixedCap);
  return a;
}

// sparsp_attn_fwd, and sparsp_attn_masked_fwd with `masked`: both validate alike;
// a masked call without plan and cap is the plain one.
sparsp_status_t attn_fwd(const sparsp_shape_t* shape, const void* q, const void* k, const void* v,
                         const int32_t* row_ptr, const int32_t* col_idx, float scale, bool masked, float cap,
                         const void* plan, void* o, float* lse, void* ws, size_t ws_bytes, uint32_t flags,
                         uint64_t* prof, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (isnan(scale) || isinf(scale)) return SPARSP_ERR_INVALID_ARG;
  if (flags & ~kKnownFlags) return SPARSP_ERR_INVALID_ARG;
  s.max_ctas = (int)((flags & SPARSP_GRID_CAP_MASK) >> SPARSP_GRID_CAP_SHIFT);
  CHECK_PTR(q);
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(o);
  CHECK_PTR(lse);
  CHECK_PTR(ws);
  CHECK_OPT_PTR(prof);
  CHECK_OPT_PTR(d_status);
  CHECK_OPT_PTR(plan);
  if (!cap_ok(cap, scale, s.d)) return SPARSP_ERR_INVALID_ARG;
  AttnWs w = attn_ws_layout(s, false, ws, masked);
  if (ws_bytes < w.bytes) return SPARSP_ERR_WORKSPACE;
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)s.d);
  const AttnSteps steps = attn_steps(s, flags, plan != nullptr, cap, false);
  const bool tc = steps.tc;
  const bool raster = (flags & SPARSP_OUT_RASTER) != 0;
  const bool in_raster = (flags & SPARSP_IN_RASTER) != 0;
  if ((raster || in_raster) && !tc) return SPARSP_ERR_UNSUPPORTED;   // only the tcgen05 kernel reads or writes raster rows
  if (masked && !tc) return SPARSP_ERR_UNSUPPORTED;
  masked = steps.masked;
  cudaStream_t st = (cudaStream_t)stream;
  const MaskView mask = mask_view(s, plan);
  if (steps.compacts) {
    r = launch_mask_csr(s, mask, row_ptr, col_idx, w.seen_ptr, w.seen_idx, d_status, st);
    if (r != SPARSP_OK) return r;
    row_ptr = w.seen_ptr;
    col_idx = w.seen_idx;
  }
  const bool flat = steps.flat;
  // the general kernel's list of a masked call: marks, then count and pull counter, in one stretch
  const int64_t masked_items = masked ? (int64_t)s.B * s.H * steps.per_head : 0;
  const int64_t cleared = steps.twice ? masked_items + 2 : 0;
  if (steps.one_order) {
    r = launch_order_items(s, steps.per_head, row_ptr, w.items, w.counter, w.fix_mark, (int)cleared, st);
  } else if (cleared > 0 && cudaMemsetAsync(w.fix_mark, 0, cleared * sizeof(int32_t), st) != cudaSuccess) {
    return SPARSP_ERR_CUDA;
  } else if (steps.pairs) {
    // the tcgen05 kernel's items are pairs of query blocks: order the pairs,
    // each costing the sum of its two rows
    r = launch_pair_ptr(s, row_ptr, w.pair_ptr, st);
    if (r != SPARSP_OK) return r;
    Dims sp = s;
    sp.nb = steps.per_head;
    r = launch_lpt(sp, w.pair_ptr, flat, w.items, w.counter, w.hist, st, 2 * s.nb);
  } else {
    r = launch_lpt(s, row_ptr, flat, w.items, w.counter, w.hist, st);
  }
  if (r != SPARSP_OK) return r;
  if (s.dtype == SPARSP_F32)
    return launch_attn_fwd_f32(s, (const float*)q, (const float*)k, (const float*)v, row_ptr,
                               col_idx, scale, (float*)o, lse, w.items, w.counter, prof, d_status,
                               st);
  if (masked) {
    const FixList fix{w.fix_items, w.fix_mark, w.fix_mark + masked_items, w.fix_mark + masked_items + 1};
    return launch_attn_fwd_masked(s, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v,
                                  row_ptr, col_idx, scale, cap, mask, (__nv_bfloat16*)o, lse, raster, in_raster,
                                  w.items, w.counter, fix, prof, d_status, st);
  }
  if (tc)
    return launch_attn_fwd_tc(s, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k,
                              (const __nv_bfloat16*)v, row_ptr, col_idx, scale,
                              (__nv_bfloat16*)o, lse, raster, in_raster, w.items, w.counter, prof, d_status, st);
  return launch_attn_fwd_mma(s, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k,
                             (const __nv_bfloat16*)v, row_ptr, col_idx, scale, (__nv_bfloat16*)o,
                             lse, w.items, w.counter, prof, d_status, st);
}

// sparsp_attn_bwd, and sparsp_attn_masked_bwd with `masked`.
sparsp_status_t attn_bwd(const sparsp_shape_t* shape, const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dout, const int32_t* row_ptr, const int32_t* col_idx,
                         float scale, bool masked, float cap, const void* plan, void* dq, void* dk, void* dv, void* ws,
                         size_t ws_bytes, uint32_t flags, uint64_t* prof, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (s.dtype != SPARSP_BF16) return SPARSP_ERR_UNSUPPORTED;
  if (isnan(scale) || isinf(scale)) return SPARSP_ERR_INVALID_ARG;
  if (flags & ~kKnownFlags) return SPARSP_ERR_INVALID_ARG;
  if (flags & SPARSP_IN_RASTER) return SPARSP_ERR_UNSUPPORTED;   // the backward reads block-ordered tiles
  s.max_ctas = (int)((flags & SPARSP_GRID_CAP_MASK) >> SPARSP_GRID_CAP_SHIFT);
  CHECK_PTR(q);
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK_PTR(o);
  CHECK_PTR(lse);
  CHECK_PTR(dout);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(dq);
  CHECK_PTR(dk);
  CHECK_PTR(dv);
  CHECK_PTR(ws);
  CHECK_OPT_PTR(prof);
  CHECK_OPT_PTR(d_status);
  CHECK_OPT_PTR(plan);
  if (!cap_ok(cap, scale, s.d)) return SPARSP_ERR_INVALID_ARG;
  AttnWs w = attn_ws_layout(s, true, ws, masked);
  if (ws_bytes < w.bytes) return SPARSP_ERR_WORKSPACE;
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)s.d);
  cudaStream_t st = (cudaStream_t)stream;
  typedef const __nv_bfloat16* cb;
  const AttnSteps steps = attn_steps(s, flags, plan != nullptr, cap, true);
  const bool tc = steps.tc, flat = steps.flat;
  const bool raster = (flags & SPARSP_OUT_RASTER) != 0;
  if (raster && !tc) return SPARSP_ERR_UNSUPPORTED;   // only the tcgen05 kernels write raster rows
  if (masked && !tc) return SPARSP_ERR_UNSUPPORTED;
  masked = steps.masked;
  const MaskView mask = mask_view(s, plan);
  if (steps.compacts) {
    r = launch_mask_csr(s, mask, row_ptr, col_idx, w.seen_ptr, w.seen_idx, d_status, st);
    if (r != SPARSP_OK) return r;
    row_ptr = w.seen_ptr;
    col_idx = w.seen_idx;
  }
  r = launch_bwd_rowdot(s, (cb)o, (cb)dout, w.delta, lse, tc ? w.lse2 : nullptr, raster, st);
  if (r != SPARSP_OK) return r;
  r = launch_csr_transpose(s, row_ptr, col_idx, w.col_ptr, w.row_idx, d_status, st);
  if (r != SPARSP_OK) return r;
  // the tcgen05 kernels' items with 64-token blocks are pairs of blocks, each
  // costing the sum of its two lists (CSR rows for dQ, CSC columns for dK/dV)
  const bool pairs = steps.pairs;
  Dims sp = s;
  sp.nb = steps.per_head;
  if (steps.one_order) {
    r = launch_order_items(s, sp.nb, row_ptr, w.items, w.counter, nullptr, 0, st);
  } else if (pairs) {
    r = launch_pair_ptr(s, row_ptr, w.pair_ptr, st);
    if (r != SPARSP_OK) return r;
    r = launch_lpt(sp, w.pair_ptr, flat, w.items, w.counter, w.hist, st, 2 * s.nb);
  } else {
    r = launch_lpt(s, row_ptr, flat, w.items, w.counter, w.hist, st);
  }
  if (r != SPARSP_OK) return r;
  if (tc) {
    r = masked ? launch_attn_bwd_masked(s, 0, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, row_ptr, col_idx, scale,
                                        (__nv_bfloat16*)dq, nullptr, w.items, w.counter, prof, d_status, raster, mask,
                                        cap, st)
               : launch_attn_bwd_tc(s, 0, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, row_ptr, col_idx, scale,
                                    (__nv_bfloat16*)dq, nullptr, w.items, w.counter, prof, d_status, raster, st);
    if (r != SPARSP_OK) return r;
    if (steps.one_order) {
      r = launch_order_items(s, sp.nb, w.col_ptr, w.items2, w.counter + 1, nullptr, 0, st);
    } else if (pairs) {   // pair_ptr is free again: the dQ kernel reads only its item list
      r = launch_pair_ptr(s, w.col_ptr, w.pair_ptr, st);
      if (r != SPARSP_OK) return r;
      r = launch_lpt(sp, w.pair_ptr, flat, w.items2, w.counter + 1, w.hist, st, 2 * s.nb);
    } else {
      r = launch_lpt(s, w.col_ptr, flat, w.items2, w.counter + 1, w.hist, st);
    }
    if (r != SPARSP_OK) return r;
    if (masked)
      return launch_attn_bwd_masked(s, 3, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, w.col_ptr, w.row_idx, scale,
                                    (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, w.items2, w.counter + 1, prof, d_status,
                                    raster, mask, cap, st);
    if (!(flags & SPARSP_BWD_SPLIT_KV))
      return launch_attn_bwd_tc(s, 3, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, w.col_ptr, w.row_idx,
                                scale, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, w.items2, w.counter + 1, prof,
                                d_status, raster, st);
    r = launch_attn_bwd_tc(s, 1, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, w.col_ptr, w.row_idx,
                           scale, (__nv_bfloat16*)dk, nullptr, w.items2, w.counter + 1, prof, d_status, raster,
                           st);
    if (r != SPARSP_OK) return r;
    if (cudaMemsetAsync(w.counter + 2, 0, sizeof(int32_t), st) != cudaSuccess) return SPARSP_ERR_CUDA;
    return launch_attn_bwd_tc(s, 2, (cb)q, (cb)k, (cb)v, (cb)dout, w.lse2, w.delta, w.col_ptr, w.row_idx,
                              scale, (__nv_bfloat16*)dv, nullptr, w.items2, w.counter + 2, prof, d_status, raster,
                              st);
  }
  r = launch_attn_bwd_dq(s, (cb)q, (cb)k, (cb)v, (cb)dout, lse, w.delta, row_ptr, col_idx, scale,
                         (__nv_bfloat16*)dq, w.items, w.counter, prof, d_status, st);
  if (r != SPARSP_OK) return r;
  r = launch_lpt(s, w.col_ptr, flat, w.items2, w.counter + 1, w.hist, st);
  if (r != SPARSP_OK) return r;
  return launch_attn_bwd_dkdv(s, (cb)q, (cb)k, (cb)v, (cb)dout, lse, w.delta, w.col_ptr,
                              w.row_idx, scale, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, w.items2,
                              w.counter + 1, prof, d_status, st);
}

}  // namespace

extern "C" {

const char* sparsp_status_string(int32_t st) {
  switch (st) {
    case SPARSP_OK: return "SPARSP_OK";
    case SPARSP_ERR_INVALID_ARG: return "SPARSP_ERR_INVALID_ARG";
    case SPARSP_ERR_UNSUPPORTED: return "SPARSP_ERR_UNSUPPORTED";
    case SPARSP_ERR_SHAPE: return "SPARSP_ERR_SHAPE";
    case SPARSP_ERR_ALIGN: return "SPARSP_ERR_ALIGN";
    case SPARSP_ERR_WORKSPACE: return "SPARSP_ERR_WORKSPACE";
    case SPARSP_ERR_CAPACITY: return "SPARSP_ERR_CAPACITY";
    case SPARSP_ERR_DATA: return "SPARSP_ERR_DATA";
    case SPARSP_ERR_CUDA: return "SPARSP_ERR_CUDA";
    case SPARSP_ERR_TIMEOUT: return "SPARSP_ERR_TIMEOUT";
    default: return "SPARSP_ERR_UNKNOWN";
  }
}

int32_t sparsp_version(void) { return SPARSP_VERSION; }

int32_t sparsp_device_sm_count(void) { return device_sm_count(); }

sparsp_status_t sparsp_reorder(const sparsp_shape_t* shape, const void* in, void* out,
                               int32_t inverse, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(in);
  CHECK_PTR(out);
  const size_t bytes = (size_t)s.B * s.H * s.N * s.d * s.elem;
  const uint8_t* a = (const uint8_t*)in;
  const uint8_t* b = (const uint8_t*)out;
  if (a < b + bytes && b < a + bytes) return SPARSP_ERR_INVALID_ARG;   // overlap
  return launch_reorder(s, in, out, inverse != 0, (cudaStream_t)stream);
}

sparsp_status_t sparsp_reorder_pool(const sparsp_shape_t* shape, const void* in, void* out,
                                    float* means, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(in);
  CHECK_OPT_PTR(out);
  CHECK_PTR(means);
  const size_t bytes = (size_t)s.B * s.H * s.N * s.d * s.elem;
  const uint8_t* a = (const uint8_t*)in;
  const uint8_t* b = (const uint8_t*)out;
  if (b != nullptr && a < b + bytes && b < a + bytes) return SPARSP_ERR_INVALID_ARG;   // overlap
  return launch_reorder(s, in, out, false, (cudaStream_t)stream, means);
}

size_t sparsp_block_scores_pooled_workspace_size(const sparsp_shape_t* shape, int32_t estimator,
                                                 int32_t rank) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  if (estimator == SPARSP_EST_LOWRANK && (rank < 1 || rank > 64)) return 0;
  return scores_from_means_ws(s, estimator, rank);
}

sparsp_status_t sparsp_block_scores_pooled(const sparsp_shape_t* shape, int32_t estimator,
                                           const float* qmeans, const float* kmeans,
                                           const float* wq, const float* wk, int32_t rank,
                                           float* scores, void* ws, size_t ws_bytes,
                                           sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (estimator != SPARSP_EST_MEAN && estimator != SPARSP_EST_LOWRANK)
    return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(qmeans);
  CHECK_PTR(kmeans);
  CHECK_PTR(scores);
  if (estimator == SPARSP_EST_LOWRANK) {
    if (rank < 1 || rank > 64) return SPARSP_ERR_UNSUPPORTED;
    CHECK_PTR(wq);
    CHECK_PTR(wk);
    CHECK_PTR(ws);
    if (ws_bytes < scores_from_means_ws(s, estimator, rank)) return SPARSP_ERR_WORKSPACE;
  }
  return launch_scores_from_means(s, estimator, qmeans, kmeans, wq, wk, rank, scores, ws,
                                  (cudaStream_t)stream);
}

size_t sparsp_block_scores_workspace_size(const sparsp_shape_t* shape, int32_t estimator,
                                          int32_t rank) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  if (estimator == SPARSP_EST_LOWRANK && (rank < 1 || rank > 64)) return 0;
  return block_scores_ws(s, estimator, rank);
}

sparsp_status_t sparsp_block_scores(const sparsp_shape_t* shape, int32_t estimator,
                                    const void* q, const void* k, const float* wq,
                                    const float* wk, int32_t rank, float* scores, void* ws,
                                    size_t ws_bytes, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (estimator != SPARSP_EST_MEAN && estimator != SPARSP_EST_LOWRANK)
    return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(q);
  CHECK_PTR(k);
  CHECK_PTR(scores);
  CHECK_PTR(ws);
  if (estimator == SPARSP_EST_LOWRANK) {
    if (rank < 1 || rank > 64) return SPARSP_ERR_UNSUPPORTED;
    CHECK_PTR(wq);
    CHECK_PTR(wk);
  }
  if (ws_bytes < block_scores_ws(s, estimator, rank)) return SPARSP_ERR_WORKSPACE;
  return launch_block_scores(s, estimator, q, k, wq, wk, rank, scores, ws, (cudaStream_t)stream);
}

size_t sparsp_select_workspace_size(const sparsp_shape_t* shape) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return select_ws(s);
}

sparsp_status_t sparsp_select(const sparsp_shape_t* shape, const float* scores, float top_p,
                              int32_t k_floor, int32_t* row_ptr, int32_t* col_idx, void* ws,
                              size_t ws_bytes, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (isnan(top_p)) return SPARSP_ERR_INVALID_ARG;
  if (k_floor < 0) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(scores);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(ws);
  CHECK_OPT_PTR(d_status);
  if (ws_bytes < select_ws(s)) return SPARSP_ERR_WORKSPACE;
  return launch_select(s, scores, top_p, k_floor, row_ptr, col_idx, ws, d_status,
                       (cudaStream_t)stream);
}

sparsp_status_t sparsp_select_noalloc(const sparsp_shape_t* shape, const float* scores, float top_p,
                                      int32_t k_floor, int32_t* row_ptr, int32_t* col_idx,
                                      int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (isnan(top_p)) return SPARSP_ERR_INVALID_ARG;
  if (k_floor < 0) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(scores);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_OPT_PTR(d_status);
  if (s.rows() > kSelectNoAllocMaxRows) return SPARSP_ERR_WORKSPACE;
  return launch_select_noalloc(s, scores, top_p, k_floor, row_ptr, col_idx, d_status,
                               (cudaStream_t)stream);
}

sparsp_status_t sparsp_kv_demand(const sparsp_shape_t* shape, int32_t P, const int32_t* row_ptr,
                                 const int32_t* col_idx, const int32_t* owner, uint32_t* bitmap,
                                 int32_t* dem_ptr, int32_t* dem_idx, const void* k, const void* v,
                                 void* kg, void* vg, int64_t gather_cap_blocks, uint64_t* bytes,
                                 int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (P < 1 || P > s.nb) return SPARSP_ERR_SHAPE;
  if ((int64_t)s.B * s.H * P * s.nb > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;   // int32 list offsets
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_OPT_PTR(owner);
  CHECK_PTR(bitmap);
  CHECK_PTR(dem_ptr);
  CHECK_PTR(dem_idx);
  CHECK_PTR(bytes);
  CHECK_OPT_PTR(d_status);
  if ((kg == nullptr) != (vg == nullptr)) return SPARSP_ERR_INVALID_ARG;
  if (kg != nullptr) {
    CHECK_PTR(kg);
    CHECK_PTR(vg);
    CHECK_PTR(k);
    CHECK_PTR(v);
    if (gather_cap_blocks < 0) return SPARSP_ERR_INVALID_ARG;
  }
  return launch_kv_demand(s, P, row_ptr, col_idx, owner, bitmap, dem_ptr, dem_idx, k, v, kg, vg,
                          gather_cap_blocks, bytes, d_status, (cudaStream_t)stream);
}

sparsp_status_t sparsp_kv_gather(const sparsp_shape_t* shape, int32_t P, const int32_t* dem_ptr,
                                 const int32_t* dem_idx, const void* k, const void* v, void* kg, void* vg,
                                 int64_t gather_cap_blocks, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (P < 1 || P > s.nb) return SPARSP_ERR_SHAPE;
  if ((int64_t)s.B * s.H * P * s.nb > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;   // int32 list offsets
  CHECK_PTR(dem_ptr);
  CHECK_PTR(dem_idx);
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK_PTR(kg);
  CHECK_PTR(vg);
  CHECK_OPT_PTR(d_status);
  if (gather_cap_blocks < 0) return SPARSP_ERR_INVALID_ARG;
  return launch_kv_gather(s, P, dem_ptr, dem_idx, k, v, kg, vg, gather_cap_blocks, d_status,
                          (cudaStream_t)stream);
}

sparsp_status_t sparsp_kv_gather_raster(const sparsp_shape_t* shape, int32_t P, const int32_t* dem_ptr,
                                        const int32_t* dem_idx, const void* k, const void* v, void* kg, void* vg,
                                        int64_t gather_cap_blocks, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (P < 1 || P > s.nb) return SPARSP_ERR_SHAPE;
  if ((int64_t)s.B * s.H * P * s.nb > INT32_MAX) return SPARSP_ERR_UNSUPPORTED;   // int32 list offsets
  CHECK_PTR(dem_ptr);
  CHECK_PTR(dem_idx);
  CHECK_PTR(k);
  CHECK_PTR(v);
  CHECK_PTR(kg);
  CHECK_PTR(vg);
  CHECK_OPT_PTR(d_status);
  if (gather_cap_blocks < 0) return SPARSP_ERR_INVALID_ARG;
  return launch_kv_gather_raster(s, P, dem_ptr, dem_idx, k, v, kg, vg, gather_cap_blocks, d_status,
                                 (cudaStream_t)stream);
}

size_t sparsp_placement_workspace_size(const sparsp_shape_t* shape) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK || s.nb > kMaxBlocksNext) return 0;
  return placement_ws(s);
}

sparsp_status_t sparsp_placement(const sparsp_shape_t* shape, int32_t P, const int32_t* row_ptr,
                                 const int32_t* col_idx, int32_t* owner, void* ws, size_t ws_bytes,
                                 int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (s.nb > kMaxBlocksNext) return SPARSP_ERR_UNSUPPORTED;
  if (P < 1 || P > s.nb) return SPARSP_ERR_SHAPE;
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(owner);
  CHECK_PTR(ws);
  CHECK_OPT_PTR(d_status);
  if (ws_bytes < placement_ws(s)) return SPARSP_ERR_WORKSPACE;
  return launch_placement(s, row_ptr, col_idx, P, owner, ws, d_status, (cudaStream_t)stream);
}

sparsp_status_t sparsp_balance_heads(const sparsp_shape_t* shape, int32_t P, int32_t max_migrations,
                                     const int32_t* row_ptr, int32_t* head_rank, int64_t* loads,
                                     int32_t* migrations, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (s.H > kBalanceMaxHeads) return SPARSP_ERR_UNSUPPORTED;
  if (P < 1 || P > s.H) return SPARSP_ERR_SHAPE;
  if (max_migrations < 0) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(row_ptr);
  CHECK_PTR(head_rank);
  CHECK_PTR(loads);
  CHECK_OPT_PTR(migrations);
  return launch_balance(s, row_ptr, P, max_migrations, head_rank, loads, migrations, (cudaStream_t)stream);
}

size_t sparsp_augment_workspace_size(const sparsp_shape_t* shape, int32_t P) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK || P < 1 || s.nb > kMaxBlocksNext) return 0;
  return augment_ws(s, P);
}

sparsp_status_t sparsp_augment(const sparsp_shape_t* shape, int32_t P, const float* scores,
                               const int32_t* row_ptr, const int32_t* col_idx, const int32_t* head_rank,
                               int32_t* row_ptr_out, int32_t* col_idx_out, int64_t col_cap, int64_t* added,
                               void* ws, size_t ws_bytes, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (s.H > kBalanceMaxHeads || s.nb > kMaxBlocksNext) return SPARSP_ERR_UNSUPPORTED;
  if (P < 1 || P > s.H) return SPARSP_ERR_SHAPE;
  if (col_cap < 0) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(scores);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(head_rank);
  CHECK_PTR(row_ptr_out);
  CHECK_PTR(col_idx_out);
  CHECK_OPT_PTR(added);
  CHECK_PTR(ws);
  CHECK_OPT_PTR(d_status);
  if (ws_bytes < augment_ws(s, P)) return SPARSP_ERR_WORKSPACE;
  return launch_augment(s, P, scores, row_ptr, col_idx, head_rank, row_ptr_out, col_idx_out, col_cap, added, ws,
                        d_status, (cudaStream_t)stream);
}

size_t sparsp_predictor_workspace_size(const sparsp_shape_t* shape, int32_t rank) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK || rank < 1 || rank > 64) return 0;
  return predictor_ws(s, rank);
}

sparsp_status_t sparsp_predictor_fit(const sparsp_shape_t* shape, int32_t rank, const float* qmeans,
                                     const float* kmeans, float* wq, float* wk, float lr, float* loss,
                                     float* gwq, float* gwk, void* ws, size_t ws_bytes,
                                     sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (rank < 1 || rank > 64) return SPARSP_ERR_UNSUPPORTED;
  if (!isfinite(lr)) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(qmeans);
  CHECK_PTR(kmeans);
  CHECK_PTR(wq);
  CHECK_PTR(wk);
  CHECK_OPT_PTR(loss);
  CHECK_OPT_PTR(gwq);
  CHECK_OPT_PTR(gwk);
  CHECK_PTR(ws);
  if (ws_bytes < predictor_ws(s, rank)) return SPARSP_ERR_WORKSPACE;
  return launch_predictor_fit(s, rank, qmeans, kmeans, wq, wk, lr, loss, gwq, gwk, ws, (cudaStream_t)stream);
}

size_t sparsp_lpt_workspace_size(const sparsp_shape_t* shape) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return lpt_ws(s);
}

sparsp_status_t sparsp_lpt_schedule(const sparsp_shape_t* shape, const int32_t* row_ptr,
                                    uint32_t flags, int32_t* items, void* ws, size_t ws_bytes,
                                    sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  if (flags & ~kKnownFlags) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(row_ptr);
  CHECK_PTR(items);
  const bool flat = (flags & SPARSP_SCHED_FLAT) != 0;
  if (flat) {
    CHECK_PTR(ws);
    if (ws_bytes < lpt_ws(s)) return SPARSP_ERR_WORKSPACE;
  }
  return launch_lpt(s, row_ptr, flat, items, nullptr, ws, (cudaStream_t)stream);
}

sparsp_status_t sparsp_csr_transpose(const sparsp_shape_t* shape, const int32_t* row_ptr,
                                     const int32_t* col_idx, int32_t* col_ptr, int32_t* row_idx,
                                     int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(col_ptr);
  CHECK_PTR(row_idx);
  CHECK_OPT_PTR(d_status);
  return launch_csr_transpose(s, row_ptr, col_idx, col_ptr, row_idx, d_status,
                              (cudaStream_t)stream);
}

int32_t sparsp_attn_launches(const sparsp_shape_t* shape, int32_t backward, int32_t plan, float cap, uint32_t flags) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK || !cap_ok(cap, 0.f, s.d) || (flags & ~kKnownFlags)) return 0;
  const AttnSteps a = attn_steps(s, flags, plan != 0, cap, backward != 0);
  if (a.masked && !a.tc) return 0;
  const int lists = a.compacts ? 3 : 0;
  if (!backward) return lists + a.order_launches() + (a.twice ? 2 : 1);
  // row dot and CSR transpose; an order before each of dQ and dK, dV
  return lists + 2 + 2 * a.order_launches() + 1 + (a.tc && !a.masked && (flags & SPARSP_BWD_SPLIT_KV) ? 2 : 1);
}

size_t sparsp_attn_workspace_size(const sparsp_shape_t* shape, int32_t backward) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return attn_ws_layout(s, backward != 0, nullptr).bytes;
}

sparsp_status_t sparsp_attn_fwd(const sparsp_shape_t* shape, const void* q, const void* k,
                                const void* v, const int32_t* row_ptr, const int32_t* col_idx,
                                float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                                uint32_t flags, uint64_t* prof, int32_t* d_status,
                                sparsp_stream_t stream) {
  return attn_fwd(shape, q, k, v, row_ptr, col_idx, scale, false, 0.f, nullptr, o, lse, ws, ws_bytes, flags, prof,
                  d_status, stream);
}

sparsp_status_t sparsp_attn_bwd(const sparsp_shape_t* shape, const void* q, const void* k,
                                const void* v, const void* o, const float* lse, const void* dout,
                                const int32_t* row_ptr, const int32_t* col_idx, float scale,
                                void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                uint32_t flags, uint64_t* prof, int32_t* d_status,
                                sparsp_stream_t stream) {
  return attn_bwd(shape, q, k, v, o, lse, dout, row_ptr, col_idx, scale, false, 0.f, nullptr, dq, dk, dv, ws, ws_bytes,
                  flags, prof, d_status, stream);
}

size_t sparsp_mask_plan_size(const sparsp_shape_t* shape) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return mask_plan_layout(s).bytes;
}

sparsp_status_t sparsp_mask_plan(const sparsp_shape_t* shape, const int32_t* pos, const int32_t* lo, const int32_t* hi,
                                 void* plan, size_t plan_bytes, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(pos);
  CHECK_PTR(lo);
  CHECK_PTR(hi);
  CHECK_PTR(plan);
  if (plan_bytes < mask_plan_layout(s).bytes) return SPARSP_ERR_WORKSPACE;
  return launch_mask_plan(s, pos, lo, hi, plan, (cudaStream_t)stream);
}

sparsp_status_t sparsp_mask_scores(const sparsp_shape_t* shape, const void* plan, float* scores,
                                   sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(plan);
  CHECK_PTR(scores);
  return launch_mask_scores(s, mask_view(s, plan), scores, (cudaStream_t)stream);
}

sparsp_status_t sparsp_mask_csr(const sparsp_shape_t* shape, const void* plan, const int32_t* row_ptr,
                                const int32_t* col_idx, int32_t* row_ptr_out, int32_t* col_idx_out, int32_t* d_status,
                                sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  CHECK_PTR(plan);
  CHECK_PTR(row_ptr);
  CHECK_PTR(col_idx);
  CHECK_PTR(row_ptr_out);
  CHECK_PTR(col_idx_out);
  CHECK_OPT_PTR(d_status);
  const uintptr_t a = (uintptr_t)row_ptr, b = (uintptr_t)row_ptr_out, n = (uintptr_t)(s.rows() + 1) * sizeof(int32_t);
  if ((a < b + n && b < a + n) || col_idx == col_idx_out) return SPARSP_ERR_INVALID_ARG;   // overlap
  return launch_mask_csr(s, mask_view(s, plan), row_ptr, col_idx, row_ptr_out, col_idx_out, d_status,
                         (cudaStream_t)stream);
}

int32_t sparsp_attn_masked_compacts(const sparsp_shape_t* shape, int32_t backward) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return drops_unseen(s, backward ? attn_bwd_tc_items_per_head(s) : attn_fwd_tc_items_per_head(s)) ? 1 : 0;
}

size_t sparsp_attn_masked_workspace_size(const sparsp_shape_t* shape, int32_t backward) {
  Dims s;
  if (check_shape(shape, &s) != SPARSP_OK) return 0;
  return attn_ws_layout(s, backward != 0, nullptr, true).bytes;
}

sparsp_status_t sparsp_attn_masked_fwd(const sparsp_shape_t* shape, const void* q, const void* k, const void* v,
                                       const int32_t* row_ptr, const int32_t* col_idx, float scale, float cap,
                                       const void* plan, void* o, float* lse, void* ws, size_t ws_bytes,
                                       uint32_t flags, uint64_t* prof, int32_t* d_status, sparsp_stream_t stream) {
  return attn_fwd(shape, q, k, v, row_ptr, col_idx, scale, true, cap, plan, o, lse, ws, ws_bytes, flags, prof, d_status,
                  stream);
}

sparsp_status_t sparsp_attn_masked_bwd(const sparsp_shape_t* shape, const void* q, const void* k, const void* v,
                                       const void* o, const float* lse, const void* dout, const int32_t* row_ptr,
                                       const int32_t* col_idx, float scale, float cap, const void* plan, void* dq,
                                       void* dk, void* dv, void* ws, size_t ws_bytes, uint32_t flags, uint64_t* prof,
                                       int32_t* d_status, sparsp_stream_t stream) {
  return attn_bwd(shape, q, k, v, o, lse, dout, row_ptr, col_idx, scale, true, cap, plan, dq, dk, dv, ws, ws_bytes,
                  flags, prof, d_status, stream);
}

sparsp_status_t sparsp_norm_fwd(const sparsp_shape_t* shape, uint32_t flags, const void* x, int64_t x_stride,
                                const float* w, const float* b, float eps, void* y, float* mean, float* rstd,
                                sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_norm(shape, flags, &s);
  if (r != SPARSP_OK) return r;
  if (!(eps >= 0.f) || isinf(eps)) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(x);
  CHECK_PTR(y);
  CHECK_OPT_PTR(w);
  CHECK_OPT_PTR(b);
  CHECK_OPT_PTR(mean);
  CHECK_OPT_PTR(rstd);
  r = check_stride(s, &x_stride);
  if (r != SPARSP_OK) return r;
  if (overlap(s, x, x_stride, y, (int64_t)s.H * s.d)) return SPARSP_ERR_INVALID_ARG;
  return launch_norm_fwd(s, (flags & SPARSP_NORM_HEAD) != 0, (flags & SPARSP_NORM_RMS) != 0, x, x_stride, w, b, eps, y,
                         mean, rstd, (cudaStream_t)stream);
}

size_t sparsp_norm_workspace_size(const sparsp_shape_t* shape, uint32_t flags) {
  Dims s;
  if (check_norm(shape, flags, &s) != SPARSP_OK) return 0;
  return norm_ws(s, (flags & SPARSP_NORM_HEAD) != 0);
}

sparsp_status_t sparsp_norm_bwd(const sparsp_shape_t* shape, uint32_t flags, const void* dy, const void* x,
                                int64_t x_stride, const float* w, const float* mean, const float* rstd, void* dx,
                                int64_t dx_stride, float* dw, float* db, void* ws, size_t ws_bytes,
                                sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_norm(shape, flags, &s);
  if (r != SPARSP_OK) return r;
  const bool head = (flags & SPARSP_NORM_HEAD) != 0, rms = (flags & SPARSP_NORM_RMS) != 0;
  CHECK_PTR(dy);
  CHECK_PTR(x);
  CHECK_OPT_PTR(w);
  if (!rms) CHECK_PTR(mean);
  CHECK_PTR(rstd);
  CHECK_PTR(dx);
  CHECK_OPT_PTR(dw);
  CHECK_OPT_PTR(db);
  r = check_stride(s, &x_stride);
  if (r != SPARSP_OK) return r;
  r = check_stride(s, &dx_stride);
  if (r != SPARSP_OK) return r;
  if (overlap(s, x, x_stride, dx, dx_stride) || overlap(s, dy, (int64_t)s.H * s.d, dx, dx_stride))
    return SPARSP_ERR_INVALID_ARG;
  if (dw != nullptr || db != nullptr) {
    CHECK_PTR(ws);
    if (ws_bytes < norm_ws(s, head)) return SPARSP_ERR_WORKSPACE;
  }
  return launch_norm_bwd(s, head, rms, dy, x, x_stride, w, mean, rstd, dx, dx_stride, dw, db, ws,
                         (cudaStream_t)stream);
}

size_t sparsp_rope_table_size(const sparsp_rope_t* rope) {
  if (check_rope(rope) != SPARSP_OK) return 0;
  return (size_t)rope_table_entries(*rope) * 2 * sizeof(float);
}

sparsp_status_t sparsp_rope_table(const sparsp_rope_t* rope, double theta, const double offset[3],
                                  const double scale[3], float* table, size_t table_bytes, sparsp_stream_t stream) {
  sparsp_status_t r = check_rope(rope);
  if (r != SPARSP_OK) return r;
  if (!(theta > 0.0) || isinf(theta) || offset == nullptr || scale == nullptr) return SPARSP_ERR_INVALID_ARG;
  for (int ax = 0; ax < 3; ++ax)
    if (!isfinite(offset[ax]) || !isfinite(scale[ax])) return SPARSP_ERR_INVALID_ARG;
  CHECK_PTR(table);
  if (table_bytes < (size_t)rope_table_entries(*rope) * 2 * sizeof(float)) return SPARSP_ERR_WORKSPACE;
  return launch_rope_table(*rope, theta, offset, scale, table, (cudaStream_t)stream);
}

sparsp_status_t sparsp_rope(const sparsp_shape_t* shape, const sparsp_rope_t* rope, const float* table,
                            const int32_t* pos, const void* in, int64_t in_stride, void* out, int64_t out_stride,
                            uint32_t flags, float* means, int32_t* d_status, sparsp_stream_t stream) {
  Dims s;
  sparsp_status_t r = check_shape(shape, &s);
  if (r != SPARSP_OK) return r;
  r = check_rope(rope);
  if (r != SPARSP_OK) return r;
  if (flags & ~(SPARSP_ROPE_INVERSE | SPARSP_ROPE_IN_BLOCKED | SPARSP_ROPE_OUT_BLOCKED)) return SPARSP_ERR_INVALID_ARG;
  const int turned = rope->cols[0] + rope->cols[1] + rope->cols[2];
  if (turned > s.d || (rope->half && turned != s.d)) return SPARSP_ERR_SHAPE;
  const int grid[3] = {s.T, s.Y, s.X};
  if (pos == nullptr)
    for (int ax = 0; ax < 3; ++ax)
      if (rope->cols[ax] > 0 && rope->extent[ax] < grid[ax]) return SPARSP_ERR_SHAPE;
  CHECK_PTR(table);
  CHECK_OPT_PTR(pos);
  CHECK_PTR(in);
  CHECK_PTR(out);
  CHECK_OPT_PTR(means);
  CHECK_OPT_PTR(d_status);
  const bool in_blocked = (flags & SPARSP_ROPE_IN_BLOCKED) != 0, out_blocked = (flags & SPARSP_ROPE_OUT_BLOCKED) != 0;
  if (in_blocked) in_stride = 0;
  if (out_blocked) out_stride = 0;
  r = check_stride(s, &in_stride);
  if (r != SPARSP_OK) return r;
  r = check_stride(s, &out_stride);
  if (r != SPARSP_OK) return r;
  if (overlap(s, in, in_stride, out, out_stride)) return SPARSP_ERR_INVALID_ARG;
  return launch_rope(s, *rope, table, pos, in, in_stride, in_blocked, out, out_stride, out_blocked,
                     (flags & SPARSP_ROPE_INVERSE) != 0, means, d_status, (cudaStream_t)stream);
}

}  // extern "C"
