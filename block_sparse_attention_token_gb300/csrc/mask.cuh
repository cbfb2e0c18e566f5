// Token mask of attention: query n sees key m where lo[n] <= pos[m] < hi[n].
// A plan holds the three arrays in tile order and the ranges of each block.
#pragma once

#include "common.cuh"

namespace sparsp {

// A plan's parts (sparsp_mask_plan), or all null: no mask. A query's interval
// is lo and its length (0 when hi <= lo), so that with unsigned arithmetic
// "sees" is pos - lo < len for every int32 value.
struct MaskView {
  const int32_t* pos;     // [B, N] tile order
  const int32_t* lo;      // [B, N]
  const uint32_t* len;    // [B, N]
  const int2* krange;     // [B, nb] smallest and largest pos of a block
  const int2* qrange;     // [B, nb] largest lo and smallest hi of a block: what every query sees
  const int2* qhull;      // [B, nb] smallest lo and largest hi over queries that see anything
};

// May some query of a block with hull q see some key of a block with range k?
__device__ __forceinline__ bool blocks_meet(const int2& q, const int2& k) { return k.y >= q.x && k.x < q.y; }

// Does every query of a block with common range q see every key of a block with range k?
__device__ __forceinline__ bool all_seen(const int2& q, const int2& k) { return q.x <= k.x && k.y < q.y; }

// Rows of a warp that see alike. The 32 rows of a warp hold few different
// intervals (or positions), so the keys each row sees come as bits from one
// ballot per group and 32 columns, not from a comparison per score.
struct RowGroups {
  uint32_t mine;      // the lanes of this lane's group
  uint32_t leaders;   // one lane of each group
  __device__ __forceinline__ void make(uint32_t a, uint32_t b, int lane) {
    mine = __match_any_sync(0xffffffffu, a) & __match_any_sync(0xffffffffu, b);
    leaders = __ballot_sync(0xffffffffu, __ffs(mine) - 1 == lane);
  }
};
// Rows are queries with interval (lo, len); each lane brings the positions k0,
// k1 of two columns (lane and 32 + lane): bit c of w0 / w1 = the row sees the column.
__device__ __forceinline__ void query_bits(const RowGroups& g, uint32_t lo, uint32_t len, int32_t k0, int32_t k1,
                                           int lane, uint32_t& w0, uint32_t& w1) {
  w0 = w1 = 0u;
  for (uint32_t rem = g.leaders; rem != 0u; rem &= rem - 1u) {
    const int l = __ffs(rem) - 1;
    const uint32_t a = __shfl_sync(0xffffffffu, lo, l), n = __shfl_sync(0xffffffffu, len, l);
    const uint32_t b0 = __ballot_sync(0xffffffffu, (uint32_t)k0 - a < n);
    const uint32_t b1 = __ballot_sync(0xffffffffu, (uint32_t)k1 - a < n);
    if ((g.mine >> l) & 1u) {
      w0 = b0;
      w1 = b1;
    }
  }
}
// The same for 32 columns, one per lane.
__device__ __forceinline__ uint32_t query_bits(const RowGroups& g, uint32_t lo, uint32_t len, int32_t k) {
  uint32_t w = 0u;
  for (uint32_t rem = g.leaders; rem != 0u; rem &= rem - 1u) {
    const int l = __ffs(rem) - 1;
    const uint32_t a = __shfl_sync(0xffffffffu, lo, l), n = __shfl_sync(0xffffffffu, len, l);
    const uint32_t b = __ballot_sync(0xffffffffu, (uint32_t)k - a < n);
    if ((g.mine >> l) & 1u) w = b;
  }
  return w;
}
// Rows are keys at position pos; each lane brings the interval of one query column.
__device__ __forceinline__ uint32_t key_bits(const RowGroups& g, int32_t pos, int32_t lo, uint32_t len) {
  uint32_t w = 0u;
  for (uint32_t rem = g.leaders; rem != 0u; rem &= rem - 1u) {
    const int l = __ffs(rem) - 1;
    const uint32_t x = (uint32_t)__shfl_sync(0xffffffffu, pos, l);
    const uint32_t b = __ballot_sync(0xffffffffu, x - (uint32_t)lo < len);
    if ((g.mine >> l) & 1u) w = b;
  }
  return w;
}

// Byte layout of a plan.
struct MaskPlan {
  size_t pos, lo, len, krange, qrange, qhull, bytes;
};
inline MaskPlan mask_plan_layout(const Dims& s) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t t = up((size_t)s.B * s.N * 4), r = up((size_t)s.B * s.nb * 8);
  return MaskPlan{0, t, 2 * t, 3 * t, 3 * t + r, 3 * t + 2 * r, 3 * t + 3 * r};
}
inline MaskView mask_view(const Dims& s, const void* plan) {
  if (plan == nullptr) return MaskView{};
  const MaskPlan l = mask_plan_layout(s);
  const uint8_t* p = (const uint8_t*)plan;
  return MaskView{(const int32_t*)(p + l.pos),   (const int32_t*)(p + l.lo),   (const uint32_t*)(p + l.len),
                  (const int2*)(p + l.krange), (const int2*)(p + l.qrange), (const int2*)(p + l.qhull)};
}

sparsp_status_t launch_mask_plan(const Dims& s, const int32_t* pos, const int32_t* lo, const int32_t* hi, void* plan,
                                 cudaStream_t st);
sparsp_status_t launch_mask_scores(const Dims& s, const MaskView& m, float* scores, cudaStream_t st);
// The CSR without the block pairs that see nothing of each other. A malformed
// row becomes empty and reports SPARSP_ERR_DATA.
sparsp_status_t launch_mask_csr(const Dims& s, const MaskView& m, const int32_t* row_ptr, const int32_t* col_idx,
                                int32_t* out_ptr, int32_t* out_idx, int32_t* d_status, cudaStream_t st);

// The longest-first order of a problem whose items one CTA orders at once: one launch in
// place of the pairs' costs, the order and a memset, for problems of one wave (1,024
// tokens, 2 heads: forward 33 -> 30 us, backward 68 -> 61 us), and for lists a mask
// makes uneven whose K and V stay in L2 (64 MB at most), so that heads need not be taken
// one after the other. Head by head against this order, clips of 8,192 tokens: 24 MB of K and
// V forward 226 -> 216 us, backward 689 -> 672; 48 MB 423 -> 409 and 1,406 -> 1,399 (d = 128: 195
// -> 177, 730 -> 683); 64 MB 240 -> 217, 914 -> 855. Beyond, the two are near each other or this
// one loses: 96 MB 323 -> 310 us with 24 heads, 367 -> 371 with 12 longer ones, 128 MB 1,834
// -> 1,871, 192 MB 2,314 -> 2,566. Without a mask (lists of about one length, capped) it gains
// or loses as much: 24 MB 280 -> 291 us, 64 MB 362 -> 341, backward 1,226 -> 1,247 at 48 MB.
bool order_items_fits(const Dims& s, int per_head, bool uneven);
sparsp_status_t launch_order_items(const Dims& s, int per_head, const int32_t* row_ptr, int32_t* items,
                                   int32_t* counter, int32_t* zero, int n_zero, cudaStream_t st);

// Up to this cap one reference c0 = max(0, cap log2(e) - 20) holds every score: P lies
// in [2^-37.8, 2^20], so that sums of 2^19 terms and their products with values from
// 2^-88 to 2^88 stay normal fp32 numbers. Beyond it c0 = 0 and the rows are checked.
constexpr float kFixedCap = 20.0f;

// Items the fast forward kernels pass on to the general one.
struct FixList {
  int32_t* items;     // [items]
  int32_t* mark;      // [items], count and counter behind it, all zeroed before
  int32_t* count;     // 1
  int32_t* counter;   // 1: the general kernel's pull counter
};

// tcgen05 attention with a token mask (may be empty) and a score cap (0: none).
sparsp_status_t launch_attn_fwd_masked(const Dims& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                       const __nv_bfloat16* v, const int32_t* row_ptr, const int32_t* col_idx,
                                       float scale, float cap, const MaskView& mask, __nv_bfloat16* o, float* lse,
                                       bool raster, bool in_raster, const int32_t* items, int32_t* counter,
                                       const FixList& fix, uint64_t* prof, int32_t* d_status, cudaStream_t st);
sparsp_status_t launch_attn_bwd_masked(const Dims& s, int mode, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                       const __nv_bfloat16* v, const __nv_bfloat16* dout, const float* lse2,
                                       const float* delta, const int32_t* ptr, const int32_t* idx, float scale,
                                       __nv_bfloat16* out, __nv_bfloat16* out2, const int32_t* items,
                                       int32_t* counter, uint64_t* prof, int32_t* d_status, bool raster,
                                       const MaskView& mask, float cap, cudaStream_t st);

}  // namespace sparsp
