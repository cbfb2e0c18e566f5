// What the kernels of attention over the cache share: the items that work is dealt out by, the checks of look-ups,
// the parts of items that several CTAs share, and what scales do to scores and weights.
#pragma once

#include <float.h>

#include "cache.cuh"

namespace sparsp {

// Entries are requests (every block is seen, all key heads alike), or with lists request and
// key head.
struct Entry {
  int b, hk, n, len, s0;        // n: new tokens, s0: the first one's row; hk: with lists
  int units;                    // of 64 keys
  int groups;                   // of rows: the kernel's own count, as are
  int64_t per_head, weight;
};
__device__ __forceinline__ int entries_of(const CacheAttn& a) { return a.row_ptr != nullptr ? a.B * a.c.heads : a.B; }
// What cannot be right is reported (with tell) and counts as nothing: rows, keys or list.
__device__ __forceinline__ Entry entry_at(const CacheAttn& a, int e, bool tell) {
  Entry x;
  x.hk = a.row_ptr != nullptr ? e % a.c.heads : 0;
  x.b = a.row_ptr != nullptr ? e / a.c.heads : e;
  x.s0 = a.start[x.b];
  const int s1 = a.start[x.b + 1];
  x.n = (int)max((int64_t)-1, (int64_t)s1 - x.s0);
  x.len = a.len[x.b];
  if (x.s0 < 0 || x.n < 0 || s1 > a.tokens || x.n > a.max_add) {
    if (tell) report(a.d_status, SPARSP_ERR_DATA);
    x.n = 0;
  }
  if (x.len < 0 || x.len > (int64_t)a.max_blocks * a.c.bt) {
    if (tell) report(a.d_status, SPARSP_ERR_DATA);
    x.len = 0;
  }
  if (a.row_ptr != nullptr) {
    const int64_t p0 = a.row_ptr[e], p1 = a.row_ptr[e + 1];
    int64_t count = p1 - p0;
    if (p0 < 0 || count < 0 || count > a.max_blocks || p1 > a.col_cap) {
      if (tell) report(a.d_status, SPARSP_ERR_DATA);
      count = 0;
    }
    x.units = (int)count * (a.c.bt / kUnit);
  } else {
    x.units = (x.len + kUnit - 1) / kUnit;
  }
  x.groups = 0;
  x.per_head = x.weight = 0;
  return x;
}

// Does a block that a list names hold tokens of the request; is what a table names a block of the pool?
__device__ __forceinline__ bool has_tokens(const CacheAttn& a, const Entry& x, int j) { return j >= 0 && (int64_t)j * a.c.bt < x.len; }
__device__ __forceinline__ bool in_pool(const CacheAttn& a, int page) { return page >= 0 && page < a.c.blocks; }

// The sum over the CTA's threads below this one, and over all of its WARPS warps.
template <int WARPS>
__device__ __forceinline__ int64_t scan_below(int64_t mine, int64_t* sm, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t below = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, below, off);
    if (lane >= off) below += v;
  }
  if (lane == 31) sm[warp] = below;
  below -= mine;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) below += sm[i];
    all += sm[i];
  }
  *total = all;
  return below;
}

// What the joining kernel needs to know of the item that starts in a CTA and goes on in others.
struct Open {
  int hk, row0, rows, s0, last;   // last: the CTA of its last unit; -1: there is none
};
struct Parts {
  Open* open;      // [ctas]
  float2* ml;      // [2 ctas][rows] log2 of the sum of the weights, and 1 (0: none); a CTA's parts: an item that goes on, one that starts
  float* o;        // [2 ctas][rows][d] the part's own result
};
inline size_t parts_align(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t parts_bytes(int ctas, int rows, int d) {
  return parts_align(ctas * sizeof(Open)) + parts_align((size_t)2 * ctas * rows * sizeof(float2)) +
         (size_t)2 * ctas * rows * d * sizeof(float);
}
inline Parts parts_of(void* ws, int ctas, int rows) {
  uint8_t* at = (uint8_t*)ws;
  Parts p;
  p.open = (Open*)at;
  at += parts_align(ctas * sizeof(Open));
  p.ml = (float2*)at;
  at += parts_align((size_t)2 * ctas * rows * sizeof(float2));
  p.o = (float*)at;
  return p;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// What a product of codes is a score by: the row's factor times the keys' scale, but a number (or NaN) in whose place a
// product of 0 gives 0; with SIZE a normal one, so that the -inf of a hidden key stays -inf. (Rows of zeros and blocks of
// zeros have the least factors there are, and their product is 0 in fp32. At 2^-126 a product of codes, below
// 2^32, still is a score of 0.)
template <bool SIZE>
__device__ __forceinline__ float score_factor(float row, float ks) {
  const float f = row * ks;
  return SIZE && f < FLT_MIN ? FLT_MIN : f > FLT_MAX ? FLT_MAX : f;
}

// The scales vs of V's blocks go into the exponents against u, a scale near the largest of a piece's blocks so far:
//   P = 2^(y + log2 (vs / u) - R),  l = sum P u / vs,  O = u sum P V / l,  LSE = (R + log2 l) ln 2
// (y: scores in base 2), so that blocks of different scales add up in one accumulator and l holds plain weights. u
// rises where a scale is 2^kAbove beyond it, and what has been summed of O goes down by as much. The values of a block
// 2^kBelow under u are 0 beside the others' (its vs counts as u). So P of a row's largest weights is at least
// 2^-(kAbove + kBelow), which neither vanishes nor, in l, overflows, whatever scales come side by side: zeros are held
// under 2^-100.
constexpr float kAbove = 8.f, kBelow = 80.f;
constexpr float kLeastScale = 0x1p-120f;   // of V that counts

// Writes four columns of a finished row, and its LSE (in base 2 here); none: it has seen nothing.
template <int D>
__device__ __forceinline__ void finish(const CacheAttn& a, int s0, int hk, int row, int c, bool none, float lse2,
                                       const float4& o) {
  const int64_t at = (int64_t)(s0 + row / a.group) * a.H + hk * a.group + row % a.group;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
  *reinterpret_cast<uint2*>(a.o + at * D + c) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (c == 0) a.lse[at] = none ? -INFINITY : lse2 * 0.6931471805599453f;
}

// A part's weight in its row's join, against the largest part's: at most 1.
__device__ __forceinline__ float part_weight(const float2& ml, float top) { return ml.y == 0.f ? 0.f : exp2_fast(ml.x - top); }
// The joined row, of the weights' sum and the weighted results.
template <int D>
__device__ __forceinline__ void finish_join(const CacheAttn& a, int s0, int hk, int row, int c, float top, float sum,
                                            const float4& all) {
  const bool none = sum == 0.f;
  const float f = none ? 0.f : 1.0f / sum;
  finish<D>(a, s0, hk, row, c, none, top + log2f(sum), make_float4(all.x * f, all.y * f, all.z * f, all.w * f));
}

}  // namespace sparsp
