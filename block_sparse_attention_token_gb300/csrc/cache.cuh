// A cache of keys and values in 8 bits: pools of blocks, found through a table per
// request, one scale per block and head.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sparsp {

constexpr int kCacheMaxRequests = 16384;
constexpr int kUnit = 64;                 // keys that the attention kernels count work by

// A cache that the API layer has checked.
struct CacheDims {
  int blocks, heads, d, bt;
};

struct CacheExtend {
  int B, max_blocks, n_free, tokens;
  const int32_t *len, *add, *free_blocks, *used;
  int32_t *table, *len_out, *start, *slots, *used_out;
};
sparsp_status_t launch_cache_extend(const CacheDims& c, const CacheExtend& a, int32_t* d_status, cudaStream_t st);

struct CacheWrite {
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;   // elements between tokens, and between heads
  const int32_t* slots;
  int tokens;
  uint8_t *kc, *vc;
  float *ks, *vs;
};
sparsp_status_t launch_cache_write(const CacheDims& c, int dtype, const CacheWrite& a, int32_t* d_status,
                                   cudaStream_t st);

struct CacheAttn {
  CacheDims c;
  int B, H, group;           // group: query heads to a key head
  int max_blocks, tokens, max_add;
  const __nv_bfloat16* q;
  int64_t q_token;           // elements between query tokens
  const int32_t *start, *len, *table;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *row_ptr, *col_idx;   // null: every block
  int64_t col_cap;
  float scale_log2;          // scale * log2(e)
  bool causal;
  __nv_bfloat16* o;          // [tokens, H, d]
  float* lse;                // [tokens, H]
  int32_t* d_status;
  int few;                   // rows of a request up to which it is the kernel's for few rows (0: it takes every one)
};
// Few rows of a request, and the dispatch; many rows.
size_t attn_cache_ws(const CacheDims& c, int group, int max_add);
sparsp_status_t launch_attn_cache(const CacheAttn& a, void* ws, cudaStream_t st);
size_t attn_cache_tc_ws(const CacheDims& c);
sparsp_status_t launch_attn_cache_tc(const CacheAttn& a, void* ws, cudaStream_t st);

// Two fp32 values as e4m3 codes, lo in the low byte (round to nearest even, at most +-448), and the low two bytes as the
// values that they stand for.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ float2 e4m3_values(uint32_t two) {
  const uint32_t h = f16x2_of_e4m3(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace sparsp
