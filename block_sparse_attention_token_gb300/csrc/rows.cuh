// Pieces of the passes over query / key rows (rotary positions, with or without the
// norm): 16-byte vectors of a row as fp32 values, copies into shared memory, and the
// rotation's table.
#pragma once

#include "tc_helpers.cuh"

namespace sparsp {

struct RopeArgs {
  int cols[3];          // columns per axis
  int extent[3];        // table rows per axis
  int base[3];          // first table entry per axis
  const float2* table;
  const int32_t* pos;   // [B, N, 3] or null: grid coordinates
  float sign;           // -1: inverse
};


inline RopeArgs rope_args(const sparsp_rope_t& r, const float* table) {
  RopeArgs a{};
  int64_t at = 0;
  for (int ax = 0; ax < 3; ++ax) {
    a.cols[ax] = r.cols[ax];
    a.extent[ax] = r.extent[ax];
    a.base[ax] = (int)at;
    at += (int64_t)r.extent[ax] * (r.cols[ax] / 2);
  }
  a.table = reinterpret_cast<const float2*>(table);
  a.sign = 1.f;
  return a;
}

template <typename T>
struct Row16;
template <>
struct Row16<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __bfloat1622float2(h[e]);
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    return v;
  }
};
template <>
struct Row16<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }


}  // namespace sparsp
