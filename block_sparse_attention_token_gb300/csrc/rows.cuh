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

// Two fp32 values in one 64-bit register pair, for the packed fp32 instructions:
// held as one operand from load to store, so that no moves are spent on pairing.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("sub.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float hsum(f32x2 v) {
  const float2 t = both(v);
  return t.x + t.y;
}

// 1 / sqrt(x) to 2^-22: a row's factor, of which fp32 sums know no more.
__device__ __forceinline__ float inv_sqrt(float x) { return rsqrtf(x); }

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


// What a lane holds of a row as pairs to be turned: pair i is (x[i], y[i]), two pairs to a
// packed operand. A unit is one 16-byte vector with columns (2i, 2i + 1) paired, or with
// HALF two, from the two halves of the row.
template <typename T, bool HALF>
struct Unit;
template <>
struct Unit<__nv_bfloat16, false> {
  static constexpr int P2 = 2;
  static __device__ __forceinline__ void unpack(const uint4* v, f32x2* x, f32x2* y) {
    const uint32_t w[4] = {v->x, v->y, v->z, v->w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // a bf16 is the upper half of its fp32
      x[i] = pair(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
      y[i] = pair(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ void pack(const f32x2* x, const f32x2* y, uint4* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = both(x[i]), b = both(y[i]);
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(a.x, b.x), h1 = __floats2bfloat162_rn(a.y, b.y);
      w[2 * i] = *reinterpret_cast<const uint32_t*>(&h0);
      w[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h1);
    }
    *v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Unit<__nv_bfloat16, true> {
  static constexpr int P2 = 4;
  static __device__ __forceinline__ void unpack(const uint4* v, f32x2* x, f32x2* y) {
    const uint32_t a[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, b[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = pair(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
      y[i] = pair(__uint_as_float(b[i] << 16), __uint_as_float(b[i] & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ void pack(const f32x2* x, const f32x2* y, uint4* v) {
    uint32_t w[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = both(x[i]), b = both(y[i]);
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(a.x, a.y), h1 = __floats2bfloat162_rn(b.x, b.y);
      w[0][i] = *reinterpret_cast<const uint32_t*>(&h0);
      w[1][i] = *reinterpret_cast<const uint32_t*>(&h1);
    }
    v[0] = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
    v[1] = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
  }
};
template <>
struct Unit<float, false> {
  static constexpr int P2 = 1;
  static __device__ __forceinline__ void unpack(const uint4* v, f32x2* x, f32x2* y) {
    x[0] = pair(__uint_as_float(v->x), __uint_as_float(v->z));
    y[0] = pair(__uint_as_float(v->y), __uint_as_float(v->w));
  }
  static __device__ __forceinline__ void pack(const f32x2* x, const f32x2* y, uint4* v) {
    const float2 a = both(x[0]), b = both(y[0]);
    *v = make_uint4(__float_as_uint(a.x), __float_as_uint(b.x), __float_as_uint(a.y), __float_as_uint(b.y));
  }
};
template <>
struct Unit<float, true> {
  static constexpr int P2 = 2;
  static __device__ __forceinline__ void unpack(const uint4* v, f32x2* x, f32x2* y) {
    x[0] = pair(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
    x[1] = pair(__uint_as_float(v[0].z), __uint_as_float(v[0].w));
    y[0] = pair(__uint_as_float(v[1].x), __uint_as_float(v[1].y));
    y[1] = pair(__uint_as_float(v[1].z), __uint_as_float(v[1].w));
  }
  static __device__ __forceinline__ void pack(const f32x2* x, const f32x2* y, uint4* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = both(h ? y[0] : x[0]), b = both(h ? y[1] : x[1]);
      v[h] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
  }
};

// Launches a kernel that may begin before the one before it ends, and waits for it itself.
template <typename... Params, typename... Args>
sparsp_status_t launch_after(void (*kern)(Params...), dim3 grid, int threads, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

}  // namespace sparsp
