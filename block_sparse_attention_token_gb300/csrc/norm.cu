// Token norm: layer norm or RMS norm of query / key (or hidden) rows in raster
// order [B, N, H, d], over the d values of a head or the H*d values of a token,
// forward and backward.
//
//   mean = sum x / C (0 for RMS), var = sum (x - mean)^2 / C,
//   rstd = 1 / sqrt(var + eps), y = (x - mean) rstd w + b;
//   xh = (x - mean) rstd, g = dy w,
//   dx = rstd (g - [mean_C(g)] - xh mean_C(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
// ([.] is left out for RMS). The variance is taken about the mean in a second
// sweep over registers, so a row with a large mean loses nothing.
//
// Bound by HBM: the forward reads x and writes y, the backward reads x and dy
// and writes dx, each once. A thread owns the same columns of every row its
// CTA visits, so w, b and the column sums of dw and db stay in registers; the
// row sums are warp shuffles (rows of up to 128 16-byte vectors) or one
// shared-memory exchange per batch of rows (longer rows, a CTA per row). Two bf16
// values are one fp32 pair from load to store (packed instructions): with scalar
// arithmetic the backward was bound by what it issues (343 us against 164 below,
// together with the rings). Rows are copied into shared memory some steps ahead
// (cp.async), each thread its own vectors, as registers for so many loads are not there.
// Measured, cold cache, against a copy's 6.67 TB/s (bf16):
//   forward,  RMS, 30,720 rows of 5,120: 107 us, 5.9 TB/s (0.88)
//   backward, 30,720 rows of 5,120 with dw and db: 164 us, 5.7 TB/s (0.86), of it 9 us the
//   sum over the CTAs' parts
//   backward, 1,572,864 rows of 128 (a head's norm): 195 us, 6.3 TB/s (0.94)
//   forward, 1,572,864 rows of 128: 150 us, 5.4 TB/s (0.80); fp32, 30,720 rows of 5,120: RMS 210 us
//   (0.90), layer norm 259 us (0.73)
//   forward, 2,048 fp32 rows of 64: 8.6 us, the call and its launch
// Rows beyond 1,024 vectors have four vectors a thread in CTAs of 512 (bf16) or 1,024 (fp32)
// threads, whose registers do not hold the backward's sums: it spills 288 to 372 bytes a
// thread and takes about twice the bytes' time (fp32, 30,720 rows of 5,120: 641 us, floor 283;
// bf16, rows of 12,288: 687, floor 340).
#include "common.cuh"
#include "tc_helpers.cuh"

namespace sparsp {
namespace {

constexpr int kWarpThreads = 256;   // CTA of the shuffle kernels
constexpr int kMaxWarps = 32;

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
__device__ __forceinline__ float hsum(f32x2 v) {
  const float2 t = both(v);
  return t.x + t.y;
}

// 16 bytes of a row as fp32 pairs and back.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, f32x2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)   // a bf16 is the upper half of its fp32
      f[e] = pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2* f) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = both(f[e]);
      h[e] = __floats2bfloat162_rn(t.x, t.y);
    }
    return v;
  }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, f32x2* f) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2* f) {
    const float2 a = both(f[0]), b = both(f[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};

// Rows are numbered token-major: row = token * groups + group, with one group
// of C = H*d values per token or H groups of C = d values. A strided tensor
// has `stride` elements between tokens; the others are contiguous.
struct Rows {
  int64_t rows;
  int groups;   // 1, or H
  int C;        // values per row
  int V;        // 16-byte vectors per row
  __device__ __forceinline__ int64_t at(int64_t row, int64_t stride) const {
    if (stride == (int64_t)groups * C) return row * C;
    const int64_t tok = groups == 1 ? row : (int64_t)((uint32_t)row / (uint32_t)groups);
    return tok * stride + (row - tok * groups) * C;
  }
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// Until at most n of this thread's copy groups are in flight (n < 4).
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copy_wait(int n) {
  if (n == 3) copy_wait<3>();
  else if (n == 2) copy_wait<2>();
  else if (n == 1) copy_wait<1>();
  else copy_wait<0>();
}

// Sum of K values over the threads that share a row: L lanes of a warp, or the
// whole CTA (L = 0) through shared memory, in a fixed order. `buf` alternates
// between calls so that one barrier per call is enough.
template <int L, int K, int MAXT = 1024>
__device__ __forceinline__ void row_sum(float (&v)[K], float* sm, int& buf) {
#pragma unroll
  for (int off = (L == 0 ? 32 : L) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if (L == 0) {
    float* s = sm + buf * (kMaxWarps * K);
    buf ^= 1;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[warp * K + k] = v[k];
    __syncthreads();
    // four values per load: 4 / K warps' sums (zeros past the last warp), all loads at once
    static_assert(K == 1 || K == 2 || K == 4, "row sums per step");
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < MAXT / 32; w += 4 / K) {
      const float4 p = reinterpret_cast<const float4*>(s)[w * K / 4];
      q.x += p.x;
      q.y += p.y;
      q.z += p.z;
      q.w += p.w;
    }
    const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = f[k];
#pragma unroll
    for (int i = K; i < 4; ++i) v[i % K] += f[i];
  }
}

// One thread's share of a row: U vectors, t + u * T (T threads per row). `have`
// is how many of them exist; the others hold zeros.
template <typename T, int U, bool RMS>
struct Share {
  using X = Vec<T>;
  static constexpr int E = X::E, P = E / 2;   // values and pairs of a vector
  static __device__ __forceinline__ void values(const uint4 (&x)[U], f32x2 (&f)[U * P]) {
#pragma unroll
    for (int u = 0; u < U; ++u) X::unpack(x[u], f + u * P);
  }
  static __device__ __forceinline__ float mean_part(const f32x2 (&f)[U * P]) {
    f32x2 a = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < U * P; ++i) a = add2(a, f[i]);
    return hsum(a);
  }
  // x - mu in place, and the sum of its square over the vectors that exist (a
  // missing one held zeros, not the mean)
  static __device__ __forceinline__ float var_part(f32x2 (&f)[U * P], float mu, int have) {
    f32x2 a = pair(0.f, 0.f);
    const f32x2 m = pair(-mu, -mu);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (RMS || u < have)
#pragma unroll
        for (int i = u * P; i < (u + 1) * P; ++i) {
          if (!RMS) f[i] = add2(f[i], m);
          a = fma2(f[i], f[i], a);
        }
    return hsum(a);
  }
  // (x - mu) rs w + b of one vector of x - mu
  static __device__ __forceinline__ uint4 out(const f32x2* f, float rs, const f32x2* w, const f32x2* b) {
    const f32x2 r = pair(rs, rs);
    f32x2 y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = fma2(mul2(f[i], r), w[i], b[i]);
    return X::pack(y);
  }
  // column sums of dw and db, row sums of g xh and g (g = dy w, xh = x rs - mu rs),
  // and xh and g themselves for grad_out
  static __device__ __forceinline__ void grad_part(const uint4 (&x)[U], const uint4 (&dy)[U], float mu, float rs,
                                                   const f32x2* w, f32x2* dw, f32x2* db, f32x2 (&h)[U * P],
                                                   f32x2 (&g)[U * P], float& sgx, float& sg) {
    f32x2 a = pair(0.f, 0.f), c = a;
    const f32x2 r = pair(rs, rs), shift = pair(-mu * rs, -mu * rs);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      X::unpack(x[u], h + u * P);
      X::unpack(dy[u], g + u * P);   // zero past the row and past the last row, whatever xh is there
#pragma unroll
      for (int k = u * P; k < (u + 1) * P; ++k) {
        h[k] = RMS ? mul2(h[k], r) : fma2(h[k], r, shift);
        dw[k] = fma2(g[k], h[k], dw[k]);
        db[k] = add2(db[k], g[k]);
        g[k] = mul2(g[k], w[k]);
        a = fma2(g[k], h[k], a);
        if (!RMS) c = add2(c, g[k]);
      }
    }
    sgx = hsum(a);
    sg = hsum(c);
  }
  // dx = rs (g - mg - xh mgx) of one vector
  static __device__ __forceinline__ uint4 grad_out(const f32x2* h, const f32x2* g, float rs, float mg, float mgx) {
    const f32x2 scale = pair(-rs * mgx, -rs * mgx), offset = pair(-rs * mg, -rs * mg), r = pair(rs, rs);
    f32x2 f[P];
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = fma2(g[i], r, RMS ? mul2(h[i], scale) : fma2(h[i], scale, offset));
    return X::pack(f);
  }
  // this thread's columns of a parameter vector
  static __device__ __forceinline__ void params(const float* p, float missing, int t, int T_row, int V, f32x2* out) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int v = t + u * T_row;
        const bool there = v < V && p != nullptr;
        out[u * P + i] = pair(there ? p[v * E + 2 * i] : missing, there ? p[v * E + 2 * i + 1] : missing);
      }
  }
};

// Rows of up to 128 vectors: L lanes per row with U vectors each (two where the
// row allows: fewer shuffles per value), RB rows in flight per lane group.
template <typename T, int L, int U, int RB, bool RMS>
__global__ void __launch_bounds__(kWarpThreads)
norm_fwd_kernel(const Rows R, const T* __restrict__ x, int64_t x_stride, const float* __restrict__ w,
                const float* __restrict__ b, float eps, T* __restrict__ y, float* __restrict__ mean,
                float* __restrict__ rstd) {
  using S = Share<T, U, RMS>;
  constexpr int E = S::E;
  int buf = 0;
  const int t = threadIdx.x % L;                          // this thread's place in its row
  constexpr int slots = kWarpThreads / L;
  const int slot = threadIdx.x / L;
  const int have = (R.V - t + L - 1) / L;                 // vectors of this thread that exist
  f32x2 wr[U * S::P], br[U * S::P];
  S::params(w, 1.f, t, L, R.V, wr);
  S::params(b, 0.f, t, L, R.V, br);
  const float inv_c = 1.0f / (float)R.C;
  const int64_t step = (int64_t)gridDim.x * slots * RB;
  for (int64_t base = (int64_t)blockIdx.x * slots * RB; base < R.rows; base += step) {
    uint4 xv[RB][U];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      const uint4* src = reinterpret_cast<const uint4*>(x + (row < R.rows ? R.at(row, x_stride) : 0)) + t;
#pragma unroll
      for (int u = 0; u < U; ++u) xv[r][u] = row < R.rows && u < have ? __ldcs(src + u * L) : make_uint4(0, 0, 0, 0);
    }
    f32x2 f[RB][U * S::P];
    float mu[RB], q[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      S::values(xv[r], f[r]);
      mu[r] = 0.f;
    }
    if (!RMS) {
#pragma unroll
      for (int r = 0; r < RB; ++r) mu[r] = S::mean_part(f[r]);
      row_sum<L, RB>(mu, nullptr, buf);
#pragma unroll
      for (int r = 0; r < RB; ++r) mu[r] *= inv_c;
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) q[r] = S::var_part(f[r], mu[r], have);
    row_sum<L, RB>(q, nullptr, buf);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      if (row >= R.rows) continue;
      const float rs = 1.0f / sqrtf(q[r] * inv_c + eps);
      uint4* dst = reinterpret_cast<uint4*>(y + row * R.C) + t;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < have) __stcs(dst + u * L, S::out(f[r] + u * S::P, rs, wr + u * S::P, br + u * S::P));
      if (t == 0) {
        if (!RMS && mean != nullptr) mean[row] = mu[r];
        if (rstd != nullptr) rstd[row] = rs;
      }
    }
  }
}

// Longer rows: a CTA per row, RB rows per step. Each thread copies its own vectors
// of the next rows into its own shared-memory slots (cp.async, `depth` steps of
// them, as many of four as fit), so nothing but the row sums needs a barrier.
constexpr int kMaxDepth = 4;
constexpr size_t kRingBytes = 220000;
inline int ring_depth(size_t step, int ctas) {
  int d = kMaxDepth;
  while (d > 1 && step * d * ctas > kRingBytes) --d;
  return d;
}
// MAXT, MINB: threads and resident CTAs the registers are shared out for.
template <typename T, int U, int RB, bool RMS, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
norm_fwd_cta_kernel(const Rows R, const T* __restrict__ x, int64_t x_stride,
                                    const float* __restrict__ w, const float* __restrict__ b, float eps,
                                    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, int depth) {
  using S = Share<T, U, RMS>;
  constexpr int E = S::E;
  extern __shared__ uint4 ring[];   // [depth][RB][U][T_row]
  __shared__ __align__(16) float sm[2 * kMaxWarps * RB];
  int buf = 0;
  const int t = threadIdx.x, T_row = blockDim.x;
  const int have = (R.V - t + T_row - 1) / T_row;
  f32x2 wr[U * S::P], br[U * S::P];
  S::params(w, 1.f, t, T_row, R.V, wr);
  S::params(b, 0.f, t, T_row, R.V, br);
  for (int i = t; i < 2 * kMaxWarps * RB; i += T_row) sm[i] = 0.f;
  __syncthreads();
  const float inv_c = 1.0f / (float)R.C;
  const int64_t step = (int64_t)gridDim.x * RB;
  auto slot = [&](int st, int r, int u) { return ring + ((st * RB + r) * U + u) * T_row + t; };
  auto fetch = [&](int64_t base, int st) {
#pragma unroll
    for (int r = 0; r < RB; ++r)
      if (base + r < R.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + R.at(base + r, x_stride)) + t;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < have) copy_async16(slot(st, r, u), src + u * T_row);
      }
    copy_commit();
  };
  const int64_t first = (int64_t)blockIdx.x * RB;
  for (int s = 0; s < depth - 1; ++s) fetch(first + s * step, s);
  int st = 0;
  for (int64_t base = first; base < R.rows; base += step, st = st + 1 == depth ? 0 : st + 1) {
    fetch(base + (depth - 1) * step, st == 0 ? depth - 1 : st - 1);   // the slots of the step before
    copy_wait(depth - 1);
    uint4 xv[RB][U];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u)
        xv[r][u] = base + r < R.rows && u < have ? *slot(st, r, u) : make_uint4(0, 0, 0, 0);
    f32x2 f[RB][U * S::P];
    float mu[RB], q[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      S::values(xv[r], f[r]);
      mu[r] = 0.f;
    }
    if (!RMS) {
#pragma unroll
      for (int r = 0; r < RB; ++r) mu[r] = S::mean_part(f[r]);
      row_sum<0, RB, MAXT>(mu, sm, buf);
#pragma unroll
      for (int r = 0; r < RB; ++r) mu[r] *= inv_c;
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) q[r] = S::var_part(f[r], mu[r], have);
    row_sum<0, RB, MAXT>(q, sm, buf);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r;
      if (row >= R.rows) continue;
      const float rs = 1.0f / sqrtf(q[r] * inv_c + eps);
      uint4* dst = reinterpret_cast<uint4*>(y + row * R.C) + t;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < have) __stcs(dst + u * T_row, S::out(f[r] + u * S::P, rs, wr + u * S::P, br + u * S::P));
      if (t == 0) {
        if (!RMS && mean != nullptr) mean[row] = mu[r];
        if (rstd != nullptr) rstd[row] = rs;
      }
    }
  }
  copy_wait<0>();
}

// Column sums of this CTA's rows go to part[blockIdx][0 or 1][C]; the rows of
// one CTA are summed per thread in order, then over the CTA's row slots in
// order, then norm_reduce_kernel adds the CTAs in order: no atomics.
constexpr int kShortDepth = 4;
template <typename T, int L, int U, int RB, bool RMS>
__global__ void __launch_bounds__(kWarpThreads, U == 4 ? 1 : 2)
norm_bwd_kernel(const Rows R, const T* __restrict__ dy, const T* __restrict__ x, int64_t x_stride,
                const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                T* __restrict__ dx, int64_t dx_stride, float* __restrict__ part, int with_db) {
  using S = Share<T, U, RMS>;
  constexpr int E = S::E;
  constexpr int K = RMS ? RB : 2 * RB;
  int buf = 0;
  const int t = threadIdx.x % L;
  constexpr int slots = kWarpThreads / L;
  const int slot = threadIdx.x / L;
  const int have = (R.V - t + L - 1) / L;
  f32x2 wr[U * S::P], dw[U * S::P], db[U * S::P];
  S::params(w, 1.f, t, L, R.V, wr);
#pragma unroll
  for (int i = 0; i < U * S::P; ++i) dw[i] = db[i] = pair(0.f, 0.f);
  const float inv_c = 1.0f / (float)R.C;
  const int64_t step = (int64_t)gridDim.x * slots * RB;
  // each thread copies its own vectors of the next batches into slots of its own
  extern __shared__ uint4 ring[];   // [kShortDepth][RB][x, dy][U][kWarpThreads]
  auto place = [&](int st, int r, int which, int u) {
    return ring + (((st * RB + r) * 2 + which) * U + u) * kWarpThreads + threadIdx.x;
  };
  auto fetch = [&](int64_t base, int st) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      if (row < R.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + R.at(row, x_stride)) + t;
        const uint4* gsrc = reinterpret_cast<const uint4*>(dy + row * R.C) + t;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < have) {
            copy_async16(place(st, r, 0, u), src + u * L);
            copy_async16(place(st, r, 1, u), gsrc + u * L);
          }
      }
    }
    copy_commit();
  };
  float mu_n[RB], rs_n[RB];   // the next batch's statistics
  auto stats = [&](int64_t base) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      mu_n[r] = !RMS && row < R.rows ? mean[row] : 0.f;
      rs_n[r] = row < R.rows ? rstd[row] : 0.f;
    }
  };
  const int64_t first = (int64_t)blockIdx.x * slots * RB;
#pragma unroll
  for (int s = 0; s < kShortDepth - 1; ++s) fetch(first + s * step, s);
  stats(first);
  int st = 0;
  for (int64_t base = first; base < R.rows; base += step, st = st + 1 == kShortDepth ? 0 : st + 1) {
    fetch(base + (kShortDepth - 1) * step, st == 0 ? kShortDepth - 1 : st - 1);
    copy_wait<kShortDepth - 1>();
    uint4 xv[RB][U], gv[RB][U];
    f32x2 h[RB][U * S::P], g[RB][U * S::P];
    float mu[RB], rs[RB], s[K];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      mu[r] = mu_n[r];
      rs[r] = rs_n[r];
      const bool ok = base + r * slots + slot < R.rows;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xv[r][u] = ok && u < have ? *place(st, r, 0, u) : make_uint4(0, 0, 0, 0);
        gv[r][u] = ok && u < have ? *place(st, r, 1, u) : make_uint4(0, 0, 0, 0);
      }
    }
    stats(base + step);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float sg;
      S::grad_part(xv[r], gv[r], mu[r], rs[r], wr, dw, db, h[r], g[r], s[RMS ? r : 2 * r], sg);
      if (!RMS) s[RMS ? 0 : 2 * r + 1] = sg;
    }
    row_sum<L, K>(s, nullptr, buf);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      if (row >= R.rows) continue;
      const float mgx = s[RMS ? r : 2 * r] * inv_c, mg = RMS ? 0.f : s[RMS ? 0 : 2 * r + 1] * inv_c;
      uint4* dst = reinterpret_cast<uint4*>(dx + R.at(row, dx_stride)) + t;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < have)
          __stcs(dst + u * L, S::grad_out(h[r] + u * S::P, g[r] + u * S::P, rs[r], mg, mgx));
    }
  }
  copy_wait<0>();
  if (part == nullptr) return;
  // the CTA's row slots, one vector column at a time
  float* out = part + (int64_t)blockIdx.x * 2 * R.C;
  __shared__ float col[kWarpThreads][E + 1];
  for (int which = 0; which < (with_db ? 2 : 1); ++which)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < S::P; ++i) {
        const float2 v = both(which ? db[u * S::P + i] : dw[u * S::P + i]);
        col[threadIdx.x][2 * i] = v.x;
        col[threadIdx.x][2 * i + 1] = v.y;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < L * E; i += kWarpThreads) {
        const int tt = i / E, e = i % E, v = tt + u * L;
        if (v >= R.V) continue;
        float sum = 0.f;
        for (int sl = 0; sl < slots; ++sl) sum += col[sl * L + tt][e];
        out[which * R.C + v * E + e] = sum;
      }
    }
}

// Longer rows: a CTA per row with the forward's ring, of x and dy.
template <typename T, int U, bool RMS, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
norm_bwd_cta_kernel(const Rows R, const T* __restrict__ dy, const T* __restrict__ x, int64_t x_stride,
                    const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                    T* __restrict__ dx, int64_t dx_stride, float* __restrict__ part, int with_db, int depth) {
  using S = Share<T, U, RMS>;
  constexpr int E = S::E;
  constexpr int K = RMS ? 1 : 2;
  extern __shared__ uint4 ring[];   // [depth][x, dy][U][T_row]
  __shared__ __align__(16) float sm[2 * kMaxWarps * K];
  int buf = 0;
  const int t = threadIdx.x, T_row = blockDim.x;
  const int have = (R.V - t + T_row - 1) / T_row;
  f32x2 wr[U * S::P], dw[U * S::P], db[U * S::P];
  S::params(w, 1.f, t, T_row, R.V, wr);
#pragma unroll
  for (int i = 0; i < U * S::P; ++i) dw[i] = db[i] = pair(0.f, 0.f);
  for (int i = t; i < 2 * kMaxWarps * K; i += T_row) sm[i] = 0.f;
  __syncthreads();
  const float inv_c = 1.0f / (float)R.C;
  auto slot = [&](int st, int which, int u) { return ring + ((st * 2 + which) * U + u) * T_row + t; };
  auto fetch = [&](int64_t row, int st) {
    if (row < R.rows) {
      const uint4* src = reinterpret_cast<const uint4*>(x + R.at(row, x_stride)) + t;
      const uint4* gsrc = reinterpret_cast<const uint4*>(dy + row * R.C) + t;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < have) {
          copy_async16(slot(st, 0, u), src + u * T_row);
          copy_async16(slot(st, 1, u), gsrc + u * T_row);
        }
    }
    copy_commit();
  };
  const int64_t step = gridDim.x;
  for (int s = 0; s < depth - 1; ++s) fetch(blockIdx.x + s * step, s);
  int st = 0;
  float mu_n = 0.f, rs_n = 0.f;   // the next row's statistics
  if (blockIdx.x < R.rows) {
    mu_n = RMS ? 0.f : mean[blockIdx.x];
    rs_n = rstd[blockIdx.x];
  }
  for (int64_t row = blockIdx.x; row < R.rows; row += step, st = st + 1 == depth ? 0 : st + 1) {
    fetch(row + (depth - 1) * step, st == 0 ? depth - 1 : st - 1);
    copy_wait(depth - 1);
    const float mu = mu_n, rs = rs_n;
    if (row + step < R.rows) {
      mu_n = RMS ? 0.f : mean[row + step];
      rs_n = rstd[row + step];
    }
    uint4 xv[U], gv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xv[u] = u < have ? *slot(st, 0, u) : make_uint4(0, 0, 0, 0);
      gv[u] = u < have ? *slot(st, 1, u) : make_uint4(0, 0, 0, 0);
    }
    f32x2 h[U * S::P], g[U * S::P];
    float s[K], sg;
    S::grad_part(xv, gv, mu, rs, wr, dw, db, h, g, s[0], sg);
    if (!RMS) s[K - 1] = sg;
    row_sum<0, K, MAXT>(s, sm, buf);
    const float mgx = s[0] * inv_c, mg = RMS ? 0.f : s[K - 1] * inv_c;
    uint4* dst = reinterpret_cast<uint4*>(dx + R.at(row, dx_stride)) + t;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < have)
        __stcs(dst + u * T_row, S::grad_out(h + u * S::P, g + u * S::P, rs, mg, mgx));
  }
  copy_wait<0>();
  if (part == nullptr) return;
  float* out = part + (int64_t)blockIdx.x * 2 * R.C;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < have)
#pragma unroll
      for (int i = 0; i < S::P; ++i) {
        const int c = (t + u * T_row) * E + 2 * i;
        *reinterpret_cast<float2*>(out + c) = both(dw[u * S::P + i]);
        if (with_db) *reinterpret_cast<float2*>(out + R.C + c) = both(db[u * S::P + i]);
      }
}

// dw[c] = sum over G CTAs of part[g][0][c], db likewise: 32 columns per CTA,
// 32 slices of the CTAs each summed in order, then the slices in order.
__global__ void __launch_bounds__(1024)
norm_reduce_kernel(const float* __restrict__ part, int G, int C, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sm[32][33];
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  float s = 0.f;
  if (c < C) {
    const float* p = part + (int64_t)blockIdx.y * C + c;
#pragma unroll 4
    for (int g = sl; g < G; g += 32) s += p[(int64_t)g * 2 * C];
  }
  sm[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0 && c < C) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sm[i][threadIdx.x];
    out[c] = t;
  }
}

Rows rows_of(const Dims& s, bool head) {
  Rows R;
  R.groups = head ? s.H : 1;
  R.C = head ? s.d : s.H * s.d;
  R.V = R.C * s.elem / 16;
  R.rows = (int64_t)s.B * s.N * R.groups;
  return R;
}

// CTAs of the backward (its workspace holds one pair of column sums each), never
// more than the batches of rows. `sms` is an upper bound on the SM count.
constexpr int kSmBound = 160;
int lanes_of(const Rows& R) { return R.V <= 8 ? 4 : R.V <= 16 ? 8 : R.V <= 32 ? 16 : 32; }
int64_t bwd_ctas(const Rows& R, int sms) {
  const bool cta = R.V > 128;
  const int64_t slots = cta ? 1 : kWarpThreads / lanes_of(R);
  const int64_t need = (R.rows + slots - 1) / slots, cap = (int64_t)sms * 2;
  return need < cap ? need : cap;
}

bool set_smem(const void* kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <typename T, bool RMS>
struct Go {
  template <int U>
  static constexpr int longest() { return 16384 / (U * Vec<T>::E); }   // threads of a row of 16,384 values
  template <int L, int U, int RB>
  static bool fwd(const Rows& R, const void* x, int64_t xs, const float* w, const float* b, float eps, void* y,
                  float* mean, float* rstd, int sms, cudaStream_t st) {
    constexpr int64_t slots = kWarpThreads / L;
    int64_t grid = (R.rows + slots * RB - 1) / (slots * RB);
    if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
    norm_fwd_kernel<T, L, U, RB, RMS><<<(unsigned)grid, kWarpThreads, 0, st>>>(R, (const T*)x, xs, w, b, eps, (T*)y,
                                                                               mean, rstd);
    return true;
  }
  template <int U, int MAXT, int MINB>
  static bool fwd_cta(const Rows& R, const void* x, int64_t xs, const float* w, const float* b, float eps, void* y,
                      float* mean, float* rstd, int sms, cudaStream_t st) {
    const int threads = 32 * ((R.V + 32 * U - 1) / (32 * U));
    // rows per step: two share the two barriers of a layer norm (131 us against 135 for
    // one, 30,720 rows of 5,120 bf16 values, cold cache); with the one barrier of an
    // RMS norm one row at a time is faster (124 us against 130)
    constexpr int RB = U == 4 || RMS ? 1 : 2, kThreads = U == 4 ? longest<U>() : MAXT;
    const size_t step = (size_t)RB * U * threads * 16;
    const int depth = ring_depth(step, MINB);
    const size_t smem = step * depth;
    auto kern = norm_fwd_cta_kernel<T, U, RB, RMS, kThreads, MINB>;
    if (!set_smem((const void*)kern, smem)) return false;
    int per = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, smem) != cudaSuccess || per < 1) return false;
    int64_t grid = (R.rows + RB - 1) / RB;
    if (grid > (int64_t)sms * per) grid = (int64_t)sms * per;
    kern<<<(unsigned)grid, threads, smem, st>>>(R, (const T*)x, xs, w, b, eps, (T*)y, mean, rstd, depth);
    return true;
  }
  template <int L, int U, int RB>
  static bool bwd(const Rows& R, const void* dy, const void* x, int64_t xs, const float* w, const float* mean,
                  const float* rstd, void* dx, int64_t dxs, float* part, int with_db, int64_t grid, cudaStream_t st) {
    const size_t smem = (size_t)kShortDepth * RB * 2 * U * kWarpThreads * 16;   // 64 KB with two vectors a thread
    auto kern = norm_bwd_kernel<T, L, U, RB, RMS>;
    if (!set_smem((const void*)kern, smem)) return false;
    kern<<<(unsigned)grid, kWarpThreads, smem, st>>>(
        R, (const T*)dy, (const T*)x, xs, w, mean, rstd, (T*)dx, dxs, part, with_db);
    return true;
  }
  template <int U, int MAXT, int MINB>
  static bool bwd_cta(const Rows& R, const void* dy, const void* x, int64_t xs, const float* w, const float* mean,
                      const float* rstd, void* dx, int64_t dxs, float* part, int with_db, int64_t grid,
                      cudaStream_t st) {
    const int threads = 32 * ((R.V + 32 * U - 1) / (32 * U));
    const size_t step = (size_t)2 * U * threads * 16;
    const int depth = ring_depth(step, MINB);
    constexpr int kThreads = U == 4 ? longest<U>() : MAXT;
    auto kern = norm_bwd_cta_kernel<T, U, RMS, kThreads, MINB>;
    if (!set_smem((const void*)kern, step * depth)) return false;
    kern<<<(unsigned)grid, threads, step * depth, st>>>(R, (const T*)dy, (const T*)x, xs, w, mean, rstd, (T*)dx, dxs,
                                                        part, with_db, depth);
    return true;
  }
};

// Threads per row and vectors per thread by the row's length in 16-byte vectors:
// up to 128 vectors part of a warp, longer rows a CTA with two vectors a
// thread, four beyond 1,024.
#define NORM_ROWS(WARP, CTA)                     \
  do {                                           \
    if (R.V <= 8) WARP(4, 2, 2);                 \
    else if (R.V <= 16) WARP(8, 2, 2);           \
    else if (R.V <= 32) WARP(16, 2, 2);          \
    else if (R.V <= 64) WARP(32, 2, 2);          \
    else if (R.V <= 128) WARP(32, 4, 1);         \
    else if (R.V <= 640) CTA(2, 320, 2);         \
    else if (R.V <= 1024) CTA(2, 512, 1);        \
    else CTA(4, 1024, 1);                        \
  } while (0)

}  // namespace

size_t norm_ws(const Dims& s, bool head) {
  const Rows R = rows_of(s, head);
  return (size_t)bwd_ctas(R, kSmBound) * 2 * R.C * sizeof(float);
}

sparsp_status_t launch_norm_fwd(const Dims& s, bool head, bool rms, const void* x, int64_t x_stride, const float* w,
                                const float* b, float eps, void* y, float* mean, float* rstd, cudaStream_t st) {
  const Rows R = rows_of(s, head);
  const int sms = device_sm_count();
  if (sms <= 0) return SPARSP_ERR_CUDA;
  bool ok = false;
#define NORM_TYPED(CALL)                                                  \
  do {                                                                    \
    if (s.dtype == SPARSP_F32) ok = rms ? Go<float, true>::CALL : Go<float, false>::CALL; \
    else ok = rms ? Go<__nv_bfloat16, true>::CALL : Go<__nv_bfloat16, false>::CALL;      \
  } while (0)
#define NORM_WARP(L, U, RB) NORM_TYPED(template fwd<L NORM_COMMA U NORM_COMMA RB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st))
#define NORM_CTA(U, MAXT, MINB) NORM_TYPED(template fwd_cta<U NORM_COMMA MAXT NORM_COMMA MINB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st))
#define NORM_COMMA ,
  NORM_ROWS(NORM_WARP, NORM_CTA);
#undef NORM_WARP
#undef NORM_CTA
  if (!ok) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_norm_bwd(const Dims& s, bool head, bool rms, const void* dy, const void* x, int64_t x_stride,
                                const float* w, const float* mean, const float* rstd, void* dx, int64_t dx_stride,
                                float* dw, float* db, void* ws, cudaStream_t st) {
  const Rows R = rows_of(s, head);
  int sms = device_sm_count();
  if (sms <= 0) return SPARSP_ERR_CUDA;
  if (sms > kSmBound) sms = kSmBound;
  const int64_t grid = bwd_ctas(R, sms);
  float* part = dw != nullptr || db != nullptr ? (float*)ws : nullptr;
  const int with_db = db != nullptr;
  bool ok = false;
#define NORM_WARP(L, U, RB)                                                                                          \
  NORM_TYPED(template bwd<L NORM_COMMA U NORM_COMMA 1>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part,        \
                                                        with_db, grid, st))
#define NORM_CTA(U, MAXT, MINB)                                                                                      \
  NORM_TYPED(template bwd_cta<U NORM_COMMA MAXT NORM_COMMA MINB>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part, \
                                                                 with_db, grid, st))
  NORM_ROWS(NORM_WARP, NORM_CTA);
#undef NORM_WARP
#undef NORM_CTA
#undef NORM_TYPED
#undef NORM_COMMA
  if (!ok) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  if (part != nullptr) {
    dim3 g((R.C + 31) / 32, with_db ? 2 : 1);
    norm_reduce_kernel<<<g, 1024, 0, st>>>(part, (int)grid, R.C, dw, db);
    SPARSP_LAUNCH_CHECK();
  }
  return SPARSP_OK;
}

}  // namespace sparsp
