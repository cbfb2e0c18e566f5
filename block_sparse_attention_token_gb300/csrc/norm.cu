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
// shared-memory exchange per batch of rows (longer rows, a CTA per row).
#include "common.cuh"

namespace sparsp {
namespace {

constexpr int kWarpThreads = 256;   // CTA of the shuffle kernels
constexpr int kMaxWarps = 32;

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
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
struct Vec<float> {
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

// Rows are numbered token-major: row = token * groups + group, with one group
// of C = H*d values per token or H groups of C = d values. A strided tensor
// has `stride` elements between tokens; the others are contiguous.
struct Rows {
  int64_t rows;
  int groups;   // 1, or H
  int C;        // values per row
  int V;        // 16-byte vectors per row
  __device__ __forceinline__ int64_t at(int64_t row, int64_t stride) const {
    const int64_t tok = groups == 1 ? row : (int64_t)((uint32_t)row / (uint32_t)groups);
    return tok * stride + (row - tok * groups) * C;
  }
};

// Threads of a CTA at most: rows of up to 16,384 values, U vectors a thread.
template <typename T, int L, int U>
constexpr int max_threads() {
  return L != 0 ? kWarpThreads : U == 2 ? 512 : 16384 / (Vec<T>::E * U);
}

// Sum of K values over the threads that share a row: L lanes of a warp, or the
// whole CTA (L = 0) through shared memory, in a fixed order. `buf` alternates
// between calls so that one barrier per call is enough.
template <int L, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* sm, int& buf) {
#pragma unroll
  for (int off = (L == 0 ? 32 : L) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if (L == 0) {
    float* s = sm + buf * (kMaxWarps * K);
    buf ^= 1;
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[warp * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = 0.f;
      for (int w = 0; w < nw; ++w) t += s[w * K + k];
      v[k] = t;
    }
  }
}

template <typename T, int L, int U, int RB, bool RMS>
__global__ void __launch_bounds__(max_threads<T, L, U>())
norm_fwd_kernel(const Rows R, const T* __restrict__ x, int64_t x_stride, const float* __restrict__ w,
                const float* __restrict__ b, float eps, T* __restrict__ y, float* __restrict__ mean,
                float* __restrict__ rstd) {
  using X = Vec<T>;
  constexpr int E = X::E;
  __shared__ float sm[L == 0 ? 2 * kMaxWarps * RB : 1];
  int buf = 0;
  const int T_row = L == 0 ? blockDim.x : L;             // threads of a row
  const int t = L == 0 ? threadIdx.x : threadIdx.x % L;  // this thread's place in its row
  const int slots = L == 0 ? 1 : blockDim.x / L, slot = L == 0 ? 0 : threadIdx.x / L;
  float wr[U * E], br[U * E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int v = t + u * T_row, c = v * E + e;
      wr[u * E + e] = v < R.V && w != nullptr ? w[c] : 1.f;
      br[u * E + e] = v < R.V && b != nullptr ? b[c] : 0.f;
    }
  const float inv_c = 1.0f / (float)R.C;
  const int64_t step = (int64_t)gridDim.x * slots * RB;
  for (int64_t base = (int64_t)blockIdx.x * slots * RB; base < R.rows; base += step) {
    uint4 xv[RB][U];
    float s[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      const uint4* src = reinterpret_cast<const uint4*>(x + (row < R.rows ? R.at(row, x_stride) : 0));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = t + u * T_row;
        xv[r][u] = row < R.rows && v < R.V ? __ldcs(src + v) : make_uint4(0, 0, 0, 0);
      }
    }
    float mu[RB], q[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) mu[r] = 0.f;
    if (!RMS) {
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        s[r] = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[E];
          X::unpack(xv[r][u], f);
#pragma unroll
          for (int e = 0; e < E; ++e) s[r] += f[e];
        }
      }
      row_sum<L, RB>(s, sm, buf);
#pragma unroll
      for (int r = 0; r < RB; ++r) mu[r] = s[r] * inv_c;
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      q[r] = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[E];
        X::unpack(xv[r][u], f);
        if (t + u * T_row < R.V)   // a vector past the row holds zeros, not the mean
#pragma unroll
          for (int e = 0; e < E; ++e) q[r] += (f[e] - mu[r]) * (f[e] - mu[r]);
      }
    }
    row_sum<L, RB>(q, sm, buf);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      if (row >= R.rows) continue;
      const float rs = 1.0f / sqrtf(q[r] * inv_c + eps);
      uint4* dst = reinterpret_cast<uint4*>(y + row * R.C);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = t + u * T_row;
        if (v >= R.V) continue;
        float f[E];
        X::unpack(xv[r][u], f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = (f[e] - mu[r]) * rs * wr[u * E + e] + br[u * E + e];
        __stcs(dst + v, X::pack(f));
      }
      if (t == 0) {
        if (!RMS && mean != nullptr) mean[row] = mu[r];
        if (rstd != nullptr) rstd[row] = rs;
      }
    }
  }
}

// Column sums of this CTA's rows go to part[blockIdx][0 or 1][C]; the rows of
// one CTA are summed per thread in order, then over the CTA's row slots in
// order, then norm_reduce_kernel adds the CTAs in order: no atomics.
template <typename T, int L, int U, int RB, bool RMS>
__global__ void __launch_bounds__(max_threads<T, L, U>())
norm_bwd_kernel(const Rows R, const T* __restrict__ dy, const T* __restrict__ x, int64_t x_stride,
                const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
                T* __restrict__ dx, int64_t dx_stride, float* __restrict__ part, int with_db) {
  using X = Vec<T>;
  constexpr int E = X::E;
  constexpr int K = RMS ? RB : 2 * RB;
  __shared__ float sm[L == 0 ? 2 * kMaxWarps * K : 1];
  int buf = 0;
  const int T_row = L == 0 ? blockDim.x : L;
  const int t = L == 0 ? threadIdx.x : threadIdx.x % L;
  const int slots = L == 0 ? 1 : blockDim.x / L, slot = L == 0 ? 0 : threadIdx.x / L;
  float wr[U * E], dw[U * E], db[U * E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int v = t + u * T_row, c = v * E + e;
      wr[u * E + e] = v < R.V && w != nullptr ? w[c] : 1.f;
      dw[u * E + e] = db[u * E + e] = 0.f;
    }
  const float inv_c = 1.0f / (float)R.C;
  const int64_t step = (int64_t)gridDim.x * slots * RB;
  for (int64_t base = (int64_t)blockIdx.x * slots * RB; base < R.rows; base += step) {
    uint4 xv[RB][U], gv[RB][U];
    float mu[RB], rs[RB], s[K];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      const bool ok = row < R.rows;
      const uint4* src = reinterpret_cast<const uint4*>(x + (ok ? R.at(row, x_stride) : 0));
      const uint4* gsrc = reinterpret_cast<const uint4*>(dy + (ok ? row * R.C : 0));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = t + u * T_row;
        const bool in = ok && v < R.V;
        xv[r][u] = in ? __ldcs(src + v) : make_uint4(0, 0, 0, 0);
        gv[r][u] = in ? __ldcs(gsrc + v) : make_uint4(0, 0, 0, 0);
      }
      mu[r] = !RMS && ok ? mean[row] : 0.f;
      rs[r] = ok ? rstd[row] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float sg = 0.f, sgx = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[E], g[E];
        X::unpack(xv[r][u], f);
        X::unpack(gv[r][u], g);   // zero past the row and past the last row
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xh = (f[e] - mu[r]) * rs[r], gw = g[e] * wr[u * E + e];
          dw[u * E + e] += g[e] * xh;
          db[u * E + e] += g[e];
          sg += gw;
          sgx += gw * xh;
        }
      }
      s[RMS ? r : 2 * r] = sgx;
      if (!RMS) s[RMS ? 0 : 2 * r + 1] = sg;
    }
    row_sum<L, K>(s, sm, buf);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = base + r * slots + slot;
      if (row >= R.rows) continue;
      const float mgx = s[RMS ? r : 2 * r] * inv_c, mg = RMS ? 0.f : s[RMS ? 0 : 2 * r + 1] * inv_c;
      uint4* dst = reinterpret_cast<uint4*>(dx + R.at(row, dx_stride));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = t + u * T_row;
        if (v >= R.V) continue;
        float f[E], g[E];
        X::unpack(xv[r][u], f);
        X::unpack(gv[r][u], g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xh = (f[e] - mu[r]) * rs[r];
          f[e] = rs[r] * (g[e] * wr[u * E + e] - mg - xh * mgx);
        }
        __stcs(dst + v, X::pack(f));
      }
    }
  }
  if (part == nullptr) return;
  float* out = part + (int64_t)blockIdx.x * 2 * R.C;
  if (L == 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = t + u * T_row;
      if (v >= R.V) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        out[v * E + e] = dw[u * E + e];
        if (with_db) out[R.C + v * E + e] = db[u * E + e];
      }
    }
  } else {
    // the CTA's row slots, one vector column at a time
    __shared__ float col[kWarpThreads][E + 1];
    for (int which = 0; which < (with_db ? 2 : 1); ++which)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) col[threadIdx.x][e] = which ? db[u * E + e] : dw[u * E + e];
        __syncthreads();
        for (int i = threadIdx.x; i < T_row * E; i += blockDim.x) {
          const int tt = i / E, e = i % E, v = tt + u * T_row;
          if (v >= R.V) continue;
          float sum = 0.f;
          for (int sl = 0; sl < slots; ++sl) sum += col[sl * T_row + tt][e];
          out[which * R.C + v * E + e] = sum;
        }
      }
  }
}

// dw[c] = sum over G CTAs of part[g][0][c], db likewise: 32 columns per CTA,
// 8 slices of the CTAs each summed in order, then the slices in order.
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float* __restrict__ part, int G, int C, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sm[8][33];
  float* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  float s = 0.f;
  if (c < C) {
    const float* p = part + (int64_t)blockIdx.y * C + c;
#pragma unroll 8
    for (int g = sl; g < G; g += 8) s += p[(int64_t)g * 2 * C];
  }
  sm[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0 && c < C) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sm[i][threadIdx.x];
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

// CTAs of the backward (its workspace holds one pair of column sums each): one
// or two per SM for CTA rows, eight for shuffle rows, never more than the
// batches of rows. `sms` is an upper bound on the SM count.
constexpr int kSmBound = 160;
int64_t bwd_ctas(const Rows& R, int sms) {
  const bool cta = R.V > 128;
  const int64_t per = cta ? 2 : 8;
  const int64_t slots = cta ? 1 : kWarpThreads / (R.V <= 8 ? 8 : R.V <= 16 ? 16 : 32);
  const int64_t need = (R.rows + slots - 1) / slots;
  return need < per * sms ? need : per * sms;
}

template <typename T, bool RMS>
struct Go {
  template <int L, int U, int RB>
  static void fwd(const Rows& R, const void* x, int64_t xs, const float* w, const float* b, float eps, void* y,
                  float* mean, float* rstd, int sms, cudaStream_t st) {
    const int threads = L == 0 ? 32 * ((R.V + 32 * U - 1) / (32 * U)) : kWarpThreads;
    const int64_t slots = L == 0 ? 1 : kWarpThreads / (L == 0 ? 1 : L);
    int64_t grid = (R.rows + slots * RB - 1) / (slots * RB);
    const int64_t cap = (int64_t)sms * (L == 0 ? (2048 / threads) : 8);
    if (grid > cap) grid = cap;
    norm_fwd_kernel<T, L, U, RB, RMS><<<(unsigned)grid, threads, 0, st>>>(R, (const T*)x, xs, w, b, eps, (T*)y, mean,
                                                                          rstd);
  }
  template <int L, int U, int RB>
  static void bwd(const Rows& R, const void* dy, const void* x, int64_t xs, const float* w, const float* mean,
                  const float* rstd, void* dx, int64_t dxs, float* part, int with_db, int64_t grid, cudaStream_t st) {
    const int threads = L == 0 ? 32 * ((R.V + 32 * U - 1) / (32 * U)) : kWarpThreads;
    norm_bwd_kernel<T, L, U, RB, RMS><<<(unsigned)grid, threads, 0, st>>>(R, (const T*)dy, (const T*)x, xs, w, mean,
                                                                          rstd, (T*)dx, dxs, part, with_db);
  }
};

// Threads per row and vectors per thread by the row's length in 16-byte vectors:
// up to 128 vectors a quarter, half or whole warp; longer rows a CTA with two
// vectors a thread, four beyond 1,024.
#define NORM_ROWS(CALL)                          \
  do {                                           \
    if (R.V <= 8) CALL(8, 1, 4);                 \
    else if (R.V <= 16) CALL(16, 1, 4);          \
    else if (R.V <= 32) CALL(32, 1, 4);          \
    else if (R.V <= 64) CALL(32, 2, 2);          \
    else if (R.V <= 128) CALL(32, 4, 1);         \
    else if (R.V <= 1024) CALL(0, 2, 1);         \
    else CALL(0, 4, 1);                          \
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
#define NORM_FWD_CALL(L, U, RB)                                                                        \
  do {                                                                                                 \
    if (s.dtype == SPARSP_F32) {                                                                       \
      if (rms) Go<float, true>::fwd<L, U, RB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st);      \
      else Go<float, false>::fwd<L, U, RB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st);         \
    } else {                                                                                           \
      if (rms) Go<__nv_bfloat16, true>::fwd<L, U, RB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st); \
      else Go<__nv_bfloat16, false>::fwd<L, U, RB>(R, x, x_stride, w, b, eps, y, mean, rstd, sms, st); \
    }                                                                                                  \
  } while (0)
  NORM_ROWS(NORM_FWD_CALL);
#undef NORM_FWD_CALL
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
#define NORM_BWD_CALL(L, U, RB)                                                                                     \
  do {                                                                                                              \
    if (s.dtype == SPARSP_F32) {                                                                                    \
      if (rms) Go<float, true>::bwd<L, U, RB>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part, with_db, grid, st); \
      else Go<float, false>::bwd<L, U, RB>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part, with_db, grid, st);    \
    } else {                                                                                                        \
      if (rms) Go<__nv_bfloat16, true>::bwd<L, U, RB>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part, with_db, grid, st); \
      else Go<__nv_bfloat16, false>::bwd<L, U, RB>(R, dy, x, x_stride, w, mean, rstd, dx, dx_stride, part, with_db, grid, st);    \
    }                                                                                                               \
  } while (0)
  NORM_ROWS(NORM_BWD_CALL);
#undef NORM_BWD_CALL
  SPARSP_LAUNCH_CHECK();
  if (part != nullptr) {
    dim3 g((R.C + 31) / 32, with_db ? 2 : 1);
    norm_reduce_kernel<<<g, 256, 0, st>>>(part, (int)grid, R.C, dw, db);
    SPARSP_LAUNCH_CHECK();
  }
  return SPARSP_OK;
}

}  // namespace sparsp
