// The norm of every head's query and key row with the three-axis rotary positions in
// the same pass, over both tensors in one launch, forward and backward.
//
//   mean = sum x / d (0 for RMS), var = sum (x - mean)^2 / d, rstd = 1 / sqrt(var + eps),
//   xh = (x - mean) rstd, y = R(w xh + b), R the rotation of the row's token;
//   backward, with g = R^T dy and gw = g w:
//   dx = rstd (gw - [mean_d(gw)] - xh mean_d(gw xh)), dw = sum_rows g xh, db = sum_rows g
// ([.] is left out for RMS). The variance is taken about the mean in a second sweep over
// registers. The backward takes the statistics from x again, which it reads anyway, so
// that nothing but x has to be kept. The normed row is turned before it is rounded.
//
// Bound by HBM: each row is read and written once (the backward reads two). A CTA takes
// a granule of tokens and several heads of one tensor. A row is spread over few lanes
// (UPR), so its sums are shuffles; a thread keeps the (cos, sin) of its tokens and
// columns, and its columns of w and b, in registers and sweeps the heads, whose vectors are
// copied into shared-memory slots of its own some heads ahead (cp.async).
#include "rows.cuh"

namespace sparsp {
namespace {

template <typename T, int D, int GR, bool HALF>
struct Cfg {
  static constexpr int E = Row16<T>::E;                        // values per 16-byte vector
  static constexpr int NV = HALF ? 2 : 1;                      // vectors of a unit
  static constexpr int NE = NV * E;                            // values of a unit
  static constexpr int NP = NE / 2;                            // pairs of a unit
  static constexpr int UPR = D / NE;                           // units (lanes) per row
  static constexpr int VECS = GR * D / E;                      // vectors of a granule
  static constexpr int THREADS = VECS >= 2048 ? 512 : 256;      // 4 to 8 vectors a thread
  static constexpr int U = GR * UPR / THREADS;                 // units (rows) per thread
  static constexpr int kRowStep = THREADS / UPR;
  static_assert(UPR <= 32 && THREADS % UPR == 0 && U >= 1 && U * THREADS == GR * UPR, "granule split");
};

// Which tokens a granule holds: GR tokens of a tile (tile order on one side, or tile
// means), or GR raster tokens of all batch elements in a row, the last granule short.
struct Tokens {
  RasterMap rm;
  int64_t total;    // B * N
  int linear;
  int bt;           // tokens per tile
};

struct Fwd {
  const void* in;
  int64_t in_stride;
  void* out;
  int64_t out_stride;
  const float *w, *b;
  float* means;
  int heads, groups;
};
struct Bwd {
  const void *dy, *x;
  int64_t dy_stride, x_stride;
  void* dx;
  int64_t dx_stride;
  const float* w;
  float *dw, *db;
  int heads, groups;
};

// tok[o]: flat raster token (b * N + n, -1 past the end) and its table row per axis (-1: not turned).
template <int GR, int THREADS>
__device__ __forceinline__ void locate(int4* tok, const Tokens& t, const RopeArgs& a, int32_t* d_status) {
  const RasterMap& rm = t.rm;
  for (int o = threadIdx.x; o < GR; o += THREADS) {
    int64_t flat;
    int p[3];
    if (t.linear) {
      flat = (int64_t)blockIdx.x * GR + o;
      const int n = (int)(flat % rm.N);
      p[0] = n / (rm.Y * rm.X);
      p[1] = n / rm.X % rm.Y;
      p[2] = n % rm.X;
    } else {
      const int per = t.bt / GR, nb = (int)(rm.N / t.bt), tile = blockIdx.x / per;
      const int j = tile % nb, oo = (int)(blockIdx.x % per) * GR + o;
      const int bx = j % rm.nX, by = (j / rm.nX) % rm.nY, bt = j / (rm.nX * rm.nY);
      const int tbc = rm.tb * rm.tc, it = oo / tbc, rem = oo - it * tbc, iy = rem / rm.tc, ix = rem - iy * rm.tc;
      p[0] = bt * rm.ta + it;
      p[1] = by * rm.tb + iy;
      p[2] = bx * rm.tc + ix;
      flat = (int64_t)(tile / nb) * rm.N + ((int64_t)p[0] * rm.Y + p[1]) * rm.X + p[2];
    }
    if (flat >= t.total) {
      tok[o] = make_int4(-1, -1, -1, -1);
      continue;
    }
    if (a.pos != nullptr)
#pragma unroll
      for (int ax = 0; ax < 3; ++ax) {
        p[ax] = a.pos[flat * 3 + ax];
        if (a.cols[ax] > 0 && (p[ax] < 0 || p[ax] >= a.extent[ax])) {
          report(d_status, SPARSP_ERR_DATA);
          p[ax] = -1;
        }
      }
    tok[o] = make_int4((int)flat, p[0], p[1], p[2]);
  }
}

// (cos, +-sin) of pair `pair` of a token.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, const int4& tk, int pair) {
  int i = pair, ax = 0;
  if (i >= a.cols[0] / 2) { i -= a.cols[0] / 2; ax = 1; }
  if (ax == 1 && i >= a.cols[1] / 2) { i -= a.cols[1] / 2; ax = 2; }
  const int p = ax == 0 ? tk.y : ax == 1 ? tk.z : tk.w;
  float2 v = make_float2(1.f, 0.f);
  if (i < a.cols[ax] / 2 && p >= 0) v = __ldg(a.table + a.base[ax] + (int64_t)p * (a.cols[ax] / 2) + i);
  return make_float2(v.x, v.y * a.sign);
}

template <bool HALF, int E, int NP>
__device__ __forceinline__ void turn(float* f, const float2* cs) {
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    float& x = f[HALF ? k : 2 * k];
    float& y = f[HALF ? E + k : 2 * k + 1];
    const float r = x * cs[k].x - y * cs[k].y;
    y = x * cs[k].y + y * cs[k].x;
    x = r;
  }
}

// Sums over the UPR lanes that share a row.
template <int UPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K]) {
#pragma unroll
  for (int off = UPR / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
}

constexpr int kDepth = 3;   // heads in flight per CTA

template <typename T, int D, int GR, bool HALF, bool POOL>
__global__ void __launch_bounds__(Cfg<T, D, GR, HALF>::THREADS)
norm_rope_fwd_kernel(const Fwd q, const Fwd k, const Tokens tk, const RopeArgs a, bool rms, float eps, bool out_blocked,
                     int heads_per_cta, int32_t* d_status) {
  using C = Cfg<T, D, GR, HALF>;
  using X = Row16<T>;
  constexpr int E = C::E, NE = C::NE;
  __shared__ int4 tok[GR];
  constexpr int kPart = C::THREADS / 32 * C::UPR;
  __shared__ float part[POOL ? 2 : 1][POOL ? kPart : 1][POOL ? NE + 1 : 1];
  extern __shared__ uint4 ring[];   // [min(kDepth, heads)][U][NV][THREADS]
  const bool is_q = blockIdx.y < q.groups;
  const Fwd& t = is_q ? q : k;
  const int h0 = (is_q ? blockIdx.y : blockIdx.y - q.groups) * heads_per_cta, h1 = min(t.heads, h0 + heads_per_cta);
  const T* in = static_cast<const T*>(t.in);
  T* out = static_cast<T*>(t.out);
  locate<GR, C::THREADS>(tok, tk, a, d_status);
  __syncthreads();
  const int c0 = threadIdx.x % C::UPR, o0 = threadIdx.x / C::UPR;   // this thread's unit column, its first row
  float2 cs[C::U][C::NP];
  int64_t flat[C::U];
#pragma unroll
  for (int u = 0; u < C::U; ++u) {
    const int4 w = tok[o0 + u * C::kRowStep];
    flat[u] = w.x;
#pragma unroll
    for (int i = 0; i < C::NP; ++i) cs[u][i] = turn_of(a, w, c0 * C::NP + i);
  }
  float w[NE], b[NE];
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    const int c = c0 * E + (e / E) * (D / 2) + e % E;
    w[e] = t.w != nullptr ? __ldg(t.w + c) : 1.f;
    b[e] = t.b != nullptr ? __ldg(t.b + c) : 0.f;
  }
  // rows of tile order: those of head h of this granule's batch element start at blocked0(h)
  const int64_t N = tk.rm.N;
  const int64_t at = (int64_t)blockIdx.x * GR, batch = at / N, row0 = at - batch * N;
  auto place = [&](int st, int u, int v) { return ring + ((st * C::U + u) * C::NV + v) * C::THREADS + threadIdx.x; };
  auto fetch = [&](int h, int st) {
    if (h < h1) {
#pragma unroll
      for (int u = 0; u < C::U; ++u)
        if (flat[u] >= 0) {
          const T* src = in + flat[u] * t.in_stride + (int64_t)h * D + c0 * E;
#pragma unroll
          for (int v = 0; v < C::NV; ++v) copy_async16(place(st, u, v), src + v * (D / 2));
        }
    }
    copy_commit();
  };
  for (int s = 0; s < kDepth - 1; ++s) fetch(h0 + s, s);
  int st = 0;
  for (int h = h0; h < h1; ++h, st = st + 1 == kDepth ? 0 : st + 1) {
    fetch(h + kDepth - 1, st == 0 ? kDepth - 1 : st - 1);   // the slots of the head before
    copy_wait<kDepth - 1>();
    float acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = 0.f;
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      float f[NE];
#pragma unroll
      for (int v = 0; v < C::NV; ++v) X::unpack(*place(st, u, v), f + v * E);
      if (!rms) {
        float m[1] = {0.f};
#pragma unroll
        for (int e = 0; e < NE; ++e) m[0] += f[e];
        row_sum<C::UPR>(m);
#pragma unroll
        for (int e = 0; e < NE; ++e) f[e] -= m[0] * (1.0f / D);
      }
      float s[1] = {0.f};
#pragma unroll
      for (int e = 0; e < NE; ++e) s[0] += f[e] * f[e];
      row_sum<C::UPR>(s);
      const float rstd = 1.0f / sqrtf(s[0] * (1.0f / D) + eps);
#pragma unroll
      for (int e = 0; e < NE; ++e) f[e] = f[e] * rstd * w[e] + b[e];
      turn<HALF, E, C::NP>(f, cs[u]);
      if (POOL)
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] += f[e];
      if (flat[u] >= 0) {
        T* dst = out + (out_blocked ? ((batch * t.heads + h) * N + row0 + o0 + u * C::kRowStep) * D
                                    : flat[u] * t.out_stride + (int64_t)h * D);
#pragma unroll
        for (int v = 0; v < C::NV; ++v)
          __stcs(reinterpret_cast<uint4*>(dst + c0 * E + v * (D / 2)), X::pack(f + v * E));
      }
    }
    // the means of the fp32 values: summed per thread, over the lanes that share its
    // columns, then over the warps in order
    if constexpr (POOL) {
      if (t.means == nullptr) continue;   // the same for the whole CTA
      float (*sum)[NE + 1] = part[(h - h0) & 1];   // the other one may still be read
#pragma unroll
      for (int off = 16; off >= C::UPR; off >>= 1)
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], off);
      if ((threadIdx.x & 31) < C::UPR)
#pragma unroll
        for (int e = 0; e < NE; ++e) sum[(threadIdx.x >> 5) * C::UPR + c0][e] = acc[e];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += C::THREADS) {
        const int v = HALF ? c / (D / 2) : 0, cc = HALF ? c % (D / 2) : c;
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < C::THREADS / 32; ++g) s += sum[g * C::UPR + cc / E][v * E + cc % E];
        t.means[((batch * t.heads + h) * (N / GR) + row0 / GR) * D + c] = s * (1.0f / (float)GR);
      }
    }
  }
  copy_wait<0>();
}

// Each CTA leaves its columns' sums in part [CTA of q, then of k][dw, db][D].
template <typename T, int D, int GR, bool HALF>
__global__ void __launch_bounds__(Cfg<T, D, GR, HALF>::THREADS)
norm_rope_bwd_kernel(const Bwd q, const Bwd k, const Tokens tk, const RopeArgs a, bool rms, float eps, bool in_blocked,
                     int heads_per_cta, float* __restrict__ part, int32_t* d_status) {
  using C = Cfg<T, D, GR, HALF>;
  using X = Row16<T>;
  constexpr int E = C::E, NE = C::NE;
  __shared__ int4 tok[GR];
  extern __shared__ uint4 ring[];   // [min(kDepth, heads)][x, dy][U][NV][THREADS]
  const bool is_q = blockIdx.y < q.groups;
  const Bwd& t = is_q ? q : k;
  const int group = is_q ? blockIdx.y : blockIdx.y - q.groups;
  const int h0 = group * heads_per_cta, h1 = min(t.heads, h0 + heads_per_cta);
  const T* x = static_cast<const T*>(t.x);
  const T* dy = static_cast<const T*>(t.dy);
  T* dx = static_cast<T*>(t.dx);
  locate<GR, C::THREADS>(tok, tk, a, d_status);
  __syncthreads();
  const int c0 = threadIdx.x % C::UPR, o0 = threadIdx.x / C::UPR;
  float2 cs[C::U][C::NP];
  int64_t flat[C::U];
#pragma unroll
  for (int u = 0; u < C::U; ++u) {
    const int4 w = tok[o0 + u * C::kRowStep];
    flat[u] = w.x;
#pragma unroll
    for (int i = 0; i < C::NP; ++i) cs[u][i] = turn_of(a, w, c0 * C::NP + i);
  }
  float w[NE], dw[NE], db[NE];
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    w[e] = t.w != nullptr ? __ldg(t.w + c0 * E + (e / E) * (D / 2) + e % E) : 1.f;
    dw[e] = db[e] = 0.f;
  }
  const int64_t N = tk.rm.N;
  const int64_t at = (int64_t)blockIdx.x * GR, batch = at / N, row0 = at - batch * N;
  auto place = [&](int st, int which, int u, int v) {
    return ring + (((st * 2 + which) * C::U + u) * C::NV + v) * C::THREADS + threadIdx.x;
  };
  auto fetch = [&](int h, int st) {
    if (h < h1) {
#pragma unroll
      for (int u = 0; u < C::U; ++u)
        if (flat[u] >= 0) {
          const T* sx = x + flat[u] * t.x_stride + (int64_t)h * D + c0 * E;
          const T* sy = dy + (in_blocked ? ((batch * t.heads + h) * N + row0 + o0 + u * C::kRowStep) * D
                                         : flat[u] * t.dy_stride + (int64_t)h * D) + c0 * E;
#pragma unroll
          for (int v = 0; v < C::NV; ++v) {
            copy_async16(place(st, 0, u, v), sx + v * (D / 2));
            copy_async16(place(st, 1, u, v), sy + v * (D / 2));
          }
        }
    }
    copy_commit();
  };
  for (int s = 0; s < kDepth - 1; ++s) fetch(h0 + s, s);
  int st = 0;
  for (int h = h0; h < h1; ++h, st = st + 1 == kDepth ? 0 : st + 1) {
    fetch(h + kDepth - 1, st == 0 ? kDepth - 1 : st - 1);
    copy_wait<kDepth - 1>();
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const bool live = flat[u] >= 0;
      float f[NE], g[NE];
#pragma unroll
      for (int v = 0; v < C::NV; ++v) {
        X::unpack(*place(st, 0, u, v), f + v * E);
        X::unpack(*place(st, 1, u, v), g + v * E);
      }
      turn<HALF, E, C::NP>(g, cs[u]);
      if (!rms) {
        float m[1] = {0.f};
#pragma unroll
        for (int e = 0; e < NE; ++e) m[0] += f[e];
        row_sum<C::UPR>(m);
#pragma unroll
        for (int e = 0; e < NE; ++e) f[e] -= m[0] * (1.0f / D);
      }
      float s[3] = {0.f, 0.f, 0.f};   // (x - mean)^2, gw (x - mean), gw
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const float gw = g[e] * w[e];
        s[0] += f[e] * f[e];
        s[1] += gw * f[e];
        s[2] += gw;
      }
      row_sum<C::UPR>(s);
      const float rstd = 1.0f / sqrtf(s[0] * (1.0f / D) + eps);
      const float m1 = s[1] * rstd * (1.0f / D), m2 = rms ? 0.f : s[2] * (1.0f / D);
      float r[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const float xh = f[e] * rstd;
        r[e] = rstd * (g[e] * w[e] - m2 - xh * m1);
        if (live) {
          dw[e] += g[e] * xh;
          db[e] += g[e];
        }
      }
      if (live) {
        T* dst = dx + flat[u] * t.dx_stride + (int64_t)h * D + c0 * E;
#pragma unroll
        for (int v = 0; v < C::NV; ++v) __stcs(reinterpret_cast<uint4*>(dst + v * (D / 2)), X::pack(r + v * E));
      }
    }
  }
  copy_wait<0>();
  if (t.dw == nullptr && t.db == nullptr) return;
  // over the lanes of a warp that share columns, then over the warps in order
#pragma unroll
  for (int off = 16; off >= C::UPR; off >>= 1)
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], off);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], off);
    }
  float* sum = reinterpret_cast<float*>(ring);   // [warps][dw, db][D]
  __syncthreads();                               // every thread's slots are done with
  if ((threadIdx.x & 31) < C::UPR)
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int c = c0 * E + (e / E) * (D / 2) + e % E;
      sum[(threadIdx.x >> 5) * 2 * D + c] = dw[e];
      sum[(threadIdx.x >> 5) * 2 * D + D + c] = db[e];
    }
  __syncthreads();
  float* mine = part + ((is_q ? 0 : (int64_t)gridDim.x * q.groups) + (int64_t)blockIdx.x * t.groups + group) * 2 * D;
  for (int c = threadIdx.x; c < 2 * D; c += C::THREADS) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < C::THREADS / 32; ++g) s += sum[g * 2 * D + c];
    mine[c] = s;
  }
}

// Sums of the CTAs' parts in a fixed order: warp y of a CTA takes parts y, y + 32, ...,
// its lanes 32 columns; then the warps' sums in order.
template <int D>
__global__ void __launch_bounds__(1024)
norm_rope_sum_kernel(const float* __restrict__ part, int64_t parts_q, int64_t parts_k, const Bwd q, const Bwd k) {
  __shared__ float sum[32][33];
  const bool is_q = blockIdx.y == 0;
  const Bwd& t = is_q ? q : k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* from = part + (is_q ? 0 : parts_q * 2 * D) + c;
  const int64_t n = is_q ? parts_q : parts_k;
  float s = 0.f;
#pragma unroll 8
  for (int64_t i = warp; i < n; i += 32) s += from[i * 2 * D];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) r += sum[i][lane];
    float* to = c < D ? t.dw : t.db;
    if (to != nullptr) to[c % D] = r;
  }
}

// Heads per CTA: as many as leave about four CTAs per SM of the 152, at most 8. The
// workspace depends on it, so it does not depend on the device.
int heads_per_cta(int64_t granules, int heads) {
  const int64_t h = granules * heads / (152 * 4);
  return (int)(h < 1 ? 1 : h > 8 ? 8 : h);
}

template <typename T>
constexpr int granule() { return sizeof(T) == 4 ? 32 : 64; }

int64_t granules_of(const Dims& s, int gr) { return ((int64_t)s.B * s.N + gr - 1) / gr; }

template <typename T, int D, int GR, bool HALF, bool POOL>
bool go_fwd(const Dims& s, const RopeArgs& a, Fwd q, Fwd k, const Tokens& tk, bool rms, float eps, bool out_blocked,
            int32_t* d_status, cudaStream_t st) {
  using C = Cfg<T, D, GR, HALF>;
  const int64_t granules = granules_of(s, GR);
  const int hpc = heads_per_cta(granules, q.heads + k.heads);
  q.groups = (q.heads + hpc - 1) / hpc;
  k.groups = (k.heads + hpc - 1) / hpc;
  const size_t smem = (size_t)(hpc < kDepth ? hpc : kDepth) * C::VECS * 16;
  auto kern = norm_rope_fwd_kernel<T, D, GR, HALF, POOL>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  kern<<<dim3((unsigned)granules, (unsigned)(q.groups + k.groups)), C::THREADS, smem, st>>>(q, k, tk, a, rms, eps, out_blocked,
                                                                                           hpc, d_status);
  return true;
}

template <typename T, int D, bool HALF>
bool go_fwd_granule(const Dims& s, const RopeArgs& a, const Fwd& q, const Fwd& k, const Tokens& tk, bool rms, float eps,
                    bool out_blocked, int32_t* d_status, cudaStream_t st) {
  if (q.means != nullptr || k.means != nullptr) {   // means take a whole tile
    if (s.Bt == 64) return go_fwd<T, D, 64, HALF, true>(s, a, q, k, tk, rms, eps, out_blocked, d_status, st);
    return go_fwd<T, D, 128, HALF, true>(s, a, q, k, tk, rms, eps, out_blocked, d_status, st);
  }
  return go_fwd<T, D, granule<T>(), HALF, false>(s, a, q, k, tk, rms, eps, out_blocked, d_status, st);
}

template <typename T, int D, bool HALF>
bool go_bwd(const Dims& s, const RopeArgs& a, Bwd q, Bwd k, const Tokens& tk, bool rms, float eps, bool in_blocked,
            float* part, int32_t* d_status, cudaStream_t st) {
  constexpr int GR = granule<T>();
  using C = Cfg<T, D, GR, HALF>;
  const int64_t granules = granules_of(s, GR);
  const int hpc = heads_per_cta(granules, q.heads + k.heads);
  q.groups = (q.heads + hpc - 1) / hpc;
  k.groups = (k.heads + hpc - 1) / hpc;
  size_t smem = (size_t)(hpc < kDepth ? hpc : kDepth) * 2 * C::VECS * 16;
  const size_t sums = (size_t)C::THREADS / 32 * 2 * D * 4;
  if (smem < sums) smem = sums;
  auto kern = norm_rope_bwd_kernel<T, D, GR, HALF>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  kern<<<dim3((unsigned)granules, (unsigned)(q.groups + k.groups)), C::THREADS, smem, st>>>(q, k, tk, a, rms, eps, in_blocked,
                                                                                           hpc, part, d_status);
  if (q.dw != nullptr || q.db != nullptr || k.dw != nullptr || k.db != nullptr)
    norm_rope_sum_kernel<D><<<dim3(2 * D / 32, k.heads > 0 ? 2 : 1), 1024, 0, st>>>(part, granules * q.groups,
                                                                                   granules * k.groups, q, k);
  return true;
}

Tokens tokens_of(const Dims& s, bool tiles) {
  Tokens t{};
  t.rm = raster_map(s);
  t.total = (int64_t)s.B * s.N;
  t.linear = !tiles;
  t.bt = s.Bt;
  return t;
}

}  // namespace

size_t norm_rope_ws(const Dims& s, int heads_k) {
  const int64_t granules = granules_of(s, s.dtype == SPARSP_F32 ? granule<float>() : granule<__nv_bfloat16>());
  const int hpc = heads_per_cta(granules, s.H + heads_k);
  return (size_t)granules * ((s.H + hpc - 1) / hpc + (heads_k + hpc - 1) / hpc) * 2 * s.d * sizeof(float);
}

sparsp_status_t launch_norm_rope_fwd(const Dims& s, bool tiles, const sparsp_rope_t& r, const float* table,
                                     const int32_t* pos, bool rms, float eps, bool out_blocked,
                                     const sparsp_norm_rope_t& q, const sparsp_norm_rope_t& k, int32_t* d_status,
                                     cudaStream_t st) {
  RopeArgs a = rope_args(r, table);
  a.pos = pos;
  auto part = [](const sparsp_norm_rope_t& t) {
    return Fwd{t.x, t.x_stride, t.out, t.out_stride, t.w, t.b, t.means, t.heads, 0};
  };
  const Tokens tk = tokens_of(s, tiles);
  const Fwd fq = part(q), fk = part(k);
  bool ok;
#define SPARSP_GO(T, D)                                                                             \
  ok = r.half ? go_fwd_granule<T, D, true>(s, a, fq, fk, tk, rms, eps, out_blocked, d_status, st)   \
              : go_fwd_granule<T, D, false>(s, a, fq, fk, tk, rms, eps, out_blocked, d_status, st)
  if (s.dtype == SPARSP_F32 && s.d == 64) SPARSP_GO(float, 64);
  else if (s.dtype == SPARSP_F32) SPARSP_GO(float, 128);
  else if (s.d == 64) SPARSP_GO(__nv_bfloat16, 64);
  else SPARSP_GO(__nv_bfloat16, 128);
#undef SPARSP_GO
  if (!ok) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_norm_rope_bwd(const Dims& s, bool tiles, const sparsp_rope_t& r, const float* table,
                                     const int32_t* pos, bool rms, float eps, bool in_blocked,
                                     const sparsp_norm_rope_t& q, const sparsp_norm_rope_t& k, void* ws,
                                     int32_t* d_status, cudaStream_t st) {
  RopeArgs a = rope_args(r, table);
  a.pos = pos;
  a.sign = -1.f;
  auto part = [](const sparsp_norm_rope_t& t) {
    return Bwd{t.dy, t.x, t.dy_stride, t.x_stride, t.out, t.out_stride, t.w, t.dw, t.db, t.heads, 0};
  };
  const Tokens tk = tokens_of(s, tiles);
  const Bwd bq = part(q), bk = part(k);
  bool ok;
#define SPARSP_GO(T, D)                                                                                   \
  ok = r.half ? go_bwd<T, D, true>(s, a, bq, bk, tk, rms, eps, in_blocked, (float*)ws, d_status, st)      \
              : go_bwd<T, D, false>(s, a, bq, bk, tk, rms, eps, in_blocked, (float*)ws, d_status, st)
  if (s.dtype == SPARSP_F32 && s.d == 64) SPARSP_GO(float, 64);
  else if (s.dtype == SPARSP_F32) SPARSP_GO(float, 128);
  else if (s.d == 64) SPARSP_GO(__nv_bfloat16, 64);
  else SPARSP_GO(__nv_bfloat16, 128);
#undef SPARSP_GO
  if (!ok) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

}  // namespace sparsp
