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
// Measured at 30,720 tokens and 40 + 40 heads of 128 in bf16 (of a copy's rate): forward 200 us (0.93),
// with tile means 227 (0.82: a tile's means are joined over the warps at its end, through
// shared memory), backward 304 (0.91); backward of 8,192 tokens and 12 + 12 heads of 64 in fp32 35 us (0.63: the
// heads go 8 and 4 to a CTA, and 5 us are the sum of the parts); 64 tokens 5 us on the device. Norm and rotation
// one after the other take 435 us forward, without means.
#include "rows.cuh"

namespace sparsp {
namespace {

template <typename T, int D, int GR, bool HALF>
struct Cfg {
  static constexpr int E = Row16<T>::E;                        // values per 16-byte vector
  static constexpr int NV = HALF ? 2 : 1;                      // vectors of a unit
  static constexpr int NE = NV * E;                            // values of a unit
  static constexpr int NP = NE / 2;                            // pairs of a unit
  static constexpr int P2 = Unit<T, HALF>::P2;                 // the same, two to a packed operand
  static constexpr int UPR = D / NE;                           // units (lanes) per row
  static constexpr int VECS = GR * D / E;                      // vectors of a granule
  static constexpr int THREADS = 256;                          // 2 or 4 vectors each
  static_assert(VECS == 512 || VECS == 1024, "vectors of a thread");
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

// Strides are bytes between tokens (raster); below 2^32, so that an address is one multiply-add.
struct Fwd {
  const void* in;
  uint32_t in_stride;
  void* out;
  uint32_t out_stride;
  const float *w, *b;
  float* means;
  int heads, groups;
};
struct Bwd {
  const void *dy, *x;
  uint32_t dy_stride, x_stride;
  void* dx;
  uint32_t dx_stride;
  const float* w;
  float *dw, *db;
  int heads, groups;
};

// tok[o] of tokens blockIdx.x * count ..: flat raster token (b * N + n, -1 past the end) and its table row
// per axis (-1: not turned). In tile order count divides a tile's tokens.
template <int THREADS>
__device__ __forceinline__ void locate(int4* tok, int count, const Tokens& t, const RopeArgs& a, int32_t* d_status) {
  const RasterMap& rm = t.rm;
  for (int o = threadIdx.x; o < count; o += THREADS) {
    int64_t flat;
    int p[3];
    if (t.linear) {
      flat = (int64_t)blockIdx.x * count + o;
      const int n = (int)(flat % rm.N);
      p[0] = n / (rm.Y * rm.X);
      p[1] = n / rm.X % rm.Y;
      p[2] = n % rm.X;
    } else {
      const int per = t.bt / count, nb = (int)(rm.N / t.bt), tile = blockIdx.x / per;
      const int j = tile % nb, oo = (int)(blockIdx.x % per) * count + o;
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

// (x, y) -> (x c - y s, x s + y c), two pairs at a time.
template <int P2>
__device__ __forceinline__ void turn(f32x2* x, f32x2* y, const f32x2* c, const f32x2* s) {
#pragma unroll
  for (int i = 0; i < P2; ++i) {
    const f32x2 r = sub2(mul2(x[i], c[i]), mul2(y[i], s[i]));
    y[i] = fma2(y[i], c[i], mul2(x[i], s[i]));
    x[i] = r;
  }
}

// The columns of pair i of unit column c0.
template <int D, int E, bool HALF>
__device__ __forceinline__ int col_x(int c0, int i) { return c0 * E + (HALF ? i : 2 * i); }
template <int D, int E, bool HALF>
__device__ __forceinline__ int col_y(int c0, int i) { return HALF ? c0 * E + i + D / 2 : c0 * E + 2 * i + 1; }

// A parameter vector's values at a lane's columns.
template <int D, int E, bool HALF, int P2>
__device__ __forceinline__ void params(const float* p, float none, int c0, f32x2* x, f32x2* y) {
#pragma unroll
  for (int i = 0; i < P2; ++i) {
    float v[4] = {none, none, none, none};
    if (p != nullptr) {
      v[0] = __ldg(p + col_x<D, E, HALF>(c0, 2 * i));
      v[1] = __ldg(p + col_x<D, E, HALF>(c0, 2 * i + 1));
      v[2] = __ldg(p + col_y<D, E, HALF>(c0, 2 * i));
      v[3] = __ldg(p + col_y<D, E, HALF>(c0, 2 * i + 1));
    }
    x[i] = pair(v[0], v[1]);
    y[i] = pair(v[2], v[3]);
  }
}

template <int P2>
__device__ __forceinline__ float sum_of(const f32x2* x, const f32x2* y) {
  f32x2 a = add2(x[0], y[0]);
#pragma unroll
  for (int i = 1; i < P2; ++i) a = add2(a, add2(x[i], y[i]));
  return hsum(a);
}
template <int P2>   // sum of a b over both halves of the pairs
__device__ __forceinline__ float dot_of(const f32x2* ax, const f32x2* ay, const f32x2* bx, const f32x2* by) {
  f32x2 a = mul2(ax[0], bx[0]), b = mul2(ay[0], by[0]);
#pragma unroll
  for (int i = 1; i < P2; ++i) {
    a = fma2(ax[i], bx[i], a);
    b = fma2(ay[i], by[i], b);
  }
  return hsum(add2(a, b));
}

// Vector at `base` of a raster token.
template <typename P>
__device__ __forceinline__ P at_token(P base, int flat, uint32_t stride) {
  return base + (uint64_t)(uint32_t)flat * stride;
}

// Sums over the UPR lanes that share a row.
template <int UPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K]) {
#pragma unroll
  for (int off = UPR / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
}

// Heads in flight per CTA: forward with means / backward take 238 / 312 us at 2, 233 / 308 at 3, 241 / 395 at 4 (one
// CTA per SM).
constexpr int kDepth = 3;

// BIAS: there may be one (a layer norm, or an RMS norm with a bias). POOL: a CTA takes a whole
// tile, granule after granule, and leaves its means: each warp keeps its columns' sums of every
// head in shared memory, so that they are joined once, at the end.
template <typename T, int D, int GR, bool HALF, bool POOL, bool BIAS, bool BLOCKED>
__global__ void __launch_bounds__(Cfg<T, D, GR, HALF>::THREADS, 2)
norm_rope_fwd_kernel(const Fwd q, const Fwd k, const Tokens tk, const RopeArgs a, bool rms, float eps,
                     int heads_per_cta, int32_t* d_status) {
  using C = Cfg<T, D, GR, HALF>;
  using X = Unit<T, HALF>;
  constexpr int E = C::E, P2 = C::P2, kWarps = C::THREADS / 32;
  __shared__ int4 tok[POOL ? 128 : GR];
  extern __shared__ uint4 ring[];   // [min(kDepth, steps)][U][NV][THREADS], then with POOL [heads][warps][D] floats
  const bool is_q = blockIdx.y < q.groups;
  const Fwd& t = is_q ? q : k;
  const int h0 = (is_q ? blockIdx.y : blockIdx.y - q.groups) * heads_per_cta, heads = min(t.heads - h0, heads_per_cta);
  const int parts = POOL ? tk.bt / GR : 1, steps = parts * heads;   // a step: a granule of a head
  float* sums = reinterpret_cast<float*>(ring + (size_t)kDepth * C::VECS);
  locate<C::THREADS>(tok, parts * GR, tk, a, d_status);
  __syncthreads();
  const int c0 = threadIdx.x % C::UPR, o0 = threadIdx.x / C::UPR, warp = threadIdx.x >> 5;   // c0: unit column, o0: first row
  f32x2 wx[P2], wy[P2], bx[P2], by[P2];
  params<D, E, HALF, P2>(t.w, 1.f, c0, wx, wy);
  if (BIAS) params<D, E, HALF, P2>(t.b, 0.f, c0, bx, by);
  // rows of tile order: those of head h of this CTA's batch element start at (batch * heads + h) * N + row0
  const int64_t N = tk.rm.N;
  const int64_t at = (int64_t)blockIdx.x * parts * GR, batch = at / N, row0 = at - batch * N;
  auto place = [&](int st, int u, int v) { return ring + ((st * C::U + u) * C::NV + v) * C::THREADS + threadIdx.x; };
  const uint8_t* in0 = static_cast<const uint8_t*>(t.in) + ((int64_t)h0 * D + c0 * E) * sizeof(T);
  const uint8_t* in = in0;                       // of the next fetch
  int f_head = 0, f_part = 0, f_step = 0;        // of the next fetch
  auto fetch = [&]() {
    if (f_step < steps) {
      const int st = f_step % kDepth;
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        const int flat = tok[f_part * GR + o0 + u * C::kRowStep].x;
        if (POOL || flat >= 0) {                 // a tile is whole
          const uint8_t* src = at_token(in, flat, t.in_stride);
#pragma unroll
          for (int v = 0; v < C::NV; ++v) copy_async16(place(st, u, v), src + v * (D / 2) * sizeof(T));
        }
      }
      in += D * sizeof(T);
      ++f_step;
      if (++f_head == heads) {
        f_head = 0;
        ++f_part;
        in = in0;
      }
    }
    copy_commit();
  };
  for (int s = 0; s < kDepth - 1; ++s) fetch();
  int st = 0;
  for (int part = 0; part < parts; ++part) {
    f32x2 cos[C::U][P2], sin[C::U][P2];
    int flat[C::U];
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const int4 w = tok[part * GR + o0 + u * C::kRowStep];
      flat[u] = w.x;
#pragma unroll
      for (int i = 0; i < P2; ++i) {
        const float2 p = turn_of(a, w, c0 * C::NP + 2 * i), q2 = turn_of(a, w, c0 * C::NP + 2 * i + 1);
        cos[u][i] = pair(p.x, q2.x);
        sin[u][i] = pair(p.y, q2.y);
      }
    }
    uint8_t* out = static_cast<uint8_t*>(t.out) +
                   (BLOCKED ? ((batch * t.heads + h0) * N + row0 + part * GR + o0) * D + c0 * E
                            : (int64_t)h0 * D + c0 * E) * sizeof(T);
    const int64_t out_step = (BLOCKED ? N * D : (int64_t)D) * sizeof(T);
    for (int h = 0; h < heads; ++h, st = st + 1 == kDepth ? 0 : st + 1) {
      fetch();                                   // into the slots of the step before
      copy_wait<kDepth - 1>();
      f32x2 ax[P2], ay[P2];
#pragma unroll
      for (int i = 0; i < P2; ++i) ax[i] = ay[i] = 0;   // two zeros
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        f32x2 x[P2], y[P2];
        uint4 v16[C::NV];
#pragma unroll
        for (int v = 0; v < C::NV; ++v) v16[v] = *place(st, u, v);
        X::unpack(v16, x, y);
        if (BIAS && !rms) {
          float m[1] = {sum_of<P2>(x, y)};
          row_sum<C::UPR>(m);
          const f32x2 mean = pair(m[0] * (-1.0f / D), m[0] * (-1.0f / D));
#pragma unroll
          for (int i = 0; i < P2; ++i) {
            x[i] = add2(x[i], mean);
            y[i] = add2(y[i], mean);
          }
        }
        float s[1] = {dot_of<P2>(x, y, x, y)};
        row_sum<C::UPR>(s);
        const float rstd = inv_sqrt(s[0] * (1.0f / D) + eps);
        const f32x2 r2 = pair(rstd, rstd);
#pragma unroll
        for (int i = 0; i < P2; ++i) {
          x[i] = BIAS ? fma2(mul2(x[i], r2), wx[i], bx[i]) : mul2(mul2(x[i], r2), wx[i]);
          y[i] = BIAS ? fma2(mul2(y[i], r2), wy[i], by[i]) : mul2(mul2(y[i], r2), wy[i]);
        }
        turn<P2>(x, y, cos[u], sin[u]);
        if (POOL)
#pragma unroll
          for (int i = 0; i < P2; ++i) {
            ax[i] = add2(ax[i], x[i]);
            ay[i] = add2(ay[i], y[i]);
          }
        if (POOL || flat[u] >= 0) {
          uint8_t* dst = BLOCKED ? out + u * C::kRowStep * D * sizeof(T) : at_token(out, flat[u], t.out_stride);
          X::pack(x, y, v16);
#pragma unroll
          for (int v = 0; v < C::NV; ++v) __stcs(reinterpret_cast<uint4*>(dst + v * (D / 2) * sizeof(T)), v16[v]);
        }
      }
      out += out_step;
      // the sums of the fp32 values: per thread, then over the lanes that share its columns, then over granules
      if constexpr (POOL) {
        if (t.means != nullptr) {                // the same for the whole CTA
          float* mine = sums + (h * kWarps + warp) * D;
#pragma unroll
          for (int i = 0; i < C::NP; i += 2) {   // two pairs of columns: four neighbours, or HALF two and two
            const float2 px = both(ax[i / 2]), py = both(ay[i / 2]);
            float v[4] = {px.x, HALF ? px.y : py.x, HALF ? py.x : px.y, py.y};
#pragma unroll
            for (int off = 16; off >= C::UPR; off >>= 1)
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], off);
            if ((threadIdx.x & 31) < C::UPR) {
              float2* lo = reinterpret_cast<float2*>(mine + col_x<D, E, HALF>(c0, i));
              float2* hi = reinterpret_cast<float2*>(HALF ? mine + col_y<D, E, HALF>(c0, i) : mine + col_x<D, E, HALF>(c0, i + 1));
              const float2 was = part == 0 ? make_float2(0.f, 0.f) : *lo, then = part == 0 ? make_float2(0.f, 0.f) : *hi;
              *lo = make_float2(was.x + v[0], was.y + v[1]);
              *hi = make_float2(then.x + v[2], then.y + v[3]);
            }
          }
        }
      }
    }
  }
  copy_wait<0>();
  if constexpr (POOL) {
    if (t.means == nullptr) return;
    __syncthreads();
    float* to = t.means + ((batch * t.heads + h0) * (N / tk.bt) + row0 / tk.bt) * D;
    for (int i = threadIdx.x; i < heads * D; i += C::THREADS) {
      const int h = i / D, c = i % D;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[(h * kWarps + w) * D + c];   // the warps in order
      to[(int64_t)h * (N / tk.bt) * D + c] = s * (1.0f / (float)tk.bt);
    }
  }
}

// Each CTA leaves its columns' sums in part [CTA of q, then of k][dw, db][D].
template <typename T, int D, int GR, bool HALF, bool RMS, bool BLOCKED>
__global__ void __launch_bounds__(Cfg<T, D, GR, HALF>::THREADS, HALF ? 1 : 2)
norm_rope_bwd_kernel(const Bwd q, const Bwd k, const Tokens tk, const RopeArgs a, float eps,
                     int heads_per_cta, float* __restrict__ part, int32_t* d_status) {
  using C = Cfg<T, D, GR, HALF>;
  using X = Unit<T, HALF>;
  constexpr int E = C::E, P2 = C::P2;
  __shared__ int4 tok[GR];
  extern __shared__ uint4 ring[];   // [min(kDepth, heads)][x, dy][U][NV][THREADS]
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const bool is_q = blockIdx.y < q.groups;
  const Bwd& t = is_q ? q : k;
  const int group = is_q ? blockIdx.y : blockIdx.y - q.groups;
  const int h0 = group * heads_per_cta, h1 = min(t.heads, h0 + heads_per_cta);
  locate<C::THREADS>(tok, GR, tk, a, d_status);
  __syncthreads();
  const int c0 = threadIdx.x % C::UPR, o0 = threadIdx.x / C::UPR;
  f32x2 cos[C::U][P2], sin[C::U][P2];
  int flat[C::U];
#pragma unroll
  for (int u = 0; u < C::U; ++u) {
    const int4 w = tok[o0 + u * C::kRowStep];
    flat[u] = w.x;
#pragma unroll
    for (int i = 0; i < P2; ++i) {
      const float2 p = turn_of(a, w, c0 * C::NP + 2 * i), q = turn_of(a, w, c0 * C::NP + 2 * i + 1);
      cos[u][i] = pair(p.x, q.x);
      sin[u][i] = pair(p.y, q.y);
    }
  }
  f32x2 wx[P2], wy[P2], dwx[P2], dwy[P2], dbx[P2], dby[P2];
  params<D, E, HALF, P2>(t.w, 1.f, c0, wx, wy);
#pragma unroll
  for (int i = 0; i < P2; ++i) dwx[i] = dwy[i] = dbx[i] = dby[i] = 0;   // two zeros
  const int64_t N = tk.rm.N;
  const int64_t at = (int64_t)blockIdx.x * GR, batch = at / N, row0 = at - batch * N;
  auto place = [&](int st, int which, int u, int v) {
    return ring + (((st * 2 + which) * C::U + u) * C::NV + v) * C::THREADS + threadIdx.x;
  };
  const int64_t col0 = ((int64_t)h0 * D + c0 * E) * sizeof(T);
  const uint8_t* x = static_cast<const uint8_t*>(t.x) + col0;                                     // of the next fetch
  const uint8_t* dy = static_cast<const uint8_t*>(t.dy) +
                      (BLOCKED ? (((batch * t.heads + h0) * N + row0 + o0) * D + c0 * E) * (int64_t)sizeof(T) : col0);
  const int64_t dy_step = (BLOCKED ? N * D : (int64_t)D) * sizeof(T);
  uint8_t* dx = static_cast<uint8_t*>(t.dx) + col0;                                               // of the next store
  auto fetch = [&](int h, int st) {
    if (h < h1) {
#pragma unroll
      for (int u = 0; u < C::U; ++u)
        if (flat[u] >= 0) {
          const uint8_t* sx = at_token(x, flat[u], t.x_stride);
          const uint8_t* sy = BLOCKED ? dy + u * C::kRowStep * D * sizeof(T) : at_token(dy, flat[u], t.dy_stride);
#pragma unroll
          for (int v = 0; v < C::NV; ++v) {
            copy_async16(place(st, 0, u, v), sx + v * (D / 2) * sizeof(T));
            copy_async16(place(st, 1, u, v), sy + v * (D / 2) * sizeof(T));
          }
        }
      x += D * sizeof(T);
      dy += dy_step;
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
      f32x2 fx[P2], fy[P2], gx[P2], gy[P2];
      uint4 v16[C::NV];
#pragma unroll
      for (int v = 0; v < C::NV; ++v) v16[v] = *place(st, 1, u, v);
      X::unpack(v16, gx, gy);
#pragma unroll
      for (int v = 0; v < C::NV; ++v) v16[v] = *place(st, 0, u, v);
      X::unpack(v16, fx, fy);
      turn<P2>(gx, gy, cos[u], sin[u]);
      if (!RMS) {
        float m[1] = {sum_of<P2>(fx, fy)};
        row_sum<C::UPR>(m);
        const f32x2 mean = pair(m[0] * (-1.0f / D), m[0] * (-1.0f / D));
#pragma unroll
        for (int i = 0; i < P2; ++i) {
          fx[i] = add2(fx[i], mean);
          fy[i] = add2(fy[i], mean);
        }
      }
      f32x2 ux[P2], uy[P2];                       // gw
#pragma unroll
      for (int i = 0; i < P2; ++i) {
        ux[i] = mul2(gx[i], wx[i]);
        uy[i] = mul2(gy[i], wy[i]);
      }
      float s[RMS ? 2 : 3] = {dot_of<P2>(fx, fy, fx, fy), dot_of<P2>(ux, uy, fx, fy)};
      if (!RMS) s[RMS ? 0 : 2] = sum_of<P2>(ux, uy);
      row_sum<C::UPR>(s);
      const float rstd = inv_sqrt(s[0] * (1.0f / D) + eps);
      // dx = rstd gw - (x - mean) rstd^2 mean(gw xh) - rstd mean(gw); xh = (x - mean) rstd
      const float m1 = -s[1] * rstd * (1.0f / D), m2 = RMS ? 0.f : -s[RMS ? 0 : 2] * (1.0f / D);
      const f32x2 r2 = pair(rstd, rstd), n1 = pair(m1, m1), n2 = pair(m2, m2);
#pragma unroll
      for (int i = 0; i < P2; ++i) {
        fx[i] = mul2(fx[i], r2);
        fy[i] = mul2(fy[i], r2);
        if (live) {
          dwx[i] = fma2(gx[i], fx[i], dwx[i]);
          dwy[i] = fma2(gy[i], fy[i], dwy[i]);
          dbx[i] = add2(dbx[i], gx[i]);
          dby[i] = add2(dby[i], gy[i]);
        }
        if (!RMS) {
          ux[i] = add2(ux[i], n2);
          uy[i] = add2(uy[i], n2);
        }
        ux[i] = mul2(fma2(fx[i], n1, ux[i]), r2);
        uy[i] = mul2(fma2(fy[i], n1, uy[i]), r2);
      }
      if (live) {
        uint8_t* dst = at_token(dx, flat[u], t.dx_stride);
        X::pack(ux, uy, v16);
#pragma unroll
        for (int v = 0; v < C::NV; ++v) __stcs(reinterpret_cast<uint4*>(dst + v * (D / 2) * sizeof(T)), v16[v]);
      }
    }
    dx += D * sizeof(T);
  }
  copy_wait<0>();
  if (t.dw == nullptr && t.db == nullptr) return;
  // over the lanes of a warp that share columns, then over the warps in order
  float* sum = reinterpret_cast<float*>(ring);   // [warps][dw, db][D]
  __syncthreads();                               // every thread's slots are done with
#pragma unroll
  for (int i = 0; i < C::NP; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 px = both(k ? dbx[i / 2] : dwx[i / 2]), py = both(k ? dby[i / 2] : dwy[i / 2]);
      float vx = i & 1 ? px.y : px.x, vy = i & 1 ? py.y : py.x;
#pragma unroll
      for (int off = 16; off >= C::UPR; off >>= 1) {
        vx += __shfl_xor_sync(0xffffffffu, vx, off);
        vy += __shfl_xor_sync(0xffffffffu, vy, off);
      }
      if ((threadIdx.x & 31) < C::UPR) {
        float* to = sum + ((threadIdx.x >> 5) * 2 + k) * D;
        to[col_x<D, E, HALF>(c0, i)] = vx;
        to[col_y<D, E, HALF>(c0, i)] = vy;
      }
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

// Sums of the CTAs' parts in a fixed order: eight columns to a CTA, four parts to a warp at a time, of every 128;
// then the threads' sums in order. (32 columns to a CTA, a part to a warp: 9 us for 2,400 parts, not 6.)
constexpr int kSumCols = 8;
template <int D>
__global__ void __launch_bounds__(1024)
norm_rope_sum_kernel(const float* __restrict__ part, int64_t parts_q, int64_t parts_k, const Bwd q, const Bwd k) {
  constexpr int kAt = 1024 / kSumCols;
  __shared__ float sum[kAt][kSumCols + 1];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const bool is_q = blockIdx.y == 0;
  const Bwd& t = is_q ? q : k;
  const int at = threadIdx.x / kSumCols, col = threadIdx.x % kSumCols, c = blockIdx.x * kSumCols + col;
  const float* from = part + (is_q ? 0 : parts_q * 2 * D) + c;
  const int64_t n = is_q ? parts_q : parts_k;
  float s = 0.f;
#pragma unroll 8
  for (int64_t i = at; i < n; i += kAt) s += from[i * 2 * D];
  sum[at][col] = s;
  __syncthreads();
  for (int half = kAt / 2; half > 0; half >>= 1) {
    if (at < half) sum[at][col] += sum[at + half][col];
    __syncthreads();
  }
  if (at == 0) {
    float* to = c < D ? t.dw : t.db;
    if (to != nullptr) to[c % D] = sum[0][col];
  }
}

// Heads per CTA: as many as leave about four CTAs per SM of the 152, at most 8. The
// workspace depends on it, so it does not depend on the device.
int heads_per_cta(int64_t granules, int heads) {
  const int64_t h = granules * heads / (152 * 4);
  return (int)(h < 1 ? 1 : h > 8 ? 8 : h);
}

// Tokens of a granule: with 128 in bf16 forward / backward take 240 / 315 us, not 233 / 308; 64 in fp32 change nothing.
template <typename T>
constexpr int granule() { return sizeof(T) == 4 ? 32 : 64; }

int64_t granules_of(const Dims& s, int gr) { return ((int64_t)s.B * s.N + gr - 1) / gr; }

template <typename T, int D, bool HALF, bool POOL>
bool go_fwd(const Dims& s, const RopeArgs& a, Fwd q, Fwd k, const Tokens& tk, bool rms, float eps, bool out_blocked,
            int32_t* d_status, cudaStream_t st) {
  constexpr int GR = granule<T>();
  using C = Cfg<T, D, GR, HALF>;
  const int64_t granules = granules_of(s, POOL ? s.Bt : GR);
  const int hpc = heads_per_cta(granules, q.heads + k.heads);
  q.groups = (q.heads + hpc - 1) / hpc;
  k.groups = (k.heads + hpc - 1) / hpc;
  const int steps = hpc * (POOL ? s.Bt / GR : 1);
  const size_t smem = POOL ? (size_t)kDepth * C::VECS * 16 + (size_t)hpc * C::THREADS / 32 * D * sizeof(float)
                           : (size_t)(steps < kDepth ? steps : kDepth) * C::VECS * 16;
  const bool bias = !rms || q.b != nullptr || k.b != nullptr;
  auto kern = out_blocked ? (bias ? norm_rope_fwd_kernel<T, D, GR, HALF, POOL, true, true>
                                  : norm_rope_fwd_kernel<T, D, GR, HALF, POOL, false, true>)
                          : (bias ? norm_rope_fwd_kernel<T, D, GR, HALF, POOL, true, false>
                                  : norm_rope_fwd_kernel<T, D, GR, HALF, POOL, false, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  kern<<<dim3((unsigned)granules, (unsigned)(q.groups + k.groups)), C::THREADS, smem, st>>>(q, k, tk, a, rms, eps, hpc,
                                                                                           d_status);
  return true;
}

template <typename T, int D, bool HALF>
bool go_fwd_pool(const Dims& s, const RopeArgs& a, const Fwd& q, const Fwd& k, const Tokens& tk, bool rms, float eps,
                 bool out_blocked, int32_t* d_status, cudaStream_t st) {
  if (q.means != nullptr || k.means != nullptr)
    return go_fwd<T, D, HALF, true>(s, a, q, k, tk, rms, eps, out_blocked, d_status, st);
  return go_fwd<T, D, HALF, false>(s, a, q, k, tk, rms, eps, out_blocked, d_status, st);
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
  auto kern = in_blocked ? (rms ? norm_rope_bwd_kernel<T, D, GR, HALF, true, true>
                                : norm_rope_bwd_kernel<T, D, GR, HALF, false, true>)
                         : (rms ? norm_rope_bwd_kernel<T, D, GR, HALF, true, false>
                                : norm_rope_bwd_kernel<T, D, GR, HALF, false, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  kern<<<dim3((unsigned)granules, (unsigned)(q.groups + k.groups)), C::THREADS, smem, st>>>(q, k, tk, a, eps, hpc,
                                                                                           part, d_status);
  if (q.dw != nullptr || q.db != nullptr || k.dw != nullptr || k.db != nullptr)
    return launch_after(norm_rope_sum_kernel<D>, dim3(2 * D / kSumCols, k.heads > 0 ? 2 : 1), 1024, st, part,
                        granules * q.groups, granules * k.groups, q, k) == SPARSP_OK;
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
  const int64_t e = s.elem;
  auto part = [e](const sparsp_norm_rope_t& t) {
    return Fwd{t.x, (uint32_t)(t.x_stride * e), t.out, (uint32_t)(t.out_stride * e), t.w, t.b, t.means, t.heads, 0};
  };
  const Tokens tk = tokens_of(s, tiles);
  const Fwd fq = part(q), fk = part(k);
  bool ok;
#define SPARSP_GO(T, D)                                                                             \
  ok = r.half ? go_fwd_pool<T, D, true>(s, a, fq, fk, tk, rms, eps, out_blocked, d_status, st)   \
              : go_fwd_pool<T, D, false>(s, a, fq, fk, tk, rms, eps, out_blocked, d_status, st)
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
  const int64_t e = s.elem;
  auto part = [e](const sparsp_norm_rope_t& t) {
    return Bwd{t.dy, t.x, (uint32_t)(t.dy_stride * e), (uint32_t)(t.x_stride * e), t.out, (uint32_t)(t.out_stride * e),
               t.w, t.dw, t.db, t.heads, 0};
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
