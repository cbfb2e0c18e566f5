// Three-axis rotary positions (time, height, width) of query / key rows, in
// the pass that moves them between raster and tile order, and optionally pools
// the tile means.
//
// The d columns of a head are paired as (2i, 2i + 1), or (i, i + d/2) with
// HALF; the first cols[0] / 2 pairs turn with the token's frame, the next
// cols[1] / 2 with its row, the next cols[2] / 2 with its column, the rest not
// at all. Pair i of axis a at position p turns by
//   phi = (offset_a + scale_a p) theta^(-2 i / cols[a]):
//   (u, v) -> (u cos phi - v sin phi, u sin phi + v cos phi),
// and by -phi in the inverse (the gradient's way: the transposed rotation).
// The angles come from a table [extent_a, cols[a] / 2] of (cos, sin) per axis,
// computed once from 64-bit angles, so far positions lose nothing.
//
// Bound by HBM: each row is read and written once. A CTA takes one tile and
// several heads. All heads of a token turn alike, so a thread loads the (cos,
// sin) of its tokens and columns once, keeps them in registers and sweeps the
// heads; the 16-byte vectors of the next heads are on their way meanwhile, each
// thread's into shared-memory slots of its own (cp.async): without them 138 us for the
// first case here. Measured, cold cache, against a copy's 6.67 TB/s (bf16):
//   30,720 tokens, 40 heads of 128, raster to tile order with means: 111 us, 5.7 TB/s (0.86)
//   65,536 tokens, 24 heads of 128, the inverse with given positions: 138 us, 5.8 TB/s (0.87)
//   8,192 tokens, 12 heads of 64: 10.2 us, of which the launch is half
// The rest is the ramp of CTAs that live for 8 heads only, and the read and write streams
// of rows 10 KB apart.
#include "common.cuh"
#include "tc_helpers.cuh"

namespace sparsp {
namespace {

struct RopeArgs {
  int cols[3];          // columns per axis
  int extent[3];        // table rows per axis
  int base[3];          // first table entry per axis
  const float2* table;
  const int32_t* pos;   // [B, N, 3] or null: grid coordinates
  float sign;           // -1: inverse
};

struct Side {           // one tensor: raster rows `stride` elements apart per token, or tile order
  int64_t stride;
  int blocked;
};

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

template <typename T, int D, int BT, bool HALF>
struct RopeCfg {
  static constexpr int E = Row16<T>::E;                        // values per 16-byte vector
  static constexpr int NV = HALF ? 2 : 1;                      // vectors of a unit
  static constexpr int NP = NV * E / 2;                        // pairs of a unit
  static constexpr int UPR = D / (NV * E);                     // units per row
  static constexpr int VECS = BT * D / E;                      // vectors of a tile
  static constexpr int THREADS = VECS > 2048 ? VECS / 8 : 256; // at most 8 vectors a thread
  static constexpr int U = BT * UPR / THREADS;                 // units per thread
  static_assert(THREADS % UPR == 0 && U >= 1 && U * THREADS == BT * UPR, "tile split");
};

constexpr int kDepth = 3;   // heads in flight per CTA (three tiles: up to 96 KB with bf16, two CTAs per SM)

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <typename T, int D, int BT, bool HALF, bool POOL>
__global__ void __launch_bounds__(RopeCfg<T, D, BT, HALF>::THREADS)
rope_kernel(const T* __restrict__ in, const Side si, T* __restrict__ out, const Side so, const RasterMap rm,
            const RopeArgs a, int heads_per_cta, float* __restrict__ means, int32_t* d_status) {
  using C = RopeCfg<T, D, BT, HALF>;
  using X = Row16<T>;
  constexpr int E = C::E;
  __shared__ int4 tok[BT];   // raster token, and its table row per axis
  // POOL: per warp the sums of its unit columns (lanes UPR apart share one)
  constexpr int kPart = C::THREADS / 32 * C::UPR;
  __shared__ float part[POOL ? 2 : 1][POOL ? kPart : 1][POOL ? C::NV * E + 1 : 1];
  extern __shared__ uint4 ring[];   // [min(kDepth, heads)][U][NV][THREADS]
  const int j = blockIdx.x, b = blockIdx.z, H = rm.H;
  const int h0 = blockIdx.y * heads_per_cta, h1 = min(H, h0 + heads_per_cta);
  for (int o = threadIdx.x; o < BT; o += C::THREADS) {
    const int tbc = rm.tb * rm.tc;
    const int bx = j % rm.nX, by = (j / rm.nX) % rm.nY, bt = j / (rm.nX * rm.nY);
    const int it = o / tbc, rem = o - it * tbc, iy = rem / rm.tc, ix = rem - iy * rm.tc;
    int p[3] = {bt * rm.ta + it, by * rm.tb + iy, bx * rm.tc + ix};
    const int n = (p[0] * rm.Y + p[1]) * rm.X + p[2];
    if (a.pos != nullptr) {
      const int32_t* q = a.pos + ((int64_t)b * rm.N + n) * 3;
#pragma unroll
      for (int ax = 0; ax < 3; ++ax) {
        p[ax] = q[ax];
        if (a.cols[ax] > 0 && (p[ax] < 0 || p[ax] >= a.extent[ax])) {
          report(d_status, SPARSP_ERR_DATA);
          p[ax] = -1;   // not turned
        }
      }
    }
    tok[o] = make_int4(n, p[0], p[1], p[2]);
  }
  __syncthreads();
  const int c0 = threadIdx.x % C::UPR;          // this thread's unit column in every row
  const int o0 = threadIdx.x / C::UPR;
  constexpr int kRowStep = C::THREADS / C::UPR;
  float2 cs[C::U][C::NP];
#pragma unroll
  for (int k = 0; k < C::NP; ++k) {
    int i = c0 * C::NP + k, ax = 0;             // pair index -> axis and index within it
    if (i >= a.cols[0] / 2) { i -= a.cols[0] / 2; ax = 1; }
    if (ax == 1 && i >= a.cols[1] / 2) { i -= a.cols[1] / 2; ax = 2; }
    const bool turns = i < a.cols[ax] / 2;
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const int4 tk = tok[o0 + u * kRowStep];
      const int p = ax == 0 ? tk.y : ax == 1 ? tk.z : tk.w;
      float2 v = make_float2(1.f, 0.f);
      if (turns && p >= 0) v = __ldg(a.table + a.base[ax] + (int64_t)p * (a.cols[ax] / 2) + i);
      cs[u][k] = make_float2(v.x, v.y * a.sign);
    }
  }
  auto place = [&](int st, int u, int v) { return ring + ((st * C::U + u) * C::NV + v) * C::THREADS + threadIdx.x; };
  auto fetch = [&](int h, int st) {
    if (h < h1) {
      const T* src0 = in + (si.blocked ? (((int64_t)b * H + h) * rm.N + (int64_t)j * BT) * D
                                       : (int64_t)b * rm.N * si.stride + (int64_t)h * D) + c0 * E;
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        const int o = o0 + u * kRowStep;
        const T* src = src0 + (si.blocked ? (int64_t)o * D : (int64_t)tok[o].x * si.stride);
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
    const int64_t blocked0 = (((int64_t)b * H + h) * rm.N + (int64_t)j * BT) * D;
    float acc[C::NV * E];
#pragma unroll
    for (int e = 0; e < C::NV * E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      float f[C::NV * E];
#pragma unroll
      for (int v = 0; v < C::NV; ++v) X::unpack(*place(st, u, v), f + v * E);
#pragma unroll
      for (int k = 0; k < C::NP; ++k) {
        float& x = f[HALF ? k : 2 * k];
        float& y = f[HALF ? E + k : 2 * k + 1];
        const float r = x * cs[u][k].x - y * cs[u][k].y;
        y = x * cs[u][k].y + y * cs[u][k].x;
        x = r;
      }
      if (POOL)
#pragma unroll
        for (int e = 0; e < C::NV * E; ++e) acc[e] += f[e];
      const int o = o0 + u * kRowStep;
      T* dst = out + (so.blocked ? blocked0 + (int64_t)o * D
                                 : ((int64_t)b * rm.N + tok[o].x) * so.stride + (int64_t)h * D);
#pragma unroll
      for (int v = 0; v < C::NV; ++v) __stcs(reinterpret_cast<uint4*>(dst + c0 * E + v * (D / 2)), X::pack(f + v * E));
    }
    // the means of the fp32 values: summed per thread, over the lanes that share its
    // columns, then over the warps in order
    if constexpr (POOL) {
      float (*sum)[C::NV * E + 1] = part[(h - h0) & 1];   // the other one may still be read
#pragma unroll
      for (int off = 16; off >= C::UPR; off >>= 1)
#pragma unroll
        for (int e = 0; e < C::NV * E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], off);
      if ((threadIdx.x & 31) < C::UPR)
#pragma unroll
        for (int e = 0; e < C::NV * E; ++e) sum[(threadIdx.x >> 5) * C::UPR + c0][e] = acc[e];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += C::THREADS) {
        const int v = HALF ? c / (D / 2) : 0, cc = HALF ? c % (D / 2) : c;
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < C::THREADS / 32; ++g) s += sum[g * C::UPR + cc / E][v * E + cc % E];
        means[(((int64_t)b * H + h) * (rm.N / BT) + j) * D + c] = s * (1.0f / (float)BT);
      }
    }
  }
  copy_wait<0>();
}

__global__ void __launch_bounds__(256)
rope_table_kernel(const RopeArgs a, double theta, double off0, double off1, double off2, double sc0, double sc1,
                  double sc2, float2* __restrict__ table, int64_t total) {
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= total) return;
  const int ax = a.cols[2] > 0 && e >= a.base[2] ? 2 : a.cols[1] > 0 && e >= a.base[1] ? 1 : 0;
  const int half = a.cols[ax] / 2;
  const int64_t p = (e - a.base[ax]) / half, i = (e - a.base[ax]) % half;
  const double off = ax == 0 ? off0 : ax == 1 ? off1 : off2, sc = ax == 0 ? sc0 : ax == 1 ? sc1 : sc2;
  const double phi = (off + sc * (double)p) * pow(theta, -2.0 * (double)i / (double)a.cols[ax]);
  double s, c;
  sincos(phi, &s, &c);
  table[e] = make_float2((float)c, (float)s);
}

RopeArgs args_of(const sparsp_rope_t& r, const float* table) {
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

template <typename T, int D, int BT, bool HALF>
bool go(const Dims& s, const void* in, const Side& si, void* out, const Side& so, const RopeArgs& a, float* means,
        int32_t* d_status, cudaStream_t st) {
  using C = RopeCfg<T, D, BT, HALF>;
  // heads per CTA: as many as leave about four CTAs per SM
  const int64_t tiles = (int64_t)s.nb * s.B;
  const int sms = device_sm_count();
  int64_t hpc = tiles * s.H / ((int64_t)(sms > 0 ? sms : 152) * 4);
  hpc = hpc < 1 ? 1 : hpc > 8 ? 8 : hpc;
  const dim3 grid((unsigned)s.nb, (unsigned)((s.H + hpc - 1) / hpc), (unsigned)s.B);
  const size_t smem = (size_t)(hpc < kDepth ? hpc : kDepth) * C::VECS * 16;
  auto kern = means != nullptr ? rope_kernel<T, D, BT, HALF, true> : rope_kernel<T, D, BT, HALF, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  kern<<<grid, C::THREADS, smem, st>>>((const T*)in, si, (T*)out, so, raster_map(s), a, (int)hpc, means, d_status);
  return true;
}

template <typename T, bool HALF>
bool go_shape(const Dims& s, const void* in, const Side& si, void* out, const Side& so, const RopeArgs& a,
              float* means, int32_t* d_status, cudaStream_t st) {
  if (s.d == 64 && s.Bt == 64) return go<T, 64, 64, HALF>(s, in, si, out, so, a, means, d_status, st);
  if (s.d == 64) return go<T, 64, 128, HALF>(s, in, si, out, so, a, means, d_status, st);
  if (s.Bt == 64) return go<T, 128, 64, HALF>(s, in, si, out, so, a, means, d_status, st);
  return go<T, 128, 128, HALF>(s, in, si, out, so, a, means, d_status, st);
}

}  // namespace

int64_t rope_table_entries(const sparsp_rope_t& r) {
  int64_t n = 0;
  for (int ax = 0; ax < 3; ++ax) n += (int64_t)r.extent[ax] * (r.cols[ax] / 2);
  return n;
}

sparsp_status_t launch_rope_table(const sparsp_rope_t& r, double theta, const double* offset, const double* scale,
                                  float* table, cudaStream_t st) {
  const RopeArgs a = args_of(r, nullptr);
  const int64_t total = rope_table_entries(r);
  if (total == 0) return SPARSP_OK;
  rope_table_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(a, theta, offset[0], offset[1], offset[2],
                                                                     scale[0], scale[1], scale[2], (float2*)table,
                                                                     total);
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_rope(const Dims& s, const sparsp_rope_t& r, const float* table, const int32_t* pos,
                            const void* in, int64_t in_stride, bool in_blocked, void* out, int64_t out_stride,
                            bool out_blocked, bool inverse, float* means, int32_t* d_status, cudaStream_t st) {
  RopeArgs a = args_of(r, table);
  a.pos = pos;
  a.sign = inverse ? -1.f : 1.f;
  const Side si{in_stride, in_blocked}, so{out_stride, out_blocked};
  bool ok;
  if (s.dtype == SPARSP_F32) {
    if (r.half) ok = go_shape<float, true>(s, in, si, out, so, a, means, d_status, st);
    else ok = go_shape<float, false>(s, in, si, out, so, a, means, d_status, st);
  } else {
    if (r.half) ok = go_shape<__nv_bfloat16, true>(s, in, si, out, so, a, means, d_status, st);
    else ok = go_shape<__nv_bfloat16, false>(s, in, si, out, so, a, means, d_status, st);
  }
  if (!ok) return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

}  // namespace sparsp
