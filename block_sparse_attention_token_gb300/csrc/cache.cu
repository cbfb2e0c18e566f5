// Upkeep of a cache of keys and values in 8 bits: the tables and slots of a step from
// the requests' lengths, and the write of its new keys and values.
//
// Tables. Request b holds len tokens in ceil(len / bt) blocks and gets add more:
//   need_b = ceil((len + add) / bt) - ceil(len / bt) blocks, handed out from a list in
// the order of the requests, so that one scan over the requests gives every request its
// place in the list and its place among the packed new tokens. Every CTA scans all requests
// for itself (thousands at most, a few to a thread) and then enters its share of the blocks and
// of the slots, so that no CTA waits for another: the page of a new token comes from the
// list if its block is new, else from a table entry that no one writes. What a call may overwrite
// of its own input (the lengths, the place in the list) is written by the one CTA of a small
// call after its reads, else by a second launch.
//
// Write. A value is held as x = s c, c of e4m3 and s the scale of its block and head:
//   s = 2^e, the smallest e >= -100 with max |x| <= 448 2^e.
// A power of two costs no bit of a floating-point code, makes x / s exact, so that a code is
// one rounding of x and the same for every way of computing it, and lets a block that
// grows be brought to a larger scale with no error but the codes' own subnormals. A run
// of new tokens in one block is one pass: its values wait in registers for their
// maximum. Bound by HBM: 30,720 tokens x 40 heads of 128 take 153 us, 0.91 of a copy's rate
// (K and V of several heads to a CTA, the next ones on their way meanwhile; with one task to a CTA 199). 256 runs of
// one token take 7 us on the device, a chain of four dependent loads; tables of 4,096 requests 14 us, 5 of
// them the scan, of 64 requests 8.
#include <type_traits>

#include "cache.cuh"
#include "rows.cuh"

namespace sparsp {
namespace {

constexpr int kExtendThreads = 1024;
enum { kExtendLists = 1, kExtendState = 2 };   // what a launch writes: table, start and slots; lengths and place

// The sums over the CTA's threads below this one, and of all, of two numbers.
__device__ __forceinline__ void scan2(int64_t (&v)[2], int64_t (&total)[2], int64_t (*sm)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t in[2] = {v[0], v[1]};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t t = __shfl_up_sync(0xffffffffu, in[k], off);
      if (lane >= off) in[k] += t;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 2; ++k) sm[warp][k] = in[k];
  __syncthreads();
  int64_t below[2] = {0, 0};
  total[0] = total[1] = 0;
  for (int w = 0; w < kExtendThreads / 32; ++w)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (w < warp) below[k] += sm[w][k];
      total[k] += sm[w][k];
    }
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = below[k] + in[k] - v[k];
}

__global__ void __launch_bounds__(kExtendThreads)
cache_extend_kernel(const CacheDims c, const CacheExtend a, int what, int32_t* d_status) {
  const int rank = blockIdx.x, ranks = gridDim.x;
  extern __shared__ int32_t sm_req[];
  int32_t* s_start = sm_req;                     // [B] first packed token
  int32_t* s_len = sm_req + a.B;                 // [B] tokens held before, -1: gets no slots
  int32_t* s_place = sm_req + 2 * a.B;           // [B] place in the list of free blocks
  __shared__ int64_t s_scan[kExtendThreads / 32][2];
  __shared__ int32_t s_given;
  const int bt = c.bt, shift = bt == 64 ? 6 : 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t room = (int64_t)a.max_blocks * bt;   // < 2^31
  int used = a.used != nullptr ? *a.used : 0;
  if (used < 0 || used > a.n_free) {             // no such place in the list: nothing to hand out
    report(d_status, SPARSP_ERR_DATA);
    used = a.n_free;
  }
  if (threadIdx.x == 0) s_given = 0;
  const int per = (a.B + kExtendThreads - 1) / kExtendThreads;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  auto blocks_of = [&](int n) { return (int)(((uint32_t)n + bt - 1) >> shift); };    // (with divisions 4,096 requests took 20.5 us, now 14.4)
  // A request's length, new tokens and new blocks; one that makes no sense brings nothing.
  auto sizes = [&](int b, int& len, int& add, int& need) {
    len = a.len[b];
    add = a.add[b];
    const bool ok = len >= 0 && add >= 0 && (int64_t)len + add <= room;
    if (!ok) {
      report(d_status, SPARSP_ERR_DATA);
      add = 0;
    }
    need = ok ? blocks_of(len + add) - blocks_of(len) : 0;
    return ok;
  };
  int64_t v[2] = {0, 0}, total[2];
  for (int b = b0; b < b1; ++b) {
    int len, add, need;
    sizes(b, len, add, need);
    v[0] += add;
    v[1] += need;
  }
  scan2(v, total, s_scan);
  int given = 0;
  for (int b = b0; b < b1; ++b) {
    int len, add, need;
    const bool ok = sizes(b, len, add, need);
    // whoever finds too few blocks waits, and so does everyone behind who needs one
    const bool in = ok && v[0] + add <= a.tokens && (need == 0 || v[1] + need <= a.n_free - used);
    if (ok && !in) report(d_status, SPARSP_ERR_CAPACITY);
    s_start[b] = (int)min(v[0], (int64_t)INT32_MAX);
    s_len[b] = in ? len : -1;
    s_place[b] = used + (in ? (int)v[1] : 0);
    if (in) given += need;
    v[0] += add;
    v[1] += need;
  }
  if (given > 0) atomicAdd(&s_given, given);
  __syncthreads();                               // all of len and used has been read
  if (rank == 0 && (what & kExtendState)) {
    for (int b = b0; b < b1; ++b) {
      const int len = s_len[b];
      a.len_out[b] = len >= 0 ? len + a.add[b] : a.len[b];
    }
    if (threadIdx.x == 0 && a.used_out != nullptr) *a.used_out = used + s_given;
  }
  if (!(what & kExtendLists)) return;
  if (rank == 0) {
    for (int b = b0; b < b1; ++b) a.start[b] = s_start[b];
    if (threadIdx.x == 0) a.start[a.B] = (int)min(total[0], (int64_t)INT32_MAX);
  }
  // a block from the list (-1: none)
  auto handed = [&](int at) {
    const int id = a.free_blocks[at];
    if (id >= 0 && id < c.blocks) return id;
    report(d_status, SPARSP_ERR_DATA);
    return -1;
  };
  // the blocks handed out: a warp takes a request
  for (int b = rank * (kExtendThreads / 32) + warp; b < a.B; b += ranks * (kExtendThreads / 32)) {
    const int len = s_len[b];
    if (len < 0) continue;
    const int have = blocks_of(len), need = blocks_of(len + a.add[b]) - have;
    for (int i = lane; i < need; i += 32) a.table[(int64_t)b * a.max_blocks + have + i] = handed(s_place[b] + i);
  }
  // slots: four packed tokens to a thread, the first one's request by bisection
  for (int64_t t0 = (int64_t)(rank * kExtendThreads + threadIdx.x) * 4; t0 < a.tokens;
       t0 += (int64_t)ranks * kExtendThreads * 4) {
    int lo = 0, hi = a.B;                        // the last request that starts at or before t0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= t0) lo = mid;
      else hi = mid;
    }
    int slot[4], page = -1, page_b = -1, page_j = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      slot[i] = -1;
      if (t >= total[0] || t >= a.tokens) continue;
      while (lo + 1 < a.B && s_start[lo + 1] <= t) ++lo;
      const int len = s_len[lo];
      if (len < 0) continue;
      const int p = len + (int)(t - s_start[lo]), j = p >> shift, have = blocks_of(len);
      if (j != page_j || lo != page_b) {
        page = j >= have ? handed(s_place[lo] + j - have) : a.table[(int64_t)lo * a.max_blocks + j];
        page_j = j;
        page_b = lo;
        if (page < 0 || page >= c.blocks) {
          report(d_status, SPARSP_ERR_DATA);
          page = -1;
        }
      }
      if (page >= 0) slot[i] = (page << shift) + (p & (bt - 1));
    }
    if (t0 + 4 <= a.tokens) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < a.tokens) a.slots[t0 + i] = slot[i];
    }
  }
}

// The scale of values of up to `most` (finite, not negative; as bits): 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(uint32_t most) {
  const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}
// The smallest power of two from 2^-100 on that is not below a scale (0 < x <= 2^120).
__device__ __forceinline__ float power_above(float x) {
  const uint32_t u = __float_as_uint(x);
  const int e = (int)(u >> 23) - 127 + ((u & 0x7fffffu) != 0 ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

constexpr uint32_t kInf = 0x7f800000u;   // magnitudes as bits: from here on not finite

// 16 bytes of new values: their largest magnitude (as fp32 bits; as they come, or of the
// finite ones), and their codes under 1 / scale.
template <typename T>
struct Fresh;
template <>
struct Fresh<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ uint32_t most(const uint4& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  static __device__ __forceinline__ void values(const uint4& v, float* f) { Row16<__nv_bfloat16>::unpack(v, f); }
};
template <>
struct Fresh<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ uint32_t most(const uint4& v) {
    return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
  }
  static __device__ __forceinline__ void values(const uint4& v, float* f) { Row16<float>::unpack(v, f); }
};
template <typename T>
__device__ __forceinline__ uint32_t finite_most(const uint4& v) {
  float f[Fresh<T>::E];
  Fresh<T>::values(v, f);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < Fresh<T>::E; ++e) {
    const uint32_t u = __float_as_uint(f[e]) & 0x7fffffffu;
    if (u < kInf) m = max(m, u);
  }
  return m;
}
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* to, const uint4& v, float inverse, bool finite) {
  constexpr int E = Fresh<T>::E;
  float f[E];
  Fresh<T>::values(v, f);
  if (!finite)   // what is not finite is held as NaN
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!(fabsf(f[e]) < INFINITY)) f[e] = NAN;
  uint32_t code[E / 4];
#pragma unroll
  for (int e = 0; e < E / 4; ++e)
    code[e] = e4m3_pair(f[4 * e] * inverse, f[4 * e + 1] * inverse) |
              e4m3_pair(f[4 * e + 2] * inverse, f[4 * e + 3] * inverse) << 16;
  if (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[E / 4 - 1]);
  else *reinterpret_cast<uint32_t*>(to) = code[0];
}

constexpr int kGranule = 128;     // most packed tokens that one CTA looks for runs in
constexpr int kWriteCtas = 456;   // CTAs that a call is split into where it can be
constexpr int kShortRun = 4;      // tokens of a run that one warp takes by itself
constexpr int kWriteDepth = 2;    // blocks' parts in flight per CTA

// Threads of a CTA: at most eight vectors of a whole block to each.
template <typename T, int D, int BT>
constexpr int write_threads() { return sizeof(T) * D * BT <= 32768 ? 256 : 512; }

// CTA (granule of packed tokens, some heads). A run is new tokens in a row whose slots are next to
// each other in one block; it belongs to the granule it starts in. A short run is a warp's,
// a longer one the CTA's, which takes K and V of its heads one after the other while the
// next ones are on their way into shared memory, each thread's into slots of its own. Every warp
// finds the runs for itself.
template <typename T, int D, int BT>
__global__ void __launch_bounds__(write_threads<T, D, BT>(), sizeof(T) * D * BT <= 32768 ? 3 : 1)
cache_write_kernel(const CacheDims c, const CacheWrite a, int granule, int heads, int32_t* d_status) {
  constexpr int kWriteThreads = write_threads<T, D, BT>();
  constexpr int E = Fresh<T>::E, LPR = D / E;        // lanes per row
  constexpr int kRows = kWriteThreads / LPR, U = BT / kRows;
  extern __shared__ uint4 ring[];                    // [kWriteDepth][U][threads]
  __shared__ uint32_t s_most[2][kWriteThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h0 = blockIdx.y * heads, tasks = 2 * (min(c.heads, h0 + heads) - h0);   // K and V of a head in turn
  const int64_t capacity = (int64_t)c.blocks * BT, t0 = (int64_t)blockIdx.x * granule;
  int turn = 0, buf = 0;

  // Where a task's new values of packed token `first` start.
  auto source = [&](int task, int64_t first) {
    const int h = h0 + (task >> 1);
    return task & 1 ? static_cast<const T*>(a.v) + first * a.v_token + h * a.v_head
                    : static_cast<const T*>(a.k) + first * a.k_token + h * a.k_head;
  };
  // The part of a run that thread t of kThreads holds in w: row t / LPR + u kThreads / LPR, vector t % LPR.
  auto hold = [&](int task, int slot, int count, int t, const auto& w, auto threads, auto reduce) {
    constexpr int kPer = decltype(threads)::value / LPR, kU = sizeof(w) / sizeof(uint4);
    const int c0 = t % LPR, r0 = t / LPR, block = slot / BT, off = slot % BT;
    const int64_t at = (int64_t)block * c.heads + h0 + (task >> 1);
    float* scale_at = (task & 1 ? a.vs : a.ks) + at;
    uint8_t* base = (task & 1 ? a.vc : a.kc) + at * BT * D;
    const float old = off > 0 ? *scale_at : 0.f;
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (r0 + u * kPer < count) most = max(most, Fresh<T>::most(w[u]));
    most = reduce(most);                             // also: every thread has read the old scale
    const bool finite = most < kInf;
    if (!finite) {
      if (t == 0) report(d_status, SPARSP_ERR_DATA);
      most = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (r0 + u * kPer < count) most = max(most, finite_most<T>(w[u]));
      most = reduce(most);
    }
    float scale = scale_of(most);
    const bool kept = old > 0.f && old <= 0x1p120f;  // of older tokens (never of off == 0)
    if (off > 0 && !kept && t == 0) report(d_status, SPARSP_ERR_DATA);   // codes without a scale stay as they are
    if (kept) scale = fmaxf(scale, power_above(old));
    if (t == 0) *scale_at = scale;
    const float inverse = __uint_as_float((254u << 23) - __float_as_uint(scale));   // of a power of two
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (r0 + u * kPer < count)
        store_codes<T>(base + (off + r0 + u * kPer) * D + c0 * E, w[u], inverse, finite);
    if (kept && scale != old) {                      // older tokens, brought to the larger scale
      // eight (four) words at a time, as a warp may have 127 rows to bring along: 256 runs of one token with cold caches
      // took 43 us word by word, not 19
      constexpr int kStep = decltype(threads)::value, kAt = kStep == 32 ? 8 : 4;
      const float ratio = old * inverse;
      uint32_t* codes = reinterpret_cast<uint32_t*>(base) + t;
      for (int n = off * D / 4 - t; n > 0; n -= kAt * kStep, codes += kAt * kStep) {
        uint32_t held[kAt];
#pragma unroll
        for (int k = 0; k < kAt; ++k) held[k] = k * kStep < n ? codes[k * kStep] : 0;
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
          const float2 lo = e4m3_values(held[k]), hi = e4m3_values(held[k] >> 16);
          if (k * kStep < n)
            codes[k * kStep] = e4m3_pair(lo.x * ratio, lo.y * ratio) | e4m3_pair(hi.x * ratio, hi.y * ratio) << 16;
        }
      }
    }
  };

  for (int g0 = 0; g0 < granule; g0 += 32) {
    const int64_t t = t0 + g0 + lane;
    bool head = false;
    if (g0 + lane < granule && t < a.tokens) {
      const int slot = a.slots[t];
      if (slot >= capacity) report(d_status, SPARSP_ERR_DATA);
      else head = slot >= 0 && (t == 0 || slot % BT == 0 || a.slots[t - 1] != slot - 1);
    }
    for (uint32_t starts = __ballot_sync(0xffffffffu, head); starts != 0; starts &= starts - 1) {
      const int64_t first = t0 + g0 + __ffs(starts) - 1;
      const int slot = a.slots[first], room = BT - slot % BT;
      int count = 0;                                 // tokens that follow one another in the block
      for (int i = 0; i < room; i += 32) {
        const int r = i + lane;
        const uint32_t on = __ballot_sync(0xffffffffu, r < room && first + r < a.tokens && a.slots[first + r] == slot + r);
        count += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
        if (on != 0xffffffffu) break;
      }
      if (count <= kShortRun) {
        constexpr int kU = kShortRun * LPR / 32;
        for (int task = 0; task < tasks; ++task) {
          if (turn++ % (kWriteThreads / 32) != warp) continue;
          const int64_t stride = task & 1 ? a.v_token : a.k_token;
          const T* from = source(task, first) + lane % LPR * E;
          uint4 w[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (lane / LPR + u * (32 / LPR) < count)
              w[u] = __ldg(reinterpret_cast<const uint4*>(from + (lane / LPR + u * (32 / LPR)) * stride));
          hold(task, slot, count, lane, w, std::integral_constant<int, 32>{},
               [](uint32_t v) { return __reduce_max_sync(0xffffffffu, v); });
        }
      } else {
        auto place = [&](int st, int u) { return ring + (st * U + u) * kWriteThreads + threadIdx.x; };
        auto fetch = [&](int task) {
          if (task < tasks) {
            const int64_t stride = task & 1 ? a.v_token : a.k_token;
            const int r0 = threadIdx.x / LPR;
            const T* from = source(task, first) + r0 * stride + threadIdx.x % LPR * E;
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (r0 + u * kRows < count) copy_async16(place(task % kWriteDepth, u), from + u * kRows * stride);
          }
          copy_commit();
        };
        for (int i = 0; i < kWriteDepth - 1; ++i) fetch(i);
        for (int task = 0; task < tasks; ++task) {
          fetch(task + kWriteDepth - 1);
          copy_wait<kWriteDepth - 1>();
          uint4 w[U];
#pragma unroll
          for (int u = 0; u < U; ++u) w[u] = *place(task % kWriteDepth, u);
          hold(task, slot, count, (int)threadIdx.x, w, std::integral_constant<int, kWriteThreads>{}, [&](uint32_t v) {
            v = __reduce_max_sync(0xffffffffu, v);
            if (lane == 0) s_most[buf][warp] = v;
            __syncthreads();                         // the buffers alternate: one barrier is enough
#pragma unroll
            for (int i = 0; i < kWriteThreads / 32; ++i) v = max(v, s_most[buf][i]);
            buf ^= 1;
            return v;
          });
        }
        copy_wait<0>();
      }
    }
  }
}

template <typename T, int D, int BT>
bool go_write(const CacheDims& c, const CacheWrite& a, int32_t* d_status, cudaStream_t st) {
  // granules and groups of heads as large as still leave three CTAs per SM
  int granule = kGranule, heads = 8;
  auto ctas = [&] { return (int64_t)((a.tokens + granule - 1) / granule) * ((c.heads + heads - 1) / heads); };
  while (heads > 1 && ctas() < kWriteCtas) heads /= 2;
  while (granule > 4 && ctas() < kWriteCtas) granule /= 2;
  const size_t smem = (size_t)kWriteDepth * BT * D * sizeof(T);
  auto kern = cache_write_kernel<T, D, BT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  const dim3 grid((unsigned)((a.tokens + granule - 1) / granule), (unsigned)((c.heads + heads - 1) / heads));
  kern<<<grid, write_threads<T, D, BT>(), smem, st>>>(c, a, granule, heads, d_status);
  return true;
}

template <typename T>
bool go_write_shape(const CacheDims& c, const CacheWrite& a, int32_t* d_status, cudaStream_t st) {
  if (c.d == 64 && c.bt == 64) return go_write<T, 64, 64>(c, a, d_status, st);
  if (c.d == 64) return go_write<T, 64, 128>(c, a, d_status, st);
  if (c.bt == 64) return go_write<T, 128, 64>(c, a, d_status, st);
  return go_write<T, 128, 128>(c, a, d_status, st);
}

}  // namespace

sparsp_status_t launch_cache_extend(const CacheDims& c, const CacheExtend& a, int32_t* d_status, cudaStream_t st) {
  const size_t smem = (size_t)a.B * 3 * sizeof(int32_t);
  if (cudaFuncSetAttribute(cache_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  // one CTA where a thread has at most four requests and eight tokens, else enough for four tokens a thread
  const int64_t share = (int64_t)4 * kExtendThreads;
  const int ctas = a.tokens <= 2 * share && a.B <= share ? 1 : (int)min((int64_t)152, max((int64_t)8, a.tokens / share));
  const bool over = a.len_out == a.len || (a.used != nullptr && a.used_out == a.used);
  if (ctas > 1 && over) {
    cache_extend_kernel<<<ctas, kExtendThreads, smem, st>>>(c, a, kExtendLists, d_status);
    cache_extend_kernel<<<1, kExtendThreads, smem, st>>>(c, a, kExtendState, nullptr);
  } else {
    cache_extend_kernel<<<ctas, kExtendThreads, smem, st>>>(c, a, kExtendLists | kExtendState, d_status);
  }
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_cache_write(const CacheDims& c, int dtype, const CacheWrite& a, int32_t* d_status,
                                   cudaStream_t st) {
  if (a.tokens == 0) return SPARSP_OK;
  if (!(dtype == SPARSP_F32 ? go_write_shape<float>(c, a, d_status, st)
                            : go_write_shape<__nv_bfloat16>(c, a, d_status, st)))
    return SPARSP_ERR_CUDA;
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

}  // namespace sparsp
