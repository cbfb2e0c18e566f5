// Attention over a cache of keys and values in 8 bits, found through block tables, for
// packed queries of many requests.
//
//   O = sum_j softmax_j(scale ks_j q.K_j) vs_j V_j, K and V the e4m3 codes, ks and vs the
// scales of their block and key head. The products run on the codes: an e4m3 code is
// exact in 16 bits, ks multiplies a score and vs a sum over one block's keys in fp32.
//
// Few queries: bound by the cache's bytes. A warp holds the scores transposed, S^T = K Q^T
// (16 keys by 8 query rows: heads that share a key head, and new tokens, side by side), so that
// few rows fill a matrix instruction; O^T = V^T P^T. The codes go from shared memory into
// registers in the operands' own layout: the columns of the head are permuted alike in Q and
// K, and the rows of V^T are columns of vectors that a lane reads anyway. Every warp has a ring of
// stages of its own, filled by TMA. Work is counted in units of 64 keys over all requests
// and key heads and dealt out evenly: a CTA takes a range of units, and an item (request, key head, 8 or 16 rows) that
// spans several CTAs leaves partial results that a second kernel joins in order. vs goes into the weights and out of
// their sum again (cache_items.cuh), so that the products of all blocks add up in place.
// Measured (32 heads over 8, d = 128): 64 uneven requests of up to 32,768 tokens 80 us (0.82 of a copy's rate); 8 x 4
// rows over a tenth of 131,072 keys 56 us (0.56; 20 us of it fixed: scan and look-ups at the latency of a cold cache,
// the warps' join, the second kernel); one request of 1,024 keys 11 us on the device.
#include "cache_items.cuh"
#include "rows.cuh"

namespace sparsp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGrid = 152 * 3;     // CTAs that share the work, at most (the workspace depends on it)
// CTAs per SM: what the accumulators of 8 or 16 rows leave registers for (three with 16 rows and d = 128 spill 260
// bytes a thread: 75 us in the place of 67 for the sparse lists above).
constexpr int ctas_per_sm(int d, int nt) { return d == 128 && nt == 2 ? 2 : 3; }
// Units of a piece from which on a warp takes whole units: at 8, 16, 32 one request of 1,024 keys takes 16.4, 15.4,
// 15.5 us, 16 uneven requests 70.8, 70.2, 72.8.
constexpr int kWideUnits = 16;
// Units that an item's own work (its look-ups, queries, join) counts as: 16 uneven requests of 40 heads, d = 64, take
// 99 us at 2, 71 at 4, 69 at 6, 71 at 8, 73 at 12; 256 requests of at most 256 keys 32, 33, 34, 34 from 4 on.
constexpr int kItemCost = 6;
constexpr int kMinUnits = kItemCost + 2;   // units, an item's own among them, that are worth a CTA
constexpr float kPScale = 2048.f;  // P is at most 16 and is held as 2^11 P in f16: 2^-35 is not lost

template <int RT>   // query rows of an item
struct Walk {
  const CacheAttn& a;
  __device__ __forceinline__ Entry at(int e, bool tell) const {
    Entry x = entry_at(a, e, tell);
    if (a.few > 0 && (int64_t)x.n * a.group > a.few) x.n = 0;   // the other kernel's
    x.groups = (int)(((int64_t)x.n * a.group + RT - 1) / RT);
    // an item without keys still has its rows to write: one unit, empty
    x.weight = (int64_t)x.groups * (kItemCost + max(1, x.units)) * (a.row_ptr != nullptr ? 1 : a.c.heads);
    return x;
  }
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
// A warp's ring of 16-key stages, filled by TMA (swizzled by the length of a row, so that the reads
// below meet no bank twice) and waited for on a barrier per stage.
constexpr int kStages = 3;         // 3, 4, 5, 6: 59.9, 60.7, 62.5, 63.6 us for the sparse lists above
constexpr uint64_t kWaitNs = 2000000000ull;
template <int D>
struct Stage {
  uint8_t k[16 * D], v[16 * D];
};
// Where a lane (g, t) finds its vectors of a stage. K: rows g and g + 8; D = 128: 16-byte vectors 2t and 2t + 1,
// D = 64: vector t. V: rows 2t, 2t + 1 (and 8 further), columns D/8 g ...
template <int D>
__device__ __forceinline__ int at_k(int g, int t, int s) {
  return D == 128 ? g * 128 + (((2 * t + s) ^ g) << 4) : g * 64 + ((t ^ (g >> 1)) << 4);
}
template <int D>
__device__ __forceinline__ int at_v(int g, int t, int i) {
  const int r = 2 * t + i;
  return D == 128 ? r * 128 + ((g ^ r) << 4) : r * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
}

// Waits for a phase, at most kWaitNs; the whole warp gets the same answer.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    do ok = tc::mbar_try_wait(bar, parity);
    while (!ok && globaltimer_ns() - t0 < kWaitNs);
  }
  return __all_sync(0xffffffffu, ok);
}

template <int D, int NT>
constexpr int attn_smem() {
  constexpr int ring = kWarps * kStages * (int)sizeof(Stage<D>);
  constexpr int sums = kWarps * 8 * NT * (D + 4) * 4;    // the warps' sums, over the ring
  return (ring > sums ? ring : sums) + 1024;               // + alignment slack
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT))
attn_cache_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const CacheAttn a,
                  const Parts parts) {
  constexpr int RT = 8 * NT, SEG = D / 64;
  const Walk<RT> walk{a};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);   // swizzle atoms
  Stage<D>* ring = reinterpret_cast<Stage<D>*>(smem) + warp * kStages;
  __shared__ uint64_t s_full[kWarps][kStages];
  auto full = [&](int st) { return tc::smem_u32(&s_full[warp][st]); };
  uint32_t phases = 0;                         // of the stages' barriers
  bool late = false;                           // a wait has expired: nothing more is copied, what is on its way is waited for
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(full(i), 1);
    tc::fence_barrier_init();
  }
  __syncwarp();
  float (*s_o)[RT][D + 4] = reinterpret_cast<float (*)[RT][D + 4]>(smem);
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_begin[2];               // first entry, its unit offset
  __shared__ __align__(16) __half s_q[RT][D + 8];
  __shared__ float s_factor[RT];
  __shared__ float s_m[kWarps][RT], s_l[kWarps][RT], s_lu[kWarps];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // ---- this CTA's range of units
  const int entries = entries_of(a), per = (entries + kThreads - 1) / kThreads;
  const int e0 = min(entries, (int)threadIdx.x * per), e1 = min(entries, e0 + per);
  int64_t mine = 0;
  for (int e = e0; e < e1; ++e) mine += walk.at(e, blockIdx.x == 0).weight;
  int64_t total;
  const int64_t below = scan_below<kWarps>(mine, s_scan, &total);
  const int64_t ctas = min((int64_t)gridDim.x, max((int64_t)1, (total + kMinUnits - 1) / kMinUnits)), cta = blockIdx.x;
  const int64_t begin = cta * total / ctas, end = cta < ctas ? (cta + 1) * total / ctas : begin;
  if (threadIdx.x == 0) parts.open[cta].last = -1;
  if (cta >= ctas || begin >= end) return;      // the same for the whole CTA
  if (below <= begin && begin < below + mine) {
    int64_t at = below;
    int e = e0;
    for (;; ++e) {
      const int64_t w = walk.at(e, false).weight;
      if (begin < at + w) break;
      at += w;
    }
    s_begin[0] = e;
    s_begin[1] = begin - at;
  }
  __syncthreads();
  int entry = (int)s_begin[0];
  int64_t offset = s_begin[1], unit_at = begin;
  Entry x = walk.at(entry, false);

  while (unit_at < end) {
    while (offset >= x.weight) {               // entries without queries weigh nothing
      offset -= x.weight;
      x = walk.at(++entry, false);
    }
    // ---- an item, and this CTA's piece [u0, u1) of it
    // (its first kItemCost units stand for its own work and go with the first of its keys)
    const int units = max(1, x.units), size = kItemCost + units;
    const int item = (int)(offset / size), at0 = (int)(offset - (int64_t)item * size);
    const int at1 = (int)min((int64_t)size, at0 + (end - unit_at));
    const int64_t item_at = unit_at - at0;
    const int u0 = max(0, at0 - kItemCost), u1 = at1 - kItemCost;
    unit_at += at1 - at0;
    offset += at1 - at0;
    if (u1 <= u0) continue;
    const int hk = a.row_ptr != nullptr ? x.hk : item / x.groups, group = a.row_ptr != nullptr ? item : item % x.groups;
    const int row0 = group * RT, rows = min(RT, x.n * a.group - row0);
    const int32_t* table = a.table + (int64_t)x.b * a.max_blocks;
    const int32_t* list = a.row_ptr != nullptr ? a.col_idx + a.row_ptr[entry] : nullptr;
    const int shift = a.c.bt == kUnit ? 0 : 1, stop = min(u1, x.units);   // units per block, log2
    // A warp's steps of 16 keys: in a long piece the four of every fourth unit, so that a look-up serves
    // four steps; in a short one a quarter of every unit, so that all warps have work.
    const bool wide = u1 - u0 >= kWideUnits;
    const int first_unit = wide ? u0 + warp : u0, stride = wide ? 4 : 1;
    const int steps = wide ? max(0, u1 - first_unit + 3) / 4 * 4 : u1 - u0;

    // The key block of a unit and its place in the pool, looked up ahead of the copies: the list
    // two units of this warp ahead, the table one.
    auto block_of = [&](int u) -> int {        // -1: none
      if (u >= stop) return -1;
      return list != nullptr ? __ldg(list + (u >> shift)) : u >> shift;
    };
    auto page_of = [&](int u, int j) -> int {  // -1: none
      if (u >= stop) return -1;
      if (!has_tokens(a, x, j)) {
        report(a.d_status, SPARSP_ERR_DATA);
        return -1;
      }
      return __ldg(table + j);
    };
    int unit = first_unit;                     // the next one to be copied
    int block1 = block_of(unit), page1 = page_of(unit, block1), block2 = block_of(unit + stride);
    int pos = 0, exist = 0;                    // of the unit being copied: its first key, how many there are
    int row = 0, page = 0;                     // its place in the pool
    int first[kStages], valid[kStages];        // position of a stage's first key, and how many exist
    float ks[kStages], vs[kStages];
    // Copies step i into stage st; i rises by one from call to call.
    auto ahead = [&](int i, int st) {
      if (i < steps && (!wide || (i & 3) == 0)) {
        const int in_block = (unit & ((1 << shift) - 1)) * kUnit;
        exist = 0;
        if (in_pool(a, page1)) {
          pos = (block1 << shift) * kUnit + in_block;
          exist = min(kUnit, x.len - pos);
          row = hk * a.c.bt + in_block;
          page = page1;
        } else if (unit < stop) {
          report(a.d_status, SPARSP_ERR_DATA);
        }
        block1 = block2;
        page1 = page_of(unit + stride, block1);
        block2 = block_of(unit + 2 * stride);
        unit += stride;
      }
      valid[st] = 0;
      if (i < steps) {
        const int q = 16 * (wide ? i & 3 : warp);
        first[st] = pos + q;
        valid[st] = late ? 0 : max(0, min(16, exist - q));
        if (valid[st] > 0) {
          const int64_t block = (int64_t)page * a.c.heads + hk;
          ks[st] = __ldg(a.ks + block);
          vs[st] = __ldg(a.vs + block);
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(full(st), (uint32_t)sizeof(Stage<D>));
            tc::tma_load_3d(tc::smem_u32(ring[st].k), &map_k, full(st), 0, row + q, page);
            tc::tma_load_3d(tc::smem_u32(ring[st].v), &map_v, full(st), 0, row + q, page);
          }
        }
      }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) ahead(s, s);

    // ---- Q: f16 under a power of two per row
    for (int r = warp * (32 / (D / 8)) + lane / (D / 8); r < RT; r += kWarps * (32 / (D / 8))) {
      const int c = lane % (D / 8);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
      if (r < rows) {
        const int tok = (row0 + r) / a.group, h = hk * a.group + (row0 + r) % a.group;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(x.s0 + tok) * a.q_token + (int64_t)h * D) + c);
        const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(p[i] << 16);
          f[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
        }
      }
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fabsf(f[i]) < INFINITY ? fmaxf(most, fabsf(f[i])) : most;
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // 2^14 <= most * 2^-e < 2^15 (bf16's 8 bits stay whole down to 2^-32 of the row's largest)
      const int e = max(-100, (int)(__float_as_uint(most) >> 23) - 127 - 14);   // at most 113
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      uint4 w;
      w.x = pack_f16(f[0] * down, f[1] * down);
      w.y = pack_f16(f[2] * down, f[3] * down);
      w.z = pack_f16(f[4] * down, f[5] * down);
      w.w = pack_f16(f[6] * down, f[7] * down);
      *reinterpret_cast<uint4*>(&s_q[r][c * 8]) = w;
      if (c == 0) s_factor[r] = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
    }
    __syncthreads();
    uint32_t qf[NT][D / 16][2];
    float factor[NT][2];
    int last[NT][2];                            // the last key position that a row sees
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint2 w = *reinterpret_cast<const uint2*>(&s_q[j * 8 + g][(D == 128 ? 32 * t + 16 * (s / 4) : 16 * t) + 4 * (s % 4)]);
        qf[j][s][0] = w.x;
        qf[j][s][1] = w.y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = j * 8 + 2 * t + i;
        factor[j][i] = s_factor[r];
        last[j][i] = a.causal ? x.len - x.n + (row0 + r) / a.group : INT32_MAX;
      }
    }
    float m[NT][2], l[NT][2], o[NT][D / 16][4], lu = -INFINITY;   // lu: log2 u, of this warp
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m[j][0] = m[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
    }

    auto step = [&](const Stage<D>& st, int at, int n, float ks, float vs) {
      // vs / u goes into the weights, and out of their sum again: one fma less for every element of O
      const float lvs = __log2f(fmaxf(vs, kLeastScale)), up = lvs - lu;   // (the same for the whole warp)
      const bool rises = !(up <= kAbove), sinks = up < -kBelow;
      if (rises) lu = lvs;
      const float lv = rises || sinks ? 0.f : up, inv = exp2_fast(-lv);
      const int nv = sinks ? 0 : n;             // how many have values
      float c[NT][4], c2[NT][4];                // two sums, so that products need not wait for one another
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[j][i] = c2[j][i] = 0.f;
#pragma unroll
      for (int s4 = 0; s4 < SEG; ++s4) {
        const uint8_t* p = st.k + at_k<D>(g, t, s4);
        const uint4 ka = *reinterpret_cast<const uint4*>(p), kb = *reinterpret_cast<const uint4*>(p + 8 * D);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = f16x2_of_e4m3(wa[i]), a1 = f16x2_of_e4m3(wb[i]), a2 = f16x2_of_e4m3(wa[i] >> 16),
                         a3 = f16x2_of_e4m3(wb[i] >> 16);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma(i & 1 ? c2[j] : c[j], a0, a1, a2, a3, qf[j][s4 * 4 + i][0], qf[j][s4 * 4 + i][1]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[j][i] += c2[j][i];
      bool moved = rises;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = score_factor<false>(factor[j][i], ks);
          c[j][i] = g < n && at + g <= last[j][i] ? fmaf(c[j][i], f, lv) : -INFINITY;
          c[j][2 + i] = g + 8 < n && at + g + 8 <= last[j][i] ? fmaf(c[j][2 + i], f, lv) : -INFINITY;
          // the maximum follows when a score passes it by more than 2^4
          moved |= fmaxf(c[j][i], c[j][2 + i]) > m[j][i] + 4.f;
        }
      if (__any_sync(0xffffffffu, moved)) {
        const float down = rises ? exp2_fast(-up) : 1.f;     // 0 for the first
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float corr[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(m[j][i], fmaxf(c[j][i], c[j][2 + i]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            corr[i] = 1.f;
            if (top > m[j][i] + 4.f) {                 // by itself: not by what other rows hold
              corr[i] = exp2_fast(m[j][i] - top);      // 0 for the first
              l[j][i] *= corr[i];
              m[j][i] = top;
            }
            corr[i] *= down;
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[j][i][k] *= corr[k & 1];
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = c[j][i] == -INFINITY ? 0.f : exp2_fast(c[j][i] - m[j][i & 1]);
        }
        l[j][0] = fmaf(e[0] + e[2], inv, l[j][0]);
        l[j][1] = fmaf(e[1] + e[3], inv, l[j][1]);
        p[j][0] = transposed(pack_f16(e[0] * kPScale, e[1] * kPScale));
        p[j][1] = transposed(pack_f16(e[2] * kPScale, e[3] * kPScale));
      }
      uint32_t v[4][D / 32];                     // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = st.v + at_v<D>(g, t, i & 1) + (i >> 1) * 8 * D;
        if (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(p);
          v[i][0] = w.x;
          v[i][1] = w.y;
          v[i][D / 32 - 2] = w.z;
          v[i][D / 32 - 1] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          v[i][0] = w.x;
          v[i][1] = w.y;
        }
      }
      if (nv < 16)                               // what lies past the last token may be anything
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * t + (i & 1) + 8 * (i >> 1) >= nv)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) v[i][k] = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
        const uint32_t lo = __byte_perm(v[0][i / 2], v[1][i / 2], sel);
        const uint32_t hi = __byte_perm(v[2][i / 2], v[3][i / 2], sel);
        const uint32_t a0 = f16x2_of_e4m3(lo), a1 = f16x2_of_e4m3(lo >> 16), a2 = f16x2_of_e4m3(hi),
                       a3 = f16x2_of_e4m3(hi >> 16);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma(o[j][i], a0, a1, a2, a3, p[j][0], p[j][1]);
      }
    };

    for (int i = 0; i < steps; i += kStages) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {
        ahead(i + s + kStages - 1, (s + kStages - 1) % kStages);
        if (i + s < steps && valid[s] > 0) {
          if (!wait_for(full(s), (phases >> s) & 1u)) {
            late = true;
            report(a.d_status, SPARSP_ERR_TIMEOUT);
          }
          phases ^= 1u << s;
          step(ring[s], first[s], valid[s], ks[s], vs[s]);
          __syncwarp();                          // before the stage is filled again
        }
      }
    }

    // ---- join the warps
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], off);
        if (g == 0) {
          s_m[warp][j * 8 + 2 * t + i] = m[j][i];
          s_l[warp][j * 8 + 2 * t + i] = l[j][i];
        }
      }
    if (lane == 0) s_lu[warp] = lu;
    __syncthreads();                            // the rings are done with
    float high = s_lu[0];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) high = fmaxf(high, s_lu[q]);
    const float u = exp2_fast(high), mine_u = lu == -INFINITY ? 0.f : exp2_fast(lu - high) * (1.f / kPScale);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<float2*>(&s_o[warp][j * 8 + 2 * t + k][D / 8 * g + 2 * i]) =
              make_float2(o[j][i][k] * mine_u, o[j][i][k + 2] * mine_u);
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;
    const int slot = 2 * (int)cta + (u0 > 0 ? 0 : 1);     // a piece that goes on is the CTA's first
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float top = s_m[0][r], sum = 0.f;
      float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 1; q < kWarps; ++q) top = fmaxf(top, s_m[q][r]);
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        // a warp that saw nothing has a sum of 0; one that saw only NaN has no maximum, but a sum
        if (s_l[q][r] == 0.f) continue;
        const float f = s_m[q][r] == -INFINITY ? 1.f : exp2_fast(s_m[q][r] - top);
        const float4 w = *reinterpret_cast<const float4*>(&s_o[q][r][c]);
        sum = fmaf(f, s_l[q][r], sum);
        all.x = fmaf(f, w.x, all.x);
        all.y = fmaf(f, w.y, all.y);
        all.z = fmaf(f, w.z, all.z);
        all.w = fmaf(f, w.w, all.w);
      }
      const bool none = sum == 0.f;
      const float f = none ? 0.f : 1.0f / sum, lse2 = top + log2f(sum);   // (u by itself: a scale may be tiny)
      all = make_float4(all.x * f * u, all.y * f * u, all.z * f * u, all.w * f * u);
      if (whole) {
        finish<D>(a, x.s0, hk, row0 + r, c, none, lse2, all);
      } else {
        *reinterpret_cast<float4*>(parts.o + ((int64_t)slot * RT + r) * D + c) = all;
        if (c == 0) parts.ml[(int64_t)slot * RT + r] = make_float2(none ? -INFINITY : lse2, none ? 0.f : 1.f);
      }
    }
    if (!whole && u0 == 0 && threadIdx.x == 0) {
      parts.open[cta] = Open{hk, row0, rows, x.s0, (int)(((item_at + size) * ctas - 1) / total)};
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // the sums, before the rings are filled again
    __syncthreads();
  }
}

// CTA c joins the parts of the item that starts in CTA c of the kernel above and goes on in
// others: warps take every eighth part of a row, then their sums are joined in order. (Thousands of CTAs, most
// without work: with 43 registers, five per SM, 32 requests of 8 tokens take 166 us in the place of 164.)
template <int D, int NT>
__global__ void __launch_bounds__(256, 8)
attn_cache_join_kernel(const CacheAttn a, const Parts parts) {
  constexpr int RT = 8 * NT, W = 8, L = D / 4;           // L lanes hold a row
  __shared__ float s_top[W], s_sum[W];
  __shared__ float4 s_all[W][L];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const Open it = parts.open[blockIdx.x];
  const int r = blockIdx.y;
  if (it.last < 0 || r >= it.rows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = it.last - (int)blockIdx.x + 1;
  auto slot_of = [&](int i) { return (int64_t)(2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0)); };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < count; i += 256) top = fmaxf(top, parts.ml[slot_of(i) * RT + r].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, s_top[i]);
  float sum = 0.f;
  float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < count; i += W) {
    const float f = part_weight(parts.ml[slot_of(i) * RT + r], top);
    sum += f;
    if (lane < L) {
      const float4 w = *reinterpret_cast<const float4*>(parts.o + (slot_of(i) * RT + r) * D + 4 * lane);
      all.x = fmaf(f, w.x, all.x);
      all.y = fmaf(f, w.y, all.y);
      all.z = fmaf(f, w.z, all.z);
      all.w = fmaf(f, w.w, all.w);
    }
  }
  if (lane == 0) s_sum[warp] = sum;
  if (lane < L) s_all[warp][lane] = all;
  __syncthreads();
  if (threadIdx.x >= L) return;
  sum = 0.f;
  all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float4 w = s_all[i][threadIdx.x];
    sum += s_sum[i];
    all.x += w.x;
    all.y += w.y;
    all.z += w.z;
    all.w += w.w;
  }
  finish_join<D>(a, it.s0, it.hk, it.row0 + r, 4 * threadIdx.x, top, sum, all);
}

// Query rows of an item here: 8 where no request has more.
int rows_of(int group, int max_add) { return (int64_t)group * max_add <= 8 ? 8 : 16; }

template <int D, int NT>
sparsp_status_t go(const CacheAttn& a, void* ws, cudaStream_t st) {
  const Parts p = parts_of(ws, kGrid, 8 * NT);
  constexpr int smem = attn_smem<D, NT>();
  const int ctas = 152 * ctas_per_sm(D, NT);
  if (cudaFuncSetAttribute(attn_cache_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  CUtensorMap map_k, map_v;
  if (!make_tmap_codes(&map_k, a.kc, (uint64_t)D, (uint64_t)a.c.heads * a.c.bt, (uint64_t)a.c.blocks, 16) ||
      !make_tmap_codes(&map_v, a.vc, (uint64_t)D, (uint64_t)a.c.heads * a.c.bt, (uint64_t)a.c.blocks, 16))
    return SPARSP_ERR_CUDA;
  attn_cache_kernel<D, NT><<<ctas, kThreads, smem, st>>>(map_k, map_v, a, p);
  SPARSP_LAUNCH_CHECK();
  return launch_after(attn_cache_join_kernel<D, NT>, dim3(ctas, 8 * NT), 256, st, a, p);
}

// Requests with up to kFew rows (tokens times heads that share a key head) are this file's
// kernel's, the others those of attn_cache_tc.cu. Only the device knows the requests, so where there may be both
// both are launched (the one without work takes 8 us); a single request is taken at its word, max_add.
// 32 requests of 8,192 keys, 8 key heads of 128, with 16, 32, 64, 128 rows: here 122, 163, 255, 433 us (rows beyond 16 read
// the cache again), there 178, 204, 218, 237 (8 of each a captured call's own).
constexpr int kFew = 32;
bool many(int group, int max_add) { return (int64_t)group * max_add > kFew; }

}  // namespace

size_t attn_cache_ws(const CacheDims& c, int group, int max_add) {
  const size_t few = parts_bytes(kGrid, rows_of(group, max_add), c.d);
  return many(group, max_add) ? parts_align(few) + attn_cache_tc_ws(c) : few;
}

sparsp_status_t launch_attn_cache(const CacheAttn& args, void* ws, cudaStream_t st) {
  CacheAttn a = args;
  const int rows = rows_of(a.group, a.max_add);
  a.few = 0;
  if (many(a.group, a.max_add)) {
    const bool all = a.B == 1;
    a.few = all ? 0 : kFew;
    const sparsp_status_t r =
        launch_attn_cache_tc(a, (uint8_t*)ws + parts_align(parts_bytes(kGrid, rows, a.c.d)), st);
    if (r != SPARSP_OK || all) return r;
  }
  if (a.c.d == 64) return rows == 8 ? go<64, 1>(a, ws, st) : go<64, 2>(a, ws, st);
  return rows == 8 ? go<128, 1>(a, ws, st) : go<128, 2>(a, ws, st);
}

}  // namespace sparsp
