// Attention over a cache of keys and values in 8 bits for many queries of a request (whole
// frames, prompts): the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
//   O = sum_j softmax_j(scale ks_j q.K_j) vs_j V_j, K and V the e4m3 codes.
//
// S = Q K^T runs on the codes themselves at the rate of 8-bit products: a bf16 query has 8
// significant bits, and under a power of two per row it is the sum of two e4m3 values, q1 = e4m3(q)
// and q2 = e4m3(q - q1), but for what lies below 2^-18 of its row's largest value. Two products
// of 8 bits cost what one of 16 does, and K needs no widening. O += P V takes P in f16 (11
// bits) and V widened to f16, where an e4m3 code is exact, by four warps on its way.
// The scale of a block's values goes into the exponent: with y the score in base 2 and R the
// row's reference,
//   P = 2^(y + log2 vs - R),  O = sum P V / l,  l = sum P / vs,  LSE = (R + log2 l) ln 2,
// so that blocks of any scales add up in one accumulator; P is at most 2^15 (R follows when
// it is passed by more than 2^4) and not below 2^-24 f16 has nothing to add.
//
// A CTA per SM works on 256 query rows (heads that share a key head, and tokens, side by
// side) as two tiles of 128: while the softmax of one tile runs, the products of the other
// keep the tensor cores busy, and both read the same K and V from shared memory. Work is counted in
// stages of 128 keys over all items (request, key head, 256 rows) and dealt out evenly;
// an item in several CTAs leaves partial sums that a second kernel joins in order.
//   warps 0-7, 8-15: softmax and epilogue of tiles 0 and 1, two threads to a row (= TMEM lane), one for
//              each half of a stage's keys (and of the columns of Q and O); the two exchange their
//              largest score. At an item's start they also split its queries into shared memory.
//   warps 16-19: widen V, zeros past a request's last token (what lies there may be anything).
//   warp 20: producer: items, look-ups of lists and tables (32 at a time, a batch ahead),
//              K by TMA boxes of 64 keys, V by bulk copies.
//   warp 21: issues S of both tiles (A = q1, q2, B = K, K-major, from shared memory).
//   warp 22: issues O += P V (A = P in TMEM, written over the S it is made of, B = V MN-major).
// TMEM (512 columns): S and then P of the tiles [0, 256) (P of a half stage over the scores it is
// made of), O [256, 512).
// Every mbarrier wait is bounded (2 s); on expiry the CTA sets SPARSP_ERR_TIMEOUT, all roles
// leave their loops, copies and MMAs in flight are drained with a second bounded wait, and
// TMEM is released.
#include <cuda_fp16.h>

#include "cache_items.cuh"
#include "rows.cuh"

namespace sparsp {
namespace {

using namespace tc;

constexpr int kTileRows = 128, kItemRows = 2 * kTileRows, kStageKeys = 128;
constexpr int kItemCost = 6;       // stages that an item's own work counts as
constexpr int kMinStages = 10;     // stages, an item's own among them, that are worth a CTA
constexpr float kShift = 11.f, kMoves = 4.f;   // P is held as 2^11 times what it is against R
constexpr int kNK = 3, kNV = 2, kNW = 2, kNInfo = 8, kNItems = 2;
constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 200000000ull;

constexpr int kSoftmax = 16, W_WIDEN = kSoftmax, W_PROD = W_WIDEN + 4, W_S = W_PROD + 1, W_PV = W_PROD + 2;   // warps

enum Bars {
  K_FULL, K_EMPTY = K_FULL + kNK, V_FULL = K_EMPTY + kNK, V_EMPTY = V_FULL + kNV, W_FULL = V_EMPTY + kNV,
  W_EMPTY = W_FULL + kNW, INFO = W_EMPTY + kNW, I_FULL = INFO + kNInfo, I_EMPTY = I_FULL + kNItems,
  Q_FULL = I_EMPTY + kNItems, S_FULL = Q_FULL + 2, P_FULL = S_FULL + 2, PV_DONE = P_FULL + 2, O_EMPTY = PV_DONE + 2,
  TEAR = O_EMPTY + 2, TEAR_PV, NBAR
};

// A piece of an item: stages [e0, e1) of it. e1 < 0: no more.
struct Piece {
  int s0, hk, row0, rows, n, len, e0, e1, part;   // part: -1: the whole item, else the slot of its sums
};
// A stage's two halves of 64 keys: position of the first key, how many exist, scale of K, log2
// and inverse of the scale of V.
struct Info {
  int pos[2], valid[2];
  float ks[2], lv[2], inv[2];
};

template <int D>
struct Cfg {
  static constexpr int THREADS = 768;
  static constexpr uint32_t kRegSoftmax = 88, kRegAux = 64;
  static_assert(512 * kRegSoftmax + 256 * kRegAux == THREADS * 80, "register split of the six warpgroups");
  static constexpr uint32_t kQ = kTileRows * D, kK = kStageKeys * D, kV = kStageKeys * D;      // bytes: q1 or q2, K, V
  static constexpr uint32_t kW = kStageKeys * D * 2, kWBox = kStageKeys * 128;                 // V in f16, 64 columns of it
  static constexpr uint32_t kOffK = 4 * kQ, kOffV = kOffK + kNK * kK, kOffW = kOffV + kNV * kV;
  static constexpr uint32_t kOffBar = kOffW + kNW * kW, kOffInfo = kOffBar + 8 * NBAR;
  static constexpr uint32_t kOffPiece = kOffInfo + kNInfo * (uint32_t)sizeof(Info);
  static constexpr uint32_t kOffEx = kOffPiece + kNItems * (uint32_t)sizeof(Piece);   // [2][tile][half][row] floats
  static constexpr uint32_t kOffMisc = kOffEx + 2 * 2 * 2 * kTileRows * 4;
  static constexpr uint32_t kSmem = kOffMisc + 64 + 1024;   // + alignment slack
  static_assert(kSmem <= 232448, "shared memory");
  // K-major rows of D bytes: 128-byte swizzle, or with D = 64 the 64-byte one
  static constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : 4u, kAtom = 8 * D;
  // the 16-byte vector c of row r
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (uint32_t)(r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
  }
};

// Instruction descriptors: f32 += e4m3 e4m3, both K-major; f32 += f16 f16, B MN-major.
__host__ __device__ constexpr uint32_t idesc(int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_8bit(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

__device__ __forceinline__ bool wait_raw(uint32_t bar, uint32_t parity, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit) return false;
  return true;
}

// 32 columns of this thread's TMEM lane, and their maximum (sm_103 load with reduction).
__device__ __forceinline__ float tmem_ld32_max(uint32_t taddr, uint32_t* r) {
  float m;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
      : "r"(taddr));
  return m;
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {   // lo in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Items of the whole call, for this kernel: entries are requests, or with lists request
// and key head; an entry's items are its key heads' row groups.
struct Walk {
  const CacheAttn& a;
  __device__ __forceinline__ int stages(const Entry& x, int group) const {
    if (a.row_ptr != nullptr) return (x.units + 1) / 2;
    int keys = x.len;
    if (a.causal) {   // up to the last row's token
      const int tok = min(x.n, ((group + 1) * kItemRows - 1) / a.group + 1) - 1;
      keys = max(0, min(keys, x.len - x.n + tok + 1));
    }
    return (keys + kStageKeys - 1) / kStageKeys;
  }
  // of one item; an item without keys still has its rows to write: one stage, empty
  __device__ __forceinline__ int size(const Entry& x, int group) const { return kItemCost + max(1, stages(x, group)); }
  __device__ __forceinline__ int64_t head_weight(const Entry& x, int groups) const {
    int64_t w = 0;
    if (!a.causal || a.row_ptr != nullptr) return (int64_t)groups * (groups > 0 ? size(x, 0) : 0);
    for (int i = 0; i < groups; ++i) w += size(x, i);
    return w;
  }
  __device__ __forceinline__ Entry at(int e, bool tell) const {
    Entry x = entry_at(a, e, tell);
    if ((int64_t)x.n * a.group <= a.few) x.n = 0;   // the other kernel's
    x.groups = (int)(((int64_t)x.n * a.group + kItemRows - 1) / kItemRows);
    x.per_head = head_weight(x, x.groups);
    x.weight = x.per_head * (a.row_ptr != nullptr ? 1 : a.c.heads);
    return x;
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
attn_cache_tc_kernel(const __grid_constant__ CUtensorMap tk, const CacheAttn a, const Parts parts) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base, sK = base + C::kOffK, sV = base + C::kOffV, sW = base + C::kOffW;
  auto bar = [&](int i) -> uint32_t { return base + C::kOffBar + 8u * (uint32_t)i; };
  Info* infos = reinterpret_cast<Info*>(gbase + C::kOffInfo);
  Piece* pieces = reinterpret_cast<Piece*>(gbase + C::kOffPiece);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(gbase + C::kOffMisc + 4);
  int64_t* s_begin = reinterpret_cast<int64_t*>(gbase + C::kOffMisc + 16);   // first entry, its offset
  __shared__ int64_t s_scan[C::THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // ---- this CTA's range of stages
  const Walk walk{a};
  const int entries = entries_of(a), per = (entries + C::THREADS - 1) / C::THREADS;
  const int n0 = min(entries, (int)threadIdx.x * per), n1 = min(entries, n0 + per);
  int64_t mine = 0;
  for (int e = n0; e < n1; ++e) mine += walk.at(e, blockIdx.x == 0).weight;
  int64_t total, below = scan_below<C::THREADS / 32>(mine, s_scan, &total);
  const int64_t ctas = min((int64_t)gridDim.x, max((int64_t)1, (total + kMinStages - 1) / kMinStages)), cta = blockIdx.x;
  const int64_t begin = cta * total / ctas, end = cta < ctas ? (cta + 1) * total / ctas : begin;
  if (threadIdx.x == 0) parts.open[cta].last = -1;
  if (cta >= ctas || begin >= end) return;      // the same for the whole CTA
  if (below <= begin && begin < below + mine) {
    int64_t at = below;
    int e = n0;
    for (;; ++e) {
      const int64_t w = walk.at(e, false).weight;
      if (begin < at + w) break;
      at += w;
    }
    s_begin[0] = e;
    s_begin[1] = begin - at;
  }
  if (threadIdx.x == 0) {
    auto init = [&](int i, int n, int count) {
      for (int k = 0; k < n; ++k) mbar_init(bar(i + k), count);
    };
    init(K_FULL, kNK, 1);
    init(K_EMPTY, kNK, 1);
    init(V_FULL, kNV, 1);
    init(V_EMPTY, kNV, 4);
    init(W_FULL, kNW, 4);
    init(W_EMPTY, kNW, 1);
    init(INFO, kNInfo, 1);
    init(I_FULL, kNItems, 1);
    init(I_EMPTY, kNItems, kSoftmax + 6);   // softmax, widening and issuing warps
    init(Q_FULL, 2, 8);
    init(S_FULL, 2, 1);
    init(P_FULL, 2, 8);
    init(PV_DONE, 2, 1);
    init(O_EMPTY, 2, 8);
    init(TEAR, 2, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_PROD && lane == 0) prefetch_tmap(&tk);
  if (warp == W_S) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, a.d_status, kWaitNs};
  auto col_s = [&](int t) { return tmem + (uint32_t)t * 128u; };
  auto col_o = [&](int t) { return tmem + 256u + (uint32_t)t * 128u; };
  // The next piece from the ring; false at the end or on abort. The slot is given back at once.
  uint32_t it_use = 0;
  auto next_piece = [&](Piece& x) -> bool {
    const int ri = (int)(it_use % kNItems);
    if (!wait_warp(bar(I_FULL + ri), (it_use / kNItems) & 1u, g)) return false;
    x = pieces[ri];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(I_EMPTY + ri));
    ++it_use;
    return x.e1 >= 0;
  };
  auto tiles_of = [&](const Piece& x) { return x.rows > kTileRows ? 2 : 1; };

  if (warp >= kSoftmax) {
    regs_decrease<C::kRegAux>();
    if (warp == W_PROD) {
      // ------------------------------------------------------------ producer
      uint32_t it_fill = 0, k_fill = 0, v_fill = 0, n_info = 0;
      int entry = (int)s_begin[0];
      int64_t offset = s_begin[1], unit_at = begin;
      Entry x = walk.at(entry, false);
      bool ok = true;
      auto publish = [&](const Piece& p) -> bool {
        const int ri = (int)(it_fill % kNItems);
        if (!wait_warp(bar(I_EMPTY + ri), ((it_fill / kNItems) & 1u) ^ 1u, g)) return false;
        if (lane == 0) {
          pieces[ri] = p;
          mbar_arrive(bar(I_FULL + ri));
        }
        __syncwarp();
        ++it_fill;
        return true;
      };
      const int per_block = a.c.bt / kUnit;
      while (ok && unit_at < end) {
        while (offset >= x.weight) {            // entries without queries weigh nothing
          offset -= x.weight;
          x = walk.at(++entry, false);
        }
        // the item at this offset (its first kItemCost stages stand for its own work)
        int hk = x.hk;
        int64_t within = offset;
        if (a.row_ptr == nullptr) {
          hk = (int)(offset / x.per_head);
          within -= hk * x.per_head;
        }
        int group = 0, size = walk.size(x, 0);
        if (!a.causal || a.row_ptr != nullptr) {   // items of one size
          group = (int)(within / size);
          within -= (int64_t)group * size;
        } else {
          while (within >= size) {
            within -= size;
            size = walk.size(x, ++group);
          }
        }
        const int at0 = (int)within, at1 = (int)min((int64_t)size, at0 + (end - unit_at));
        const int64_t item_at = unit_at - at0;
        const int e0 = max(0, at0 - kItemCost), e1 = at1 - kItemCost;
        unit_at += at1 - at0;
        offset += at1 - at0;
        if (e1 <= e0) continue;
        const int row0 = group * kItemRows, rows = min(kItemRows, x.n * a.group - row0);
        const bool whole = e0 == 0 && at1 == size;
        const int slot = 2 * (int)cta + (e0 > 0 ? 0 : 1);     // a piece that goes on is the CTA's first
        if (!whole && e0 == 0 && lane == 0)
          parts.open[cta] = Open{x.b, hk, row0, rows, x.s0, (int)(((item_at + size) * ctas - 1) / total)};
        if (!(ok = publish(Piece{x.s0, hk, row0, rows, x.n, x.len, e0, e1, whole ? -1 : slot}))) break;

        // look-ups: lane i takes the half stage (64 keys) u0 + i of a batch of 32
        const int32_t* table = a.table + (int64_t)x.b * a.max_blocks;
        const int32_t* list = a.row_ptr != nullptr ? a.col_idx + a.row_ptr[entry] : nullptr;
        struct Half {
          int pos, valid, page;
          float ks, vs;
        };
        auto look = [&](int u) -> Half {
          Half h{0, 0, 0, 1.f, 1.f};
          if (u >= 2 * e1 || u >= x.units) return h;
          int j = u / per_block;
          if (list != nullptr) j = __ldg(list + j);
          if (j < 0 || (int64_t)j * a.c.bt >= x.len) {
            report(a.d_status, SPARSP_ERR_DATA);
            return h;
          }
          const int page = __ldg(table + j);
          if (page < 0 || page >= a.c.blocks) {
            report(a.d_status, SPARSP_ERR_DATA);
            return h;
          }
          const int64_t block = (int64_t)page * a.c.heads + hk;
          h.pos = j * a.c.bt + u % per_block * kUnit;
          h.valid = max(0, min(kUnit, x.len - h.pos));
          h.page = page;
          h.ks = __ldg(a.ks + block);
          h.vs = fmaxf(__ldg(a.vs + block), 0x1p-120f);
          return h;
        };
        Half now, ahead = look(2 * e0 + lane);
        for (int e = e0; e < e1; ++e) {
          const int i = 2 * (e - e0) & 31;      // this stage's halves: lanes i, i + 1
          if (i == 0) {
            now = ahead;
            ahead = look(2 * e + 32 + lane);
          }
          // the stage's facts
          const uint32_t is = n_info % kNInfo;
          const float lv = log2f(now.vs), inv = 1.0f / now.vs;
          if (lane == i || lane == i + 1) {
            Info& f = infos[is];
            const int h = lane - i;
            f.pos[h] = now.pos;
            f.valid[h] = now.valid;
            f.ks[h] = now.ks;
            f.lv[h] = lv;
            f.inv[h] = inv;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(INFO + is));
          ++n_info;
          const int v0 = __shfl_sync(0xffffffffu, now.valid, i), v1 = __shfl_sync(0xffffffffu, now.valid, i + 1);
          const int p0 = __shfl_sync(0xffffffffu, now.page, i), p1 = __shfl_sync(0xffffffffu, now.page, i + 1);
          const int q0 = __shfl_sync(0xffffffffu, now.pos, i) % a.c.bt, q1 = __shfl_sync(0xffffffffu, now.pos, i + 1) % a.c.bt;
          const uint32_t bytes = ((v0 > 0 ? 1u : 0u) + (v1 > 0 ? 1u : 0u)) * (uint32_t)(kUnit * D);
          const uint32_t ks = k_fill % kNK, vs = v_fill % kNV;
          if (!(ok = wait_warp(bar(K_EMPTY + ks), ((k_fill / kNK) & 1u) ^ 1u, g))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(K_FULL + ks), bytes);
            if (v0 > 0) tma_load_3d(sK + ks * C::kK, &tk, bar(K_FULL + ks), 0, hk * a.c.bt + q0, p0);
            if (v1 > 0) tma_load_3d(sK + ks * C::kK + kUnit * D, &tk, bar(K_FULL + ks), 0, hk * a.c.bt + q1, p1);
          }
          __syncwarp();
          ++k_fill;
          if (!(ok = wait_warp(bar(V_EMPTY + vs), ((v_fill / kNV) & 1u) ^ 1u, g))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(V_FULL + vs), bytes);
            const uint8_t* from = a.vc + (int64_t)hk * a.c.bt * D;
            const int64_t page = (int64_t)a.c.heads * a.c.bt * D;
            if (v0 > 0) bulk_load(sV + vs * C::kV, from + p0 * page + q0 * D, kUnit * D, bar(V_FULL + vs));
            if (v1 > 0) bulk_load(sV + vs * C::kV + kUnit * D, from + p1 * page + q1 * D, kUnit * D, bar(V_FULL + vs));
          }
          __syncwarp();
          ++v_fill;
        }
      }
      if (ok) publish(Piece{0, 0, 0, 0, 0, 0, 0, -1, 0});
      if (*abort_flag) {
        // copies in flight end before the CTA does
        for (uint32_t i = 0; i < kNK; ++i)
          if (k_fill > i) wait_raw(bar(K_FULL + (k_fill - 1 - i) % kNK), ((k_fill - 1 - i) / kNK) & 1u, kDrainNs);
        for (uint32_t i = 0; i < kNV; ++i)
          if (v_fill > i) wait_raw(bar(V_FULL + (v_fill - 1 - i) % kNV), ((v_fill - 1 - i) / kNV) & 1u, kDrainNs);
      }
      __syncwarp();
    } else if (warp == W_S) {
      // ------------------------------------------------------------ S = Q K^T issuer
      uint32_t k_use = 0, n_q[2] = {0, 0}, n_s[2] = {0, 0};
      bool issued = false, ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        const int tiles = tiles_of(x);
        for (int t = 0; t < tiles && ok; ++t) ok = wait_warp(bar(Q_FULL + t), n_q[t]++ & 1u, g);
        for (int e = x.e0; e < x.e1 && ok; ++e) {
          const uint32_t ks = k_use % kNK;
          if (!(ok = wait_warp(bar(K_FULL + ks), (k_use / kNK) & 1u, g))) break;
          for (int t = 0; t < tiles; ++t) {
            // the buffer held P until its PV was done
            if (!(ok = wait_warp(bar(PV_DONE + t), (n_s[t] & 1u) ^ 1u, g))) break;
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_8bit(col_s(t), smem_desc(sQ + (uint32_t)(2 * t + q) * C::kQ + 32u * kk, 16, C::kAtom, C::kSwz),
                           smem_desc(sK + ks * C::kK + 32u * kk, 16, C::kAtom, C::kSwz), idesc(kStageKeys, 0),
                           q > 0 || kk > 0 ? 1u : 0u);
              commit(bar(S_FULL + t));
              if (t + 1 == tiles) commit(bar(K_EMPTY + ks));
            }
            __syncwarp();
            ++n_s[t];
            issued = true;
          }
          ++k_use;
        }
      }
      if (*abort_flag && issued) {
        if (elect_one()) commit(bar(TEAR));
        __syncwarp();
        wait_raw(bar(TEAR), 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp == W_PV) {
      // ------------------------------------------------------------ O += P V issuer
      uint32_t w_use = 0, n_p[2] = {0, 0}, n_o[2] = {0, 0};
      bool issued = false, ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        const int tiles = tiles_of(x);
        for (int e = x.e0; e < x.e1 && ok; ++e) {
          const uint32_t ws = w_use % kNW;
          if (!(ok = wait_warp(bar(W_FULL + ws), (w_use / kNW) & 1u, g))) break;
          for (int t = 0; t < tiles; ++t) {
            if (!(ok = wait_warp(bar(P_FULL + t), n_p[t] & 1u, g))) break;
            if (e == x.e0 && !(ok = wait_warp(bar(O_EMPTY + t), (n_o[t]++ & 1u) ^ 1u, g))) break;
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kStageKeys / 16; ++kk)
                mma_ts(col_o(t), col_s(t) + 64u * (kk >> 2) + 8u * (kk & 3), smem_desc(sW + ws * C::kW + 2048u * kk, C::kWBox, 1024, kSwizzle128B),
                       idesc(D, 1), e > x.e0 || kk > 0 ? 1u : 0u);
              commit(bar(PV_DONE + t));
              if (t + 1 == tiles) commit(bar(W_EMPTY + ws));
            }
            __syncwarp();
            ++n_p[t];
            issued = true;
          }
          ++w_use;
        }
      }
      if (*abort_flag && issued) {
        if (elect_one()) commit(bar(TEAR_PV));
        __syncwarp();
        wait_raw(bar(TEAR_PV), 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp < W_PROD) {
      // ------------------------------------------------------------ V to f16
      constexpr int CH = D / 16;                // 16-code vectors of a row
      const int id = threadIdx.x - 32 * W_WIDEN;
      uint32_t n = 0;
      bool ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        for (int e = x.e0; e < x.e1; ++e) {
          const uint32_t vs = n % kNV, ws = n % kNW, is = n % kNInfo;
          if (!(ok = wait_warp(bar(INFO + is), (n / kNInfo) & 1u, g))) break;
          const int valid0 = infos[is].valid[0], valid1 = infos[is].valid[1];
          if (!(ok = wait_warp(bar(V_FULL + vs), (n / kNV) & 1u, g))) break;
          if (!(ok = wait_warp(bar(W_EMPTY + ws), ((n / kNW) & 1u) ^ 1u, g))) break;
          const uint4* from = reinterpret_cast<const uint4*>(gbase + C::kOffV + vs * C::kV);
          uint8_t* to = gbase + C::kOffW + ws * C::kW;
#pragma unroll
          for (int i = 0; i < kStageKeys * CH / 128; ++i) {
            const int v = id + 128 * i, r = v / CH, c = v % CH;   // row, and its columns 16 c ..
            uint4 w = from[v];
            if ((r & 63) >= (r < 64 ? valid0 : valid1)) w = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              out[2 * k] = f16x2_of_e4m3(in[k]);
              out[2 * k + 1] = f16x2_of_e4m3(in[k] >> 16);
            }
            // two vectors of 8 columns; the other one first in the second box, for the banks' sake
            uint8_t* row = to + (c >> 2) * C::kWBox + r * 128;
            const int c0 = 2 * (c & 3), swap = (c >> 2) & 1;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int h = k ^ swap;
              *reinterpret_cast<uint4*>(row + (((c0 + h) ^ (r & 7)) << 4)) =
                  h ? make_uint4(out[4], out[5], out[6], out[7]) : make_uint4(out[0], out[1], out[2], out[3]);
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(V_EMPTY + vs));
            mbar_arrive(bar(W_FULL + ws));
          }
          ++n;
        }
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::kRegSoftmax>();
    // -------------------------------------------------------------- softmax + epilogue of tile t
    const int t = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;   // r: row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = col_s(t) + lanes + 64u * half, t_o = col_o(t) + lanes + (uint32_t)half * (D / 2);
    const int pair_bar = 1 + t * 4 + (warp & 3);   // named barrier of the two warps that share rows
    float* ex = reinterpret_cast<float*>(gbase + C::kOffEx) + t * 2 * kTileRows + r;
    uint32_t n_info = 0, n_s = 0, n_ex = 0;
    bool ok = true;
    // The row's other half: gives its value for this one's. The two warps take every step together: a
    // warp that has given up says so here (NaN with these bits), and both leave after it.
    constexpr uint32_t kGone = 0x7fc0dead;
    auto exchange = [&](float mine, float& theirs) -> bool {
      float* at = ex + (n_ex++ & 1u) * 4 * kTileRows;   // the other buffer may still be read
      at[half * kTileRows] = ok ? mine : __uint_as_float(kGone);
      asm volatile("bar.sync %0, 64;\n" ::"r"(pair_bar) : "memory");
      theirs = at[(half ^ 1) * kTileRows];
      ok = ok && !__any_sync(0xffffffffu, __float_as_uint(theirs) == kGone);
      return ok;
    };
    Piece x;
    for (;;) {
      float theirs;
      ok = ok && next_piece(x);
      if (!exchange(0.f, theirs)) break;
      if (t >= tiles_of(x)) {
        n_info += (uint32_t)(x.e1 - x.e0);
        continue;
      }
      const int row = x.row0 + t * kTileRows + r;
      const bool live = t * kTileRows + r < x.rows;
      const int tok = row / a.group, h = x.hk * a.group + row % a.group;
      // ---- the row's queries as two e4m3 values each, under a power of two (every S of the last
      // piece is done: its scores have been read)
      float factor = 0.f;
      {
        const __nv_bfloat16* from = a.q + (int64_t)(x.s0 + tok) * a.q_token + (int64_t)h * D + half * (D / 2);
        uint4 w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          w[c] = live ? __ldg(reinterpret_cast<const uint4*>(from) + c) : make_uint4(0, 0, 0, 0);
        uint32_t most = 0;                       // of the finite ones, as bf16 bits
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t p[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = p[i] & 0x7fffu, hi = (p[i] >> 16) & 0x7fffu;
            if (lo < 0x7f80u) most = max(most, lo);
            if (hi < 0x7f80u) most = max(most, hi);
          }
        }
        exchange(__uint_as_float(most), theirs);
        most = max(most, __float_as_uint(theirs));
        // 224 < most * 2^-e <= 448
        int e2 = (int)(most >> 7) - 127 - 8 + ((most & 0x7fu) > 0x60u ? 1 : 0);
        e2 = max(-100, min(120, e2));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        factor = __uint_as_float((uint32_t)(127 + e2) << 23) * a.scale_log2;
        uint8_t* q1 = gbase + (uint32_t)(2 * t) * C::kQ;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint32_t p[8] = {w[2 * c].x,     w[2 * c].y,     w[2 * c].z,     w[2 * c].w,
                                 w[2 * c + 1].x, w[2 * c + 1].y, w[2 * c + 1].z, w[2 * c + 1].w};
          uint32_t hi4[4], lo4[4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float f0 = __uint_as_float(p[i] << 16), f1 = __uint_as_float(p[i] & 0xffff0000u);
            f0 = fabsf(f0) < INFINITY ? f0 * down : NAN;   // what is not finite is NaN to the scores
            f1 = fabsf(f1) < INFINITY ? f1 * down : NAN;
            const uint32_t big = e4m3_pair(f0, f1), back = f16x2_of_e4m3(big);
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
            const uint32_t small = e4m3_pair(f0 - b.x, f1 - b.y);
            if (i & 1) {
              hi4[i / 2] |= big << 16;
              lo4[i / 2] |= small << 16;
            } else {
              hi4[i / 2] = big;
              lo4[i / 2] = small;
            }
          }
          const uint32_t to = C::at(r, half * (D / 32) + c);
          *reinterpret_cast<uint4*>(q1 + to) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(q1 + C::kQ + to) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Q_FULL + t));
      }
      const int last = a.causal ? x.len - x.n + tok : INT32_MAX;   // the last key that the row sees
      float ref = -INFINITY, l = 0.f;            // R; l times 2^11, of this half's keys
      for (int e = x.e0; e < x.e1; ++e) {
        const uint32_t is = n_info % kNInfo;
        ok = ok && wait_warp(bar(INFO + is), (n_info / kNInfo) & 1u, g);
        ++n_info;
        const int pos = infos[is].pos[half];
        const int see = min(infos[is].valid[half], last - pos < 63 ? last - pos + 1 : 64);
        const float c = factor * infos[is].ks[half], lv = infos[is].lv[half], inv = infos[is].inv[half];
        const bool cut = __any_sync(0xffffffffu, see < 64);
        ok = ok && wait_warp(bar(S_FULL + t), n_s & 1u, g);
        ++n_s;
        fence_after();
        // the scores are read twice, for their maximum and for P: registers hold 32 of them at a time
        uint32_t s[32];
        float cm;
        if (!cut) {
          cm = tmem_ld32_max(t_s, s);
          cm = fmaxf(cm, tmem_ld32_max(t_s + 32u, s));
          wait_ld();
        } else {
          cm = -INFINITY;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            tmem_ld32(t_s + 32u * q, s);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) cm = 32 * q + k < see ? fmaxf(cm, __uint_as_float(s[k])) : cm;
          }
        }
        // a half without keys says nothing (its product with a scale might)
        float top = see > 0 ? fmaf(cm, c, lv) : -INFINITY;
        if (!exchange(top, theirs)) break;
        top = fmaxf(top, theirs);
        float f = 1.f;
        const bool moves = top > ref + kMoves;   // by itself: not by what other rows hold
        if (moves) {
          f = exp2_fast(ref - top);              // 0 for the first
          ref = top;
          l *= f;
        }
        const float off = lv + kShift - (ref == -INFINITY ? 0.f : ref);
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_ld32(t_s + 32u * q, s);
          wait_ld();
          if (cut) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * q + k >= see) s[k] = 0xff800000u;
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            fma_x2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]), c, off, x0, x1);
            const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
            add_x2(rs[2 * (i & 1)], rs[2 * (i & 1) + 1], p0, p1);
            pk[i] = pack_f16(p0, p1);
          }
          tmem_st16(t_s + 16u * q, pk);          // over scores of this half that have been read
        }
        l = fmaf((rs[0] + rs[1]) + (rs[2] + rs[3]), inv, l);
        // O follows the reference now that the scores are no longer held
        if (e > x.e0 && __any_sync(0xffffffffu, moves)) {   // PV of the last stage is done: S came after it
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t ov[32];
            tmem_ld32(t_o + 32u * i, ov);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
            tmem_st32(t_o + 32u * i, ov);
          }
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P_FULL + t));
      }
      // ---- the end of a piece: the row's whole sum, and half of O from TMEM
      ok = ok && wait_warp(bar(PV_DONE + t), (n_s - 1) & 1u, g);
      if (!exchange(l, theirs)) break;
      l = half ? theirs + l : l + theirs;
      fence_after();
      const float scale = l == 0.f ? 0.f : x.part < 0 ? 1.0f / l : 1.f;
      const int64_t at = (int64_t)(x.s0 + tok) * a.H + h;
      float* sums = parts.sum + ((int64_t)max(x.part, 0) * kItemRows + t * kTileRows + r) * D + half * (D / 2);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t ov[32];
        tmem_ld32(t_o + 32u * i, ov);
        wait_ld();
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) ov[k] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(ov[k]) * scale);
        if (x.part < 0) {
          uint4* to = reinterpret_cast<uint4*>(a.o + at * D + half * (D / 2) + 32 * i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __nv_bfloat162 v =
                  __floats2bfloat162_rn(__uint_as_float(ov[8 * k + 2 * q]), __uint_as_float(ov[8 * k + 2 * q + 1]));
              w[q] = *reinterpret_cast<const uint32_t*>(&v);
            }
            to[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(sums + 32 * i + 4 * k) = make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(O_EMPTY + t));
      if (live && half == 0) {
        if (x.part < 0) a.lse[at] = l == 0.f ? -INFINITY : (ref - kShift + log2f(l)) * 0.6931471805599453f;
        else parts.ml[(int64_t)x.part * kItemRows + t * kTileRows + r] = make_float2(ref - kShift, l);
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == W_S) tmem_dealloc(tmem, 512);
}

// The join of what items in several CTAs have left: CTA (c, rows of the item that starts in CTA c),
// a warp per row, the parts in order.
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(256)
attn_cache_tc_join_kernel(const CacheAttn a, const Parts parts) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const Open it = parts.open[blockIdx.x];
  if (it.last < 0) return;
  const int lane = threadIdx.x & 31, count = it.last - (int)blockIdx.x + 1;
  auto row_of = [&](int i, int r) { return (int64_t)(2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0)) * kItemRows + r; };
  for (int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5); r < min(it.rows, ((int)blockIdx.y + 1) * kJoinRows); r += 8) {
    float top = -INFINITY;
    for (int i = lane; i < count; i += 32) top = fmaxf(top, parts.ml[row_of(i, r)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.f;
    float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float2 ml = parts.ml[row_of(i, r)];
      const float f = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : exp2_fast(ml.x - top);
      sum = fmaf(f, ml.y, sum);
      if (4 * lane < D) {
        const float4 w = *reinterpret_cast<const float4*>(parts.sum + row_of(i, r) * D + 4 * lane);
        all.x = fmaf(f, w.x, all.x);
        all.y = fmaf(f, w.y, all.y);
        all.z = fmaf(f, w.z, all.z);
        all.w = fmaf(f, w.w, all.w);
      }
    }
    if (4 * lane < D) finish<D>(a, it.s0, it.hk, it.row0 + r, 4 * lane, top, sum, all);
  }
}

constexpr int kGrid = 152;

template <int D>
sparsp_status_t go(const CacheAttn& a, void* ws, cudaStream_t st) {
  CUtensorMap tk;
  if (!make_tmap_codes(&tk, a.kc, (uint64_t)D, (uint64_t)a.c.heads * a.c.bt, (uint64_t)a.c.blocks, kUnit))
    return SPARSP_ERR_CUDA;
  const Parts p = parts_of(ws, kGrid, kItemRows);
  constexpr int smem = Cfg<D>::kSmem;
  if (cudaFuncSetAttribute(attn_cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  attn_cache_tc_kernel<D><<<kGrid, Cfg<D>::THREADS, smem, st>>>(tk, a, p);
  SPARSP_LAUNCH_CHECK();
  return launch_after(attn_cache_tc_join_kernel<D>, dim3(kGrid, kItemRows / kJoinRows), 256, st, a, p);
}

}  // namespace

size_t attn_cache_tc_ws(const CacheDims& c) { return parts_bytes(kGrid, kItemRows, c.d); }

sparsp_status_t launch_attn_cache_tc(const CacheAttn& a, void* ws, cudaStream_t st) {
  return a.c.d == 64 ? go<64>(a, ws, st) : go<128>(a, ws, st);
}

}  // namespace sparsp
