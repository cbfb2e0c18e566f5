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
// The scale of a block's values goes into the exponent (cache_items.cuh); P is at most 2^15 (its reference follows when
// it is passed by more than 2^4) and below 2^-24 f16 has nothing to add.
//
// Measured: 1,536 queries x 30,720 keys x 40 heads of d = 128 take 650 us when they come alone (0.79 of the bf16
// peak for the two products, 0.73 back to back under the power cap), d = 64 543 us, 4 prompts of 4,096 tokens x 32
// heads 452 us (captured calls, 8 us each the replay's own). Counted in cycles, a stage of 128 keys is 1,570 (d = 64:
// 1,290) where its products take 1,090
// (545): a row's thread spends 3,140 on each second stage, 950 of them on 128 exponentials and their sum, 200 on
// handing P over, 300 each on reading what it has to know of the keys and on waiting for the other thread's
// reference, 470 on waiting for S (d = 64: 230). No pipe is full (tensor 0.70, exponentials 0.33); what bounds it
// is the round S - exponentials - P V, of which three fit tensor memory. What it gained from: pairs of SMs (846 ->
// 725), a look-up for 16 stages at a time instead of every stage (718 -> 661), P in S's place (661 -> 651).
//
// Two SMs work on 256 query rows (heads that share a key head, and tokens, side by side) as one
// cluster of two CTAs with paired products (cta_group::2): each has 128 of the rows in its tensor memory, and
// each loads one half of K's keys and of V's columns, so that every byte of the cache is loaded and widened once
// for 256 rows, and shared memory is read half as often as with a tile to each SM. Work is counted in
// stages of 128 keys over all items (request, key head, 256 rows) and dealt out evenly;
// an item in several clusters leaves partial results that a second kernel joins in order.
//   warps 0-7: softmax and epilogue of the CTA's rows, two threads to a row (= TMEM lane): one for the even
//              stages and one for the odd, which pass the row's reference from stage to stage, so that one loads
//              scores while the other takes exponentials. Each has half of the columns of Q, which they
//              split into shared memory at an item's start, and of O.
//   warps 8-11: widen V, zeros past a request's last token (what lies there may be anything).
//   warp 12: producer: items, look-ups of lists and tables (32 at a time, a batch ahead), and TMA: 64 keys
//              of K, half of the columns of V.
//   warp 13, first CTA: issues S of both (A = q1, q2, B = K, K-major, from shared memory).
//   warp 14, first CTA: issues O += P V (A = P in TMEM, B = V MN-major).
// TMEM (512 columns): S of three stages, and in its place P, [0, 384), O [384, 384 + d).
// The first CTA's barriers count what its products wait for in both CTAs (remote arrivals); its commits
// reach both. A remote arrival and its wait order no memory between the CTAs, and need not: what it stands for is read by
// the tensor cores alone, each CTA's own shared and tensor memory, where the writer's fences before the arrival have put
// it (fence.proxy.async; tcgen05.wait and tcgen05.fence::before_thread_sync). With a release at cluster scope a stage takes
// thousands of cycles more. Every mbarrier wait is bounded (2 s); on expiry the CTA sets SPARSP_ERR_TIMEOUT, all roles
// leave their loops, copies and MMAs in flight are drained with a second bounded wait, and
// TMEM is released when both CTAs are done.
#include "cache_items.cuh"
#include "rows.cuh"

namespace sparsp {
namespace {

using namespace tc;

constexpr int kTileRows = 128, kItemRows = 2 * kTileRows, kStageKeys = 128;
constexpr int kItemCost = 6;       // stages that an item's own work (queries, epilogue, join) counts as: 9,000 cycles
constexpr int kMinStages = 10;     // stages, an item's own among them, that are worth a cluster
constexpr float kShift = 11.f, kMoves = 4.f;   // P is held as 2^11 times what it is against R
constexpr int kNK = 6, kNV = 4, kNW = 3, kNItems = 2, kNS = 3;
// Batches of facts in the ring. Nobody hands one back: K's ring lets the producer run at most ten stages ahead of
// any reader, and kNItems keeps those in three pieces, so that no more than five batches are in use.
constexpr int kNInfo = 8;
constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 200000000ull;
constexpr int kSoftmax = 8, W_WIDEN = kSoftmax, W_PROD = W_WIDEN + 4, W_S = W_PROD + 1, W_PV = W_PROD + 2;   // warps

// First CTA: K_FULL, W_FULL, Q_FULL, P_FULL and O_EMPTY count both CTAs.
enum Bars {
  K_FULL, K_EMPTY = K_FULL + kNK, V_FULL = K_EMPTY + kNK, V_EMPTY = V_FULL + kNV, W_FULL = V_EMPTY + kNV,
  W_EMPTY = W_FULL + kNW, INFO = W_EMPTY + kNW, I_FULL = INFO + kNInfo, I_EMPTY = I_FULL + kNItems,
  Q_FULL = I_EMPTY + kNItems, S_FULL, P_FULL = S_FULL + kNS, PV_DONE = P_FULL + kNS, O_EMPTY = PV_DONE + kNS,
  TEAR, TEAR_PV, NBAR
};

// A piece of an item: stages [e0, e1) of it. e1 < 0: no more.
struct Piece {
  int s0, hk, row0, rows, n, len, e0, e1, part;   // part: -1: the whole item, else the slot of its sums
};
// What is to be known of half a stage (64 keys): position of the first, how many exist, scale of K, log2 and inverse of
// vs / u, log2 of how much u has risen since the stage before, of u, and how many keys have values beside u. The
// producer leaves them by batches of 16 stages of a piece, of one u.
struct alignas(16) Info {
  int pos, valid;
  float ks, lv, inv, rise, lu;
  int held;
};
constexpr int kBatch = 16;
struct Batch {
  Info half[kBatch][2];
};

template <int D>
struct Cfg {
  static constexpr int THREADS = 512;
  static constexpr uint32_t kRegSoftmax = 176, kRegAux = 80;
  static_assert(256 * (kRegSoftmax + kRegAux) == THREADS * 128, "register split of the four warpgroups");
  // bytes: q1 or q2; half of a stage's K; half of its V's columns, raw and in f16
  static constexpr uint32_t kQ = kTileRows * D, kK = kUnit * D, kV = kStageKeys * D / 2, kW = kStageKeys * D;
  static constexpr uint32_t kOffK = 2 * kQ, kOffV = kOffK + kNK * kK, kOffW = kOffV + kNV * kV;
  static constexpr uint32_t kOffInfo = kOffW + kNW * kW, kOffBar = kOffInfo + kNInfo * (uint32_t)sizeof(Batch);
  static constexpr uint32_t kOffPiece = kOffBar + 8 * NBAR;
  static constexpr uint32_t kOffEx = kOffPiece + kNItems * (uint32_t)sizeof(Piece);   // [2][half][row] floats
  static constexpr uint32_t kOffRef = kOffEx + 2 * 2 * kTileRows * 4;                 // [row] floats
  static constexpr uint32_t kOffMisc = kOffRef + kTileRows * 4;
  static constexpr uint32_t kSmem = kOffMisc + 64 + 1024;   // + alignment slack
  static_assert(kSmem <= 232448 && kOffMisc % 8 == 0, "shared memory");
  // K-major rows of D bytes, and V's rows of D / 2 columns in f16: 128-byte swizzle, or with D = 64 the 64-byte one
  static constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : 4u, kAtom = 8 * D;
  // the 16-byte vector c of row r
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (uint32_t)(r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
  }
};

// Instruction descriptors of 256 rows: f32 += e4m3 e4m3, both K-major; f32 += f16 f16, B MN-major.
__host__ __device__ constexpr uint32_t idesc(int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
}

// Products of the pair: A, B and D lie at the same addresses in both CTAs.
__device__ __forceinline__ void mma_8bit(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(id), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this address in both CTAs (one: in this one) when all earlier products of this
// thread are done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
// The address of this CTA's shared memory as the first CTA has it.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_bar) : "memory");
}
// As wait_warp, for the two warps that issue products, with one way out (whole frames of d = 128 and 64 take 654 and
// 545 us with it, with wait_warp 658 and 550).
__device__ __forceinline__ bool wait_issue(uint32_t bar, uint32_t parity, const Guard& g) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1; !ok; ++it) {
      ok = mbar_try_wait(bar, parity);
      if (!ok && (it & 63u) == 0) {
        if (*g.abort) break;
        if (globaltimer_ns() - t0 > g.limit_ns) {
          *g.abort = 1;
          report(g.d_status, SPARSP_ERR_TIMEOUT);
          break;
        }
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// A TMA box into this CTA's shared memory whose bytes count on a barrier of either CTA.
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
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

// Items of the whole call, for this kernel: entries are requests, or with lists request
// and key head; an entry's items are its key heads' row groups.
struct Walk {
  const CacheAttn& a;
  __device__ __forceinline__ int stages(const Entry& x, int group) const {
    if (a.row_ptr != nullptr) return (x.units + 1) / 2;
    int keys = x.len;
    if (a.causal) {   // up to the last row's token
      const int tok = (int)min((uint32_t)x.n, ((uint32_t)(group + 1) * kItemRows - 1) / (uint32_t)a.group + 1) - 1;
      keys = max(0, min(keys, x.len - x.n + tok + 1));
    }
    return (int)(((uint32_t)keys + kStageKeys - 1) / kStageKeys);   // keys may be 2^31 - 64
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
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<D>::THREADS, 1)
attn_cache_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const CacheAttn a,
                     const Parts parts) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base, sK = base + C::kOffK, sV = base + C::kOffV, sW = base + C::kOffW;
  auto bar = [&](int i) -> uint32_t { return base + C::kOffBar + 8u * (uint32_t)i; };
  Batch* infos = reinterpret_cast<Batch*>(gbase + C::kOffInfo);
  Piece* pieces = reinterpret_cast<Piece*>(gbase + C::kOffPiece);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(gbase + C::kOffMisc + 4);
  int64_t* s_begin = reinterpret_cast<int64_t*>(gbase + C::kOffMisc + 16);   // first entry, its offset
  __shared__ int64_t s_scan[C::THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)(blockIdx.x & 1u);
  auto lead = [&](int i) -> uint32_t { return in_first(bar(i)); };   // the first CTA's
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // ---- this cluster's range of stages
  const Walk walk{a};
  const int entries = entries_of(a), per = (entries + C::THREADS - 1) / C::THREADS;
  const int n0 = min(entries, (int)threadIdx.x * per), n1 = min(entries, n0 + per);
  int64_t mine = 0;
  for (int e = n0; e < n1; ++e) mine += walk.at(e, blockIdx.x == 0).weight;
  int64_t total, below = scan_below<C::THREADS / 32>(mine, s_scan, &total);
  const int64_t ctas = min((int64_t)gridDim.x / 2, max((int64_t)1, (total + kMinStages - 1) / kMinStages)), cta = blockIdx.x / 2;
  const int64_t begin = cta * total / ctas, end = cta < ctas ? (cta + 1) * total / ctas : begin;
  if (threadIdx.x == 0 && rank == 0) parts.open[cta].last = -1;
  if (cta >= ctas || begin >= end) return;      // the same for the whole cluster
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
    init(W_FULL, kNW, 2 * 4);
    init(W_EMPTY, kNW, 1);
    init(INFO, kNInfo, 1);
    init(I_FULL, kNItems, 1);
    init(I_EMPTY, kNItems, kSoftmax + 4 + (rank == 0 ? 2 : 0));   // softmax, widening and issuing warps
    init(Q_FULL, 1, 2 * kSoftmax);
    init(S_FULL, kNS, 1);
    init(P_FULL, kNS, kSoftmax);  // a stage is four warps' in each CTA
    init(PV_DONE, kNS, 1);
    init(O_EMPTY, 1, 2 * kSoftmax);
    init(TEAR, 2, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_PROD && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == W_S) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync();                               // the barriers of both CTAs are ready
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, a.d_status, kWaitNs};
  const uint32_t col_o = tmem + 384u;
  auto col_s = [&](uint32_t b) { return tmem + b * 128u; };   // S, and then P in the first 64 columns
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

  if (warp >= kSoftmax) {
    regs_decrease<C::kRegAux>();
    if (warp == W_PROD) {
      // ------------------------------------------------------------ producer
      uint32_t it_fill = 0, k_fill = 0, v_fill = 0, n_batch = 0;
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
        if (!whole && e0 == 0 && lane == 0 && rank == 0)
          parts.open[cta] = Open{hk, row0, rows, x.s0, (int)(((item_at + size) * ctas - 1) / total)};
        if (!(ok = publish(Piece{x.s0, hk, row0, rows, x.n, x.len, e0, e1, whole ? -1 : slot}))) break;

        // look-ups: lane i takes the half stage (64 keys) u0 + i of a batch of 32
        const int32_t* table = a.table + (int64_t)x.b * a.max_blocks;
        const int32_t* list = a.row_ptr != nullptr ? a.col_idx + a.row_ptr[entry] : nullptr;
        struct Half {
          Info info;
          int page, row;
        };
        auto look = [&](int u) -> Half {
          Half h{{0, 0, 1.f, 0.f, 1.f, 0.f, 0.f, 0}, 0, 0};
          if (u >= 2 * e1 || u >= x.units) return h;
          int j = u / per_block;
          if (list != nullptr) j = __ldg(list + j);
          if (!has_tokens(a, x, j)) {
            report(a.d_status, SPARSP_ERR_DATA);
            return h;
          }
          const int page = __ldg(table + j);
          if (!in_pool(a, page)) {
            report(a.d_status, SPARSP_ERR_DATA);
            return h;
          }
          const int64_t block = (int64_t)page * a.c.heads + hk;
          const int in_block = u % per_block * kUnit;
          h.page = page;
          h.row = hk * a.c.bt + in_block;
          h.info.pos = j * a.c.bt + in_block;
          h.info.valid = max(0, min(kUnit, x.len - j * a.c.bt - in_block));
          h.info.ks = __ldg(a.ks + block);
          h.info.lv = log2f(fmaxf(__ldg(a.vs + block), kLeastScale));
          return h;
        };
        // ... against u, the largest of the batch where that is far above what it was
        float lu = 0.f;
        auto place = [&](Info& f, bool first) {
          float most = f.valid > 0 ? f.lv : -INFINITY;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
          const float was = lu;
          if (most > -INFINITY && (first || most > lu + kAbove)) lu = most;
          f.lu = lu;
          f.rise = lane < 2 ? lu - was : 0.f;    // (of a piece's first stage: no matter)
          f.held = f.valid > 0 && f.lv >= lu - kBelow ? f.valid : 0;
          f.lv = f.held > 0 ? f.lv - lu : 0.f;
          f.inv = exp2f(-f.lv);
        };
        Half now, ahead = look(2 * e0 + lane);
        for (int e = e0; e < e1; ++e) {
          const int i = 2 * (e - e0) & 31;      // this stage's halves: lanes i, i + 1
          if (i == 0) {
            now = ahead;
            ahead = look(2 * e + 32 + lane);
            place(now.info, e == e0);
            const uint32_t is = n_batch++ % kNInfo;
            infos[is].half[lane >> 1][lane & 1] = now.info;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(INFO + is));
          }
          const int v0 = __shfl_sync(0xffffffffu, now.info.valid, i), v1 = __shfl_sync(0xffffffffu, now.info.valid, i + 1);
          const int p0 = __shfl_sync(0xffffffffu, now.page, i), p1 = __shfl_sync(0xffffffffu, now.page, i + 1);
          const int r0 = __shfl_sync(0xffffffffu, now.row, i), r1 = __shfl_sync(0xffffffffu, now.row, i + 1);
          const uint32_t halves = (v0 > 0 ? 1u : 0u) + (v1 > 0 ? 1u : 0u);
          const uint32_t ks = k_fill % kNK, vs = v_fill % kNV;
          if (!(ok = wait_warp(bar(K_EMPTY + ks), ((k_fill / kNK) & 1u) ^ 1u, g))) break;
          if (lane == 0) {                      // this CTA's half of the keys
            if (rank == 0) mbar_arrive_expect_tx(bar(K_FULL + ks), halves * (uint32_t)(kUnit * D));
            if ((rank == 0 ? v0 : v1) > 0)
              tma_pair(sK + ks * C::kK, &tk, lead(K_FULL + ks), 0, rank == 0 ? r0 : r1, rank == 0 ? p0 : p1);
          }
          __syncwarp();
          ++k_fill;
          if (!(ok = wait_warp(bar(V_EMPTY + vs), ((v_fill / kNV) & 1u) ^ 1u, g))) break;
          if (lane == 0) {                      // this CTA's half of the columns
            mbar_arrive_expect_tx(bar(V_FULL + vs), halves * (uint32_t)(kUnit * D / 2));
            if (v0 > 0) tma_load_3d(sV + vs * C::kV, &tv, bar(V_FULL + vs), rank * (D / 2), r0, p0);
            if (v1 > 0) tma_load_3d(sV + vs * C::kV + kUnit * D / 2, &tv, bar(V_FULL + vs), rank * (D / 2), r1, p1);
          }
          __syncwarp();
          ++v_fill;
        }
      }
      if (ok) publish(Piece{0, 0, 0, 0, 0, 0, 0, -1, 0});
      if (*abort_flag) {
        // copies in flight end before the CTA does
        for (uint32_t i = 0; rank == 0 && i < kNK; ++i)
          if (k_fill > i) wait_raw(bar(K_FULL + (k_fill - 1 - i) % kNK), ((k_fill - 1 - i) / kNK) & 1u, kDrainNs);
        for (uint32_t i = 0; i < kNV; ++i)
          if (v_fill > i) wait_raw(bar(V_FULL + (v_fill - 1 - i) % kNV), ((v_fill - 1 - i) / kNV) & 1u, kDrainNs);
      }
      __syncwarp();
    } else if (warp == W_S && rank == 0) {
      // ------------------------------------------------------------ S = Q K^T issuer
      uint32_t n = 0, n_q = 0;
      bool issued = false, ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        if (!(ok = wait_issue(bar(Q_FULL), n_q++ & 1u, g))) break;
        for (int e = x.e0; e < x.e1; ++e, ++n) {
          const uint32_t ks = n % kNK, b = n % kNS;
          if (!(ok = wait_issue(bar(K_FULL + ks), (n / kNK) & 1u, g))) break;
          if (!(ok = wait_warp(bar(PV_DONE + b), ((n / kNS) & 1u) ^ 1u, g))) break;
          fence_after();
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_8bit(col_s(b), smem_desc(sQ + (uint32_t)q * C::kQ + 32u * kk, 16, C::kAtom, C::kSwz),
                         smem_desc(sK + ks * C::kK + 32u * kk, 16, C::kAtom, C::kSwz), idesc(kStageKeys, 0),
                         q > 0 || kk > 0 ? 1u : 0u);
            commit_both(bar(S_FULL + b));
            commit_both(bar(K_EMPTY + ks));
          }
          __syncwarp();
          issued = true;
        }
      }
      if (*abort_flag && issued) {
        if (elect_one()) commit_one(bar(TEAR));
        __syncwarp();
        wait_raw(bar(TEAR), 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp == W_PV && rank == 0) {
      // ------------------------------------------------------------ O += P V issuer
      uint32_t n = 0, n_o = 0;
      bool issued = false, ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        for (int e = x.e0; e < x.e1; ++e, ++n) {
          const uint32_t ws = n % kNW, b = n % kNS;
          if (!(ok = wait_issue(bar(W_FULL + ws), (n / kNW) & 1u, g))) break;
          if (!(ok = wait_issue(bar(P_FULL + b), (n / kNS) & 1u, g))) break;
          if (e == x.e0 && !(ok = wait_issue(bar(O_EMPTY), (n_o++ & 1u) ^ 1u, g))) break;
          fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kStageKeys / 16; ++kk)
              mma_f16(col_o, col_s(b) + 8u * kk, smem_desc(sW + ws * C::kW + 16u * D * kk, 16, C::kAtom, C::kSwz), idesc(D, 1),
                      e > x.e0 || kk > 0 ? 1u : 0u);
            commit_both(bar(PV_DONE + b));
            commit_both(bar(W_EMPTY + ws));
          }
          __syncwarp();
          issued = true;
        }
      }
      if (*abort_flag && issued) {
        if (elect_one()) commit_one(bar(TEAR_PV));
        __syncwarp();
        wait_raw(bar(TEAR_PV), 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp < W_PROD) {
      // ------------------------------------------------------------ V to f16
      constexpr int CH = D / 32;                // 16-code vectors of this CTA's half of a row
      const int id = threadIdx.x - 32 * W_WIDEN;
      uint32_t n = 0, n_batch = 0;
      bool ok = true;
      Piece x;
      while (ok && next_piece(x)) {
        for (int e = x.e0; e < x.e1; ++e) {
          const uint32_t vs = n % kNV, ws = n % kNW;
          if ((e - x.e0) % kBatch == 0) {
            if (!(ok = wait_warp(bar(INFO + n_batch % kNInfo), (n_batch / kNInfo) & 1u, g))) break;
            ++n_batch;
          }
          const Info* half = infos[(n_batch - 1) % kNInfo].half[(e - x.e0) % kBatch];
          const int held0 = half[0].held, held1 = half[1].held;
          if (!(ok = wait_warp(bar(V_FULL + vs), (n / kNV) & 1u, g))) break;
          if (!(ok = wait_warp(bar(W_EMPTY + ws), ((n / kNW) & 1u) ^ 1u, g))) break;
          const uint4* from = reinterpret_cast<const uint4*>(gbase + C::kOffV + vs * C::kV);
          uint8_t* to = gbase + C::kOffW + ws * C::kW;
#pragma unroll
          for (int i = 0; i < kStageKeys * CH / 128; ++i) {
            const int v = id + 128 * i, r = v / CH, c = v % CH;   // row, and columns 16 c .. of the half
            uint4 w = from[v];
            if ((r & 63) >= (r < 64 ? held0 : held1)) w = make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              out[2 * k] = f16x2_of_e4m3(in[k]);
              out[2 * k + 1] = f16x2_of_e4m3(in[k] >> 16);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)         // a row of D / 2 values in f16 has D bytes, as one of K has
              *reinterpret_cast<uint4*>(to + C::at(r, 2 * c + k)) = make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(V_EMPTY + vs));
            arrive_cluster(lead(W_FULL + ws));
          }
          ++n;
        }
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::kRegSoftmax>();
    // -------------------------------------------------------------- softmax + epilogue of this CTA's rows
    const int half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;   // r: row of the CTA = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // named barriers of the two warps that share rows: of both, and of the references of even and of odd stages
    const int pair_bar = 1 + (warp & 3), ref_bar = 5 + (warp & 3);
    float* ex = reinterpret_cast<float*>(gbase + C::kOffEx) + r;
    volatile float* ref_at = reinterpret_cast<volatile float*>(gbase + C::kOffRef) + r;
    const uint32_t p_full = lead(P_FULL);
    uint32_t n = 0, n_ex = 0, n_batch = 0;       // stages, exchanges, batches of facts
    bool ok = true;
    // The row's other thread: gives its value for this one's. A warp that has given up says so here, or with the
    // reference (NaN with these bits); both leave after this.
    constexpr uint32_t kGone = 0x7fc0dead;
    auto exchange = [&](float mine, float& theirs) -> bool {
      float* at = ex + (n_ex++ & 1u) * 2 * kTileRows;   // the other buffer may still be read
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
      const int row = x.row0 + rank * kTileRows + r;
      const bool live = rank * kTileRows + r < x.rows;
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
        uint8_t* q1 = gbase;
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
            const uint32_t big = e4m3_pair(f0, f1);
            const float2 b = e4m3_values(big);
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
        if (lane == 0) arrive_cluster(lead(Q_FULL));
      }
      const int last = a.causal ? x.len - x.n + tok : INT32_MAX;   // the last key that the row sees
      float ref = -INFINITY, l = 0.f;            // R; l times 2^11, of this thread's stages
      // what the row sees of a stage's halves, and their scales
      int see[2];
      float c[2], lv[2], inv[2], rise;
      const uint32_t begin_n = n, end_n = n + (uint32_t)(x.e1 - x.e0);
      int known = -1;                            // batches of this piece that are there
      auto facts = [&](uint32_t n) {
        const int j = (int)(n - begin_n), batch = j / kBatch;
        rise = 0.f;                              // only with a batch's first stage
        const uint32_t is = (n_batch + batch) % kNInfo;
        if (batch > known) {
          ok = ok && wait_warp(bar(INFO + is), ((n_batch + batch) / kNInfo) & 1u, g);
          known = batch;
          rise = infos[is].half[j % kBatch][0].rise;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const Info& f = infos[is].half[j % kBatch][k];
          const int4 w = *reinterpret_cast<const int4*>(&f);
          see[k] = min(w.y, last - w.x < 63 ? last - w.x + 1 : 64);
          c[k] = see[k] > 0 ? score_factor<true>(factor, __int_as_float(w.z)) : 1.f;   // what is hidden says nothing
          lv[k] = __int_as_float(w.w);
          inv[k] = f.inv;
        }
      };
      if ((n & 1u) != (uint32_t)half) ++n;
      for (; n < end_n; n += 2) {
        // What needs shared memory comes while S does, as beside the products' reads every access takes hundreds of
        // cycles (651 -> 629 us): the reference after the stage before, and what is known of the keys.
        float was = -INFINITY;
        if (n > 0) {
          asm volatile("bar.sync %0, 64;\n" ::"r"(ref_bar + 4 * (half ^ 1)) : "memory");
          was = *ref_at;
        }
        facts(n);
        ok = ok && !__any_sync(0xffffffffu, __float_as_uint(was) == kGone);
        if (n == begin_n) was = -INFINITY;
        const bool cut = __any_sync(0xffffffffu, see[0] < 64 || see[1] < 64);
        const uint32_t sb = n % kNS, t_s = col_s(sb) + lanes;
        ok = ok && wait_warp(bar(S_FULL + sb), (n / kNS) & 1u, g);
        fence_after();
        uint32_t s[kStageKeys];
        float cm[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cm[i] = tmem_ld32_max(t_s + 32u * i, s + 32 * i);
        wait_ld();
        if (cut) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cm[i] = -INFINITY;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if ((i & 1) * 32 + k >= see[i >> 1]) s[32 * i + k] = 0xff800000u;
              cm[i] = fmaxf(cm[i], __uint_as_float(s[32 * i + k]));
            }
          }
        }
        // a half without keys says nothing (its product with a scale might)
        const float top = fmaxf(see[0] > 0 ? fmaf(fmaxf(cm[0], cm[1]), c[0], lv[0]) : -INFINITY,
                                see[1] > 0 ? fmaf(fmaxf(cm[2], cm[3]), c[1], lv[1]) : -INFINITY);
        // this stage's reference, for the one after
        const bool moves = top > was + kMoves;   // by itself: not by what other rows hold
        const float now = moves ? top : was;
        *ref_at = ok ? now : __uint_as_float(kGone);
        asm volatile("bar.arrive %0, 64;\n" ::"r"(ref_bar + 4 * half) : "memory");
        if (!ok) break;
        float f = moves ? exp2_fast(was - now) : 1.f;         // 0 for the first
        if (rise != 0.f) f *= exp2_fast(-rise);
        if (now != ref) l *= exp2_fast(ref - now);            // from where this thread left it
        ref = now;
        const float against = ref == -INFINITY ? 0.f : ref;
        float sum[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float off = lv[k] + kShift - against;
          float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1;
              fma_x2(__uint_as_float(s[64 * k + 32 * q + 2 * i]), __uint_as_float(s[64 * k + 32 * q + 2 * i + 1]), c[k], off, x0,
                     x1);
              const float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
              add_x2(rs[2 * (i & 1)], rs[2 * (i & 1) + 1], p0, p1);
              pk[i] = pack_f16(p0, p1);
            }
            tmem_st16(t_s + 32u * k + 16u * q, pk);
          }
          sum[k] = (rs[0] + rs[1]) + (rs[2] + rs[3]);
        }
        l = fmaf(sum[0], inv[0], fmaf(sum[1], inv[1], l));
        if (n > begin_n && __any_sync(0xffffffffu, f != 1.f)) {   // O follows the reference, after the PV of the last stage
          ok = ok && wait_warp(bar(PV_DONE + (n - 1) % kNS), ((n - 1) / kNS) & 1u, g);
          fence_after();
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t ov[32];
            tmem_ld32(col_o + lanes + 32u * i, ov);
            wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * f);
            tmem_st32(col_o + lanes + 32u * i, ov);
          }
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(p_full + 8u * sb);
      }
      n = end_n;
      n_batch += (uint32_t)(x.e1 - x.e0 + kBatch - 1) / kBatch;
      // ---- the end of a piece: the row's reference and whole sum, and half of O from TMEM
      ok = ok && wait_warp(bar(PV_DONE + (n - 1) % kNS), ((n - 1) / kNS) & 1u, g);
      if (!exchange(ref, theirs)) break;
      // the thread of the last stage has the reference that holds
      const float final_ref = ((n - 1) & 1u) == (uint32_t)half ? ref : theirs;
      if (final_ref != ref) l *= exp2_fast(ref - final_ref);
      ref = final_ref;
      if (!exchange(l, theirs)) break;
      l = half ? theirs + l : l + theirs;
      fence_after();
      const uint32_t t_o = col_o + lanes + (uint32_t)half * (D / 2);
      const bool none = l == 0.f;
      const float scale = none ? 0.f : 1.0f / l, u = exp2_fast(infos[(n_batch - 1) % kNInfo].half[0][0].lu);
      const int64_t at = (int64_t)(x.s0 + tok) * a.H + h;
      float* part_o = parts.o + ((int64_t)max(x.part, 0) * kItemRows + rank * kTileRows + r) * D + half * (D / 2);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t ov[32];
        tmem_ld32(t_o + 32u * i, ov);
        wait_ld();
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) ov[k] = none ? 0u : __float_as_uint(__uint_as_float(ov[k]) * scale * u);   // (u may be tiny)
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
            *reinterpret_cast<uint4*>(part_o + 32 * i + 4 * k) = make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(lead(O_EMPTY));
      if (live && half == 0) {
        const float lse2 = none ? -INFINITY : ref - kShift + log2f(l);
        if (x.part < 0) a.lse[at] = lse2 * 0.6931471805599453f;
        else parts.ml[(int64_t)x.part * kItemRows + rank * kTileRows + r] = make_float2(lse2, none ? 0.f : 1.f);
      }
    }
  }

  fence_before();
  __syncthreads();
  cluster_sync();                               // neither reads the other's memory any more
  fence_after();
  if (warp == W_S)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
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
      const float f = part_weight(parts.ml[row_of(i, r)], top);
      sum += f;
      if (4 * lane < D) {
        const float4 w = *reinterpret_cast<const float4*>(parts.o + row_of(i, r) * D + 4 * lane);
        all.x = fmaf(f, w.x, all.x);
        all.y = fmaf(f, w.y, all.y);
        all.z = fmaf(f, w.z, all.z);
        all.w = fmaf(f, w.w, all.w);
      }
    }
    if (4 * lane < D) finish_join<D>(a, it.s0, it.hk, it.row0 + r, 4 * lane, top, sum, all);
  }
}

constexpr int kGrid = 76;           // clusters

template <int D>
sparsp_status_t go(const CacheAttn& a, void* ws, cudaStream_t st) {
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.c.heads * a.c.bt, blocks = (uint64_t)a.c.blocks;
  if (!make_tmap_codes(&tk, a.kc, (uint64_t)D, rows, blocks, kUnit) ||
      !make_tmap_codes(&tv, a.vc, (uint64_t)D, rows, blocks, kUnit, D / 2))
    return SPARSP_ERR_CUDA;
  const Parts p = parts_of(ws, kGrid, kItemRows);
  constexpr int smem = Cfg<D>::kSmem;
  if (cudaFuncSetAttribute(attn_cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  attn_cache_tc_kernel<D><<<2 * kGrid, Cfg<D>::THREADS, smem, st>>>(tk, tv, a, p);
  SPARSP_LAUNCH_CHECK();
  return launch_after(attn_cache_tc_join_kernel<D>, dim3(kGrid, kItemRows / kJoinRows), 256, st, a, p);
}

}  // namespace

size_t attn_cache_tc_ws(const CacheDims& c) { return parts_bytes(kGrid, kItemRows, c.d); }

sparsp_status_t launch_attn_cache_tc(const CacheAttn& a, void* ws, cudaStream_t st) {
  return a.c.d == 64 ? go<64>(a, ws, st) : go<128>(a, ws, st);
}

}  // namespace sparsp
