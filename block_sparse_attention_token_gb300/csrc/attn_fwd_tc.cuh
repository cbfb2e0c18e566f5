// Step 5a, bf16, Bt and d in {64, 128} on sm_103a: block-sparse flash-attention
// forward on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// Every MMA works on 128 query rows (M = 128, the 128 TMEM lanes) and on
// stages of 128 key tokens. With 128-token blocks a work item is one query
// block and a stage one key block. With 64-token blocks a work item is a PAIR
// of neighbouring query blocks of a head (2p and 2p + 1: 128 contiguous rows)
// processed over the union of their two CSR rows, and a stage holds two key
// blocks of that union (two 64-row TMA boxes side by side); each 64-column half
// of S is masked, for each of the two query blocks, when that block did not
// select the key block (its P is zero there and no exponential is evaluated).
// So no MMA row or column is computed for nothing except where the two rows'
// selections differ ("Dynamic Sparsity in Large-Scale Video DiT Training",
// "How DSV works": queries grouped so that one key set serves several).
//
// Persistent CTAs: one per SM with 7 warps (4 softmax warps, then the
// producer, the S issuer and the PV issuer) for d = 128; two per SM for d = 64,
// each with 8 warps (4 softmax warps, the producer, one warp issuing both GEMM
// streams, two idle warps that only give their registers to the softmax
// warpgroup) and half of the TMEM and shared memory (one S and one P buffer;
// see Cfg::DUO):
//   producer: pulls items longest-first through an atomic counter,
//              validates the CSR row(s), publishes the item in a shared-memory
//              ring (for pairs with the two rows as bitmaps), and TMA-loads the
//              query tile and the K / V tiles of each stage (64-column boxes
//              with 128-byte swizzle) into 3-stage K and V rings, addressed
//              through the CSR (row coordinate = bh*N + j*Bt).
//   S issuer: S = Q K^T into one of two TMEM S buffers (M=N=128,
//              K=16 per instruction, both operands K-major from shared memory).
//   PV issuer: O += P V (A = P read from TMEM as packed bf16,
//              B = V MN-major from shared memory).
//              With d = 128 the two GEMM streams are issued by different warps
//              so that a wait in one (for P, or for a free S buffer) never
//              holds back the other; each warp runs uniformly and one elected
//              lane issues tcgen05.mma / tcgen05.commit.
//   softmax and epilogue: thread t owns query row t = TMEM lane t.
//              It reads its S row from TMEM with the sm_103 load-with-maximum
//              (tcgen05.ld.red: each 32-column load also returns the maximum of
//              the 32 values, so the row max costs no extra instructions), keeps
//              a running max m and sum l in
//              base 2, writes P = exp2(S*scale*log2e - m) as bf16 into TMEM, and
//              rescales its O row in TMEM only when the row max grows by more
//              than 8 (a factor 256); otherwise the stale max is kept, which
//              leaves the result unchanged up to rounding because O and l use
//              the same reference. At the end of the row: O / l to global
//              memory, LSE = (m + log2 l) ln 2 (O = 0, LSE = -inf for a row
//              that attended to nothing). A warp's 32 rows belong to one query
//              block, so the masks of a pair are warp-uniform.
// TMEM (512 columns): S0 [0,128), S1 [128,256), O [256,384), P0 [384,448),
// P1 [448,512); DUO (256 columns per CTA): S [0,128), O [128,192),
// P [192,256); FAST: three of S and then P [0,384), O [384,384+d).
// Every mbarrier wait is bounded (2 s); on expiry the CTA sets SPARSP_ERR_TIMEOUT, all roles leave their loops, copies and MMAs in flight
// are drained with a second bounded wait, and TMEM is released.
//
// MOD = 0 is attention over the selected blocks. MOD = 1 adds a token mask
// (mask.cuh) and MOD = 2 a score cap beside it, y = cap tanh(scale s / cap)
// (cap.cuh), for scores in the range of a softmax without a maximum (FAST); MOD = 3
// (cap) and 4 (none) are for any scores and do the items those pass on. The producer
// tells with the item which of its blocks the token mask cuts (by the blocks'
// ranges); in those each row's visible columns come as bits, the others run as
// they do without a mask. P is rounded to bf16 once, as without them (the tensor cores
// take no wider operand beside a bf16 V): O is off by 2.3e-3 in the mean square, of which
// 1.7e-3 are its own rounding; scores, sums and LSE are fp32.
#pragma once
#include <type_traits>

#include "cap.cuh"
#include "mask.cuh"
#include "pairs.cuh"
#include "tc_helpers.cuh"

namespace sparsp {
namespace {

using namespace tc;

constexpr int kMaxStages = 6, kNI = 4;   // K / V ring depth <= kMaxStages (Cfg::NK); item ring <= kNI
enum Bar {
  Q_FULL = 0, Q_EMPTY, K_FULL, K_EMPTY = K_FULL + kMaxStages, V_FULL = K_EMPTY + kMaxStages,
  V_EMPTY = V_FULL + kMaxStages, S_FULL = V_EMPTY + kMaxStages, S_FREE = S_FULL + 2, P_FULL = S_FREE + 2, PV_DONE = P_FULL + 2, O_FULL = PV_DONE + 2,
  O_EMPTY,
  I_FULL, I_EMPTY = I_FULL + kNI, TEAR = I_EMPTY + kNI, TEAR_PV, EXCH, NBAR = EXCH + 8,
  // FAST: three buffers, each S and then P, in the places of S_FULL to PV_DONE and the one
  // before (V's ring has less than kMaxStages stages there)
  S3_FULL = S_FULL - 1, P3_FULL = S3_FULL + 3, PV3_DONE = P3_FULL + 3
};
// Tile geometry for blocks of BT tokens and head dimension D. The query tile
// and a key/value stage are 128 rows each: one block, or two 64-token blocks
// (PAIR). Tiles are TMA'd as 64-column boxes of 128-byte rows with 128-byte
// swizzle; a stage of two blocks is two 64-row boxes per column box, the
// second 64 rows (8 KB, a whole number of 1 KB swizzle atoms) after the first.
template <int BT_, int D_, int MOD_ = 0>
struct Cfg {
  static constexpr int BT = BT_, D = D_, QR = 128, KR = 128;
  static constexpr bool PAIR = BT == 64;
  // d = 64 (64- or 128-token blocks): two CTAs per SM, each with half of the TMEM
  // (one S buffer [0,128), O [128,192), one P buffer [192,256)) and half of
  // the shared memory (3 K and 2 V stages), so that one CTA's softmax runs
  // while the other's MMAs keep the tensor pipe busy. The softmax warps hold
  // a whole 128-column S row in registers (one pass per stage, S released as
  // soon as it is loaded) with the 200 registers the register split below
  // gives them.
  static constexpr bool FAST = MOD_ == 1 || MOD_ == 2;
  static constexpr bool DUO = D == 64 && !FAST;
  static constexpr int NSM = FAST ? 16 : 4;           // softmax warps
  // arrivals of the softmax warps at S_FREE, P_FULL and O_EMPTY: every thread, or with
  // MOD one lane of each warp concerned
  static constexpr int kArrivals = MOD_ == 0 ? 32 * NSM : FAST ? 8 : 4;
  // MMA issuer warps: S and PV each get their own with d = 128; with DUO one
  // warp issues both streams (the softmax releases S(e-1) before it writes
  // P(e-1), so S(e) then PV(e-1) in one warp never wait on each other)
  static constexpr int NIS = DUO ? 1 : 2;
  // DUO: two idle warps complete the second warpgroup (producer, issuer), so
  // that the softmax warpgroup can take registers from it (setmaxnreg works
  // on whole warpgroups): two CTAs of 8 warps launch at 128 registers a
  // thread; the softmax warps rise to 200 and the other four drop to 56
  // (4 x 32 x 200 + 4 x 32 x 56 = 256 x 128)
  static constexpr int NIDLE = DUO ? 2 : 0;
  // FAST: the loads have a warp of their own, so that the producer prepares the next
  // item's lists and masks meanwhile
  static constexpr int NLD = FAST ? 1 : 0;
  static constexpr int THREADS = 32 * (NSM + 1 + NIS + NIDLE + NLD);   // + producer, issuer(s), idle, loader
  static constexpr int W_PROD = NSM, W_S = NSM + 1, W_PV = NSM + NIS, W_LOAD = W_PV + NIDLE + 1;
  static constexpr uint32_t kRegSoftmax = 200, kRegAux = 56;
  static_assert(!DUO || (THREADS == 256 && NSM == 4 && 128 * (kRegSoftmax + kRegAux) == 256 * 128),
                "register split of the two warpgroups");
  // K and V ring stages: 3 of each fit beside a d = 128 query tile; a DUO CTA
  // has half of the SM's shared memory for tiles of half the size: 3 K and 2 V
  // (four with FAST and d = 64, which has an SM's shared memory to itself; two V
  // stages with d = 128, whose row sums and cut bits need the room of the third)
  static constexpr int NK = FAST && D == 64 ? 4 : 3;
  static constexpr int NV = DUO || (FAST && D == 128) ? 2 : FAST ? 4 : 3;
  // S and P buffers in TMEM. FAST: three of 128 columns, P written over the S it is made
  // of, so that S of the stage after next is ready when its softmax warps come to it
  static constexpr int NSB = FAST ? 3 : DUO ? 1 : 2, NPB = NSB;
  static constexpr int B_S = FAST ? S3_FULL : S_FULL, B_P = FAST ? P3_FULL : P_FULL;
  static constexpr int B_PV = FAST ? PV3_DONE : PV_DONE;
  static constexpr int NI = DUO || PAIR || MOD_ != 0 ? 2 : kNI;   // item ring slots
  static constexpr int kMinCtas = DUO ? 2 : 1;                  // CTAs per SM
  static constexpr uint32_t kColS = 0, kColO = FAST ? 384 : DUO ? 128 : 256, kColP = DUO ? 192 : 384;
  static constexpr uint32_t kTmemCols = DUO ? 256 : 512;
  // bitmap words of one CSR row in the item ring (pairs): up to kMaxBlocks
  // blocks, except for d = 128 whose tiles leave room for 1,024 blocks only
  // (larger shapes run the portable kernel, see attn_fwd_tc_supported)
  static constexpr int MAXW = D == 64 ? kMaxBlocks / 32 : 32;
  static constexpr int NBOX = D / 64;                     // 64-column boxes per row tile
  static constexpr uint32_t kQBox = QR * 128, kKBox = KR * 128, kHalfBox = 64 * 128;
  static constexpr uint32_t kQTile = kQBox * NBOX, kKTile = kKBox * NBOX;
  static constexpr uint32_t kOffK = kQTile, kOffV = kOffK + NK * kKTile, kOffBar = kOffV + NV * kKTile;
  static constexpr uint32_t kOffRing = kOffBar + 8 * NBAR;
  static constexpr uint32_t kOffBits = kOffRing + 16 * NI;
  static constexpr uint32_t kBitsBytes = PAIR ? NI * 2 * MAXW * 4 : 0;
  // pairs: per item slot, which of the pair's two rows selected each block of
  // the union of their rows (ascending), written by the producer with the item
  // so that the softmax warps read a stage's masks with one shared-memory load:
  // one byte per block with DUO (bytes 2s, 2s + 1: stage s; bit 0 = the first
  // row, bit 1 = the second), two bits per block where shared memory is short
  // (d = 128: stage s is nibble s)
  static constexpr bool MASK_BYTES = DUO;
  // with MOD the codes of union_codes (a nibble per block), and without pairs one
  // bit per block of the row: does the token mask cut it
  static constexpr uint32_t kMaskWords = !PAIR ? (MOD_ != 0 ? kMaxBlocks / 32 : 0)
                                               : (MASK_BYTES ? 8 * MAXW + 4 : (MOD_ != 0 ? 4 : 2) * MAXW + 1);
  static constexpr uint32_t kOffMask = kOffBits + kBitsBytes;
  static constexpr uint32_t kOffEx = kOffMask + (NI * kMaskWords * 4 + 15) / 16 * 16;   // FAST: parts of the row sums
  static constexpr uint32_t kOffMisc = kOffEx + (FAST ? 2048 : 0);
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;   // + alignment slack
  static_assert(kSmemBytes <= (DUO ? 115712u : 232448u), "shared memory");
};
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

__device__ __forceinline__ bool wait_raw(uint32_t bar, uint32_t parity, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit) return false;
  return true;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// 32 columns of this thread's TMEM lane, and their maximum (sm_103 load with
// reduction)
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

struct Params {
  const int32_t* row_ptr;
  const int32_t* col_idx;
  int64_t N;
  int nb;
  int nbp;           // items per head: nb, or ceil(nb/2) pairs of 64-token blocks
  int64_t n_items;
  int64_t rows_total;   // B*H*N rows of Q, K, V, O and LSE
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  // raster output: O rows at rm.row(bh, block, token) (the layout of the inverse
  // reorder); otherwise block order like Q
  int raster;
  RasterMap rm;
  // raster input: Q, K, V read from [B, N, H, d] through 5-D maps, one block per box
  int in_raster;
  RasterBox rbox;
  const int32_t* items;
  int32_t* counter;
  uint64_t* prof;
  int32_t* d_status;
  MaskView mask;      // MOD != 0; mask.pos null: no mask
  // MOD 2, 3: 2 scale log2(e) / cap, cap log2(e) and scale / cap
  float c1, cap2, inv_cap;
  NearCap near;
  int exp_cap;           // cap <= kExpCap
  float c0;              // FAST: reference of every row, log2 units
  int32_t* fix_items;    // FAST: items for the general kernel, or null; the general kernel: its items
  int32_t* fix_count;
  int32_t* fix_mark;     // [items] zeroed: is the item on the list
};

template <int BT, int D, int MOD>
__global__ void __launch_bounds__(Cfg<BT, D, MOD>::THREADS, Cfg<BT, D, MOD>::kMinCtas)
attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  using C = Cfg<BT, D, MOD>;
  constexpr bool PAIR = C::PAIR;
  const uint32_t sQ = base, sK = base + C::kOffK, sV = base + C::kOffV;
  auto bar = [&](int idx) -> uint32_t { return base + C::kOffBar + 8u * (uint32_t)idx; };
  // ring entry: x = item, y = stages (-1: skip, -2: end), z = bad-row bits (pairs)
  volatile int4* ring = reinterpret_cast<volatile int4*>(gbase + C::kOffRing);
  uint32_t* bits = reinterpret_cast<uint32_t*>(gbase + C::kOffBits);   // [C::NI][2][C::MAXW] (pairs)
  uint32_t* masks = reinterpret_cast<uint32_t*>(gbase + C::kOffMask);   // [C::NI][C::kMaskWords] (pairs)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(gbase + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t t_start = globaltimer_ns();
  const int words = (p.nb + 31) >> 5;
  if (MOD > 2 && p.fix_count != nullptr && *p.fix_count == 0) return;   // nothing was passed on

  if (threadIdx.x == 0) {
    mbar_init(bar(Q_FULL), 1);
    mbar_init(bar(Q_EMPTY), 1);
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(bar(K_FULL + s), 1);
      mbar_init(bar(K_EMPTY + s), 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(bar(V_FULL + s), 1);
      mbar_init(bar(V_EMPTY + s), 1);
    }
    if (C::FAST) {
      static_assert(!C::FAST || C::NV < kMaxStages, "barriers");
      for (int b = 0; b < 3; ++b) {
        mbar_init(bar(S3_FULL + b), 1);
        mbar_init(bar(P3_FULL + b), C::kArrivals);
        mbar_init(bar(PV3_DONE + b), 1);
      }
    } else {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(S_FULL + b), 1);
        mbar_init(bar(S_FREE + b), C::kArrivals);
        mbar_init(bar(P_FULL + b), C::kArrivals);
      }
      mbar_init(bar(PV_DONE), 1);
      mbar_init(bar(PV_DONE + 1), 1);
    }
    mbar_init(bar(O_FULL), 1);
    mbar_init(bar(O_EMPTY), C::kArrivals);
    for (int r = 0; r < kNI; ++r) {
      mbar_init(bar(I_FULL + r), 1);
      mbar_init(bar(I_EMPTY + r), C::NSM + C::NIS + C::NLD);
    }
    mbar_init(bar(TEAR), 1);
    mbar_init(bar(TEAR_PV), 1);
    if (MOD != 0)
      for (int r = 0; r < 8; ++r) mbar_init(bar(EXCH + r), r < 4 ? 4 : 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::W_PROD && lane == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == C::W_S) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, p.d_status, kWaitNs};
  const int nb = p.nb, nbp = p.nbp;
  const int64_t n_items = MOD > 2 && p.fix_count != nullptr ? *p.fix_count : p.n_items;

  if (warp >= C::NSM) {
  if constexpr (C::DUO) regs_decrease<C::kRegAux>();   // the whole second warpgroup
  if (warp == C::W_PROD) {
    // ------------------------------------------------------------ producer
    uint32_t it_fill = 0, q_fill = 0, k_fill = 0, v_fill = 0;
    for (;;) {
      int32_t slot = 0;
      if (lane == 0) slot = atomicAdd(p.counter, 1);
      slot = __shfl_sync(0xffffffffu, slot, 0);
      const int ri = (int)(it_fill % C::NI);
      if (!wait_warp(bar(I_EMPTY + ri), ((it_fill / C::NI) & 1u) ^ 1u, g)) break;
      uint32_t* bmA = bits + ri * 2 * C::MAXW;
      uint32_t* bmB = bmA + C::MAXW;
      int32_t item = -1, len = -2, badbits = 0;
      if (slot < n_items) {
        item = p.items[slot];
        if constexpr (PAIR) {
          // the two rows as bitmaps in the ring slot; a bad row counts as empty
          const int64_t bh = item / nbp;
          const int iA = 2 * (item % nbp);
          if constexpr (MOD != 0) {
            badbits = pair_bitmaps(p.row_ptr, p.col_idx, nb, bh * nb + iA, iA + 1 < nb, bmA, bmB, words, lane);
          } else {
            for (int w = lane; w < 2 * C::MAXW; w += 32) bmA[w] = 0u;
            __syncwarp();
            const bool okA = list_bitmap(p.row_ptr, p.col_idx, nb, bh * nb + iA, bmA, words, lane);
            const bool okB = iA + 1 < nb ? list_bitmap(p.row_ptr, p.col_idx, nb, bh * nb + iA + 1, bmB, words, lane)
                                         : true;
            badbits = (okA ? 0 : 1) | (okB ? 0 : 2);
          }
          if (badbits && lane == 0) report(p.d_status, SPARSP_ERR_DATA);
          if (MOD != 0) badbits = 0;   // its bitmap is empty: it counts as an empty row
          const int u = union_count(bmA, bmB, words, lane);
          len = (badbits == 3) ? -1 : (u + 1) / 2;   // stages of two key blocks
          if constexpr (MOD != 0) {
            const int64_t blk0 = bh / p.rm.H * nb;
            const bool masked = p.mask.pos != nullptr;
            const int2 qa = masked ? __ldg(p.mask.qrange + blk0 + iA) : make_int2(0, 0);
            const int2 qb = masked && iA + 1 < nb ? __ldg(p.mask.qrange + blk0 + iA + 1) : qa;
            union_codes<false>(bmA, bmB, words, nb, u, lane, masks + ri * C::kMaskWords, [&](int j) -> uint32_t {
              if (!masked) return 0u;
              const int2 k = __ldg(p.mask.krange + blk0 + j);
              return (all_seen(qa, k) ? 0u : 1u) | (all_seen(qb, k) ? 0u : 2u);
            });
          } else if constexpr (C::MASK_BYTES)
            union_masks(bmA, bmB, words, u, lane, reinterpret_cast<uint8_t*>(masks + ri * C::kMaskWords));
          else
            union_masks2(bmA, bmB, words, u, lane, masks + ri * C::kMaskWords);
        } else {
          const int32_t a = p.row_ptr[item], b = p.row_ptr[item + 1];
          bool bad = (b < a) || (b - a > nb);
          if constexpr (MOD != 0) {
            const int64_t blk0 = (int64_t)item / nb / p.rm.H * nb;
            const bool masked = p.mask.pos != nullptr;
            const int2 q = masked ? __ldg(p.mask.qrange + blk0 + item % nb) : make_int2(0, 0);
            if (!bad)
              bad = list_cuts(p.col_idx + a, b - a, nb, lane, masks + ri * C::kMaskWords,
                              [&](int j) { return masked && !all_seen(q, __ldg(p.mask.krange + blk0 + j)); });
          } else {
            if (!bad)
              for (int32_t e = a + lane; e < b; e += 32) {
                const int32_t j = p.col_idx[e];
                if (j < 0 || j >= nb) bad = true;
              }
            bad = __any_sync(0xffffffffu, bad);
          }
          if (bad) {
            if (lane == 0) report(p.d_status, SPARSP_ERR_DATA);
            len = MOD != 0 ? 0 : -1;   // MOD: it counts as an empty row
          } else {
            len = b - a;
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        ring[ri].x = item;
        ring[ri].y = len;
        ring[ri].z = badbits;
        mbar_arrive(bar(I_FULL + ri));
      }
      __syncwarp();
      ++it_fill;
      if (len == -2) break;
      if (C::FAST || len <= 0) continue;
      const int64_t bh = item / nbp;
      const int i0 = PAIR ? 2 * (item % nbp) : item % nb;   // first query block of the item
      int32_t yq = (int32_t)(bh * p.N + (int64_t)i0 * BT);
      if (!dcheck(yq >= 0 && yq < p.rows_total, p.d_status)) yq = 0;
      if (!wait_warp(bar(Q_EMPTY), (q_fill & 1u) ^ 1u, g)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(Q_FULL), C::kQTile);
#pragma unroll
        for (int h = 0; h < C::NBOX; ++h) {
          if (p.in_raster) {   // the item's block(s), one 5-D box each
            const int4 c = p.rbox.at(bh, i0);
            tma_load_5d(sQ + h * C::kQBox, &tq, bar(Q_FULL), 64 * h, c.x, c.y, c.z, c.w);
            if (PAIR) {   // a head's last pair of an odd nb loads its first block twice (never stored)
              const int4 c2 = p.rbox.at(bh, i0 + 1 < nb ? i0 + 1 : i0);
              tma_load_5d(sQ + h * C::kQBox + C::kHalfBox, &tq, bar(Q_FULL), 64 * h, c2.x, c2.y, c2.z, c2.w);
            }
          } else {
            tma_load_2d(sQ + h * C::kQBox, &tq, bar(Q_FULL), 64 * h, yq);
          }
        }
      }
      ++q_fill;
      const int32_t e0 = PAIR ? 0 : p.row_ptr[item];
      UnionWalk walk(bmA, bmB, PAIR ? words : 0);
      bool ok = true;
      for (int e = 0; e < len && ok; ++e) {
        int32_t j1, j2 = 0;
        if constexpr (PAIR) {
          j1 = walk.next();
          j2 = walk.next();
          if (j2 < 0) j2 = j1;   // a lone last block: loaded twice, its second half masked
        } else {
          j1 = p.col_idx[e0 + e];
        }
        int32_t yk1 = (int32_t)(bh * p.N + (int64_t)j1 * BT);
        int32_t yk2 = (int32_t)(bh * p.N + (int64_t)j2 * BT);
        if (!dcheck(yk1 >= 0 && yk1 + BT <= p.rows_total && yk2 >= 0 && yk2 + BT <= p.rows_total, p.d_status))
          yk1 = yk2 = 0;   // keep the transaction counts; the result is flagged
        const uint32_t ks = k_fill % C::NK;
        if (!(ok = wait_warp(bar(K_EMPTY + ks), ((k_fill / C::NK) & 1u) ^ 1u, g))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(K_FULL + ks), C::kKTile);
#pragma unroll
          for (int h = 0; h < C::NBOX; ++h) {
            const uint32_t dst = sK + ks * C::kKTile + h * C::kKBox;
            if (p.in_raster) {
              const int4 c1 = p.rbox.at(bh, j1);
              tma_load_5d(dst, &tk, bar(K_FULL + ks), 64 * h, c1.x, c1.y, c1.z, c1.w);
              if (PAIR) {
                const int4 c2 = p.rbox.at(bh, j2);
                tma_load_5d(dst + C::kHalfBox, &tk, bar(K_FULL + ks), 64 * h, c2.x, c2.y, c2.z, c2.w);
              }
            } else {
              tma_load_2d(dst, &tk, bar(K_FULL + ks), 64 * h, yk1);
              if (PAIR) tma_load_2d(dst + C::kHalfBox, &tk, bar(K_FULL + ks), 64 * h, yk2);
            }
          }
        }
        ++k_fill;
        const uint32_t vs = v_fill % C::NV;
        if (!(ok = wait_warp(bar(V_EMPTY + vs), ((v_fill / C::NV) & 1u) ^ 1u, g))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(V_FULL + vs), C::kKTile);
#pragma unroll
          for (int h = 0; h < C::NBOX; ++h) {
            const uint32_t dst = sV + vs * C::kKTile + h * C::kKBox;
            if (p.in_raster) {
              const int4 c1 = p.rbox.at(bh, j1);
              tma_load_5d(dst, &tv, bar(V_FULL + vs), 64 * h, c1.x, c1.y, c1.z, c1.w);
              if (PAIR) {
                const int4 c2 = p.rbox.at(bh, j2);
                tma_load_5d(dst + C::kHalfBox, &tv, bar(V_FULL + vs), 64 * h, c2.x, c2.y, c2.z, c2.w);
              }
            } else {
              tma_load_2d(dst, &tv, bar(V_FULL + vs), 64 * h, yk1);
              if (PAIR) tma_load_2d(dst + C::kHalfBox, &tv, bar(V_FULL + vs), 64 * h, yk2);
            }
          }
        }
        ++v_fill;
      }
      if (!ok) break;
    }
    if (*abort_flag && lane == 0) {
      // drain copies still in flight before the shared memory goes away
      if (q_fill) wait_raw(bar(Q_FULL), (q_fill - 1) & 1u, kDrainNs);
      for (uint32_t s = 0; s < C::NK; ++s)
        if (k_fill > s) wait_raw(bar(K_FULL + s), ((k_fill - 1 - s) / C::NK) & 1u, kDrainNs);
      for (uint32_t s = 0; s < C::NV; ++s)
        if (v_fill > s) wait_raw(bar(V_FULL + s), ((v_fill - 1 - s) / C::NV) & 1u, kDrainNs);
    }
  } else if (C::FAST && warp == C::W_LOAD) {
    // ------------------------------------------------------------ loader (FAST)
    // K of the next stage, then V of the stage before it (and with an item's first V its
    // Q), so that S is not held up by V's ring. The instructions of a stage are what
    // bounds this warp (beside the softmax warps' loops they are seldom in the instruction
    // cache): one thread, no collective steps, one copy per block, running parities, the
    // next block's index read a stage early.
    if (lane == 0) {
      struct Stage {
        int32_t r1, r2;      // its blocks' first rows, or the blocks with raster inputs
        int32_t bh;
        int32_t first;       // its item's first query block where it is the first stage, else -1
        int32_t slot;        // its item's ring slot where it is the last stage, else -1
      };
      Stage now{0, 0, 0, -1, -1};   // the stage whose V is still to be loaded
      bool some = false, end = false, ok = true;
      uint32_t ks = 0, kp = 1, vs = 0, vp = 1, qp = 1, ri = 0, ip = 0;   // ring places and parities
      uint32_t k_fill = 0, v_fill = 0, q_fill = 0;
      int e = 0;
      int32_t len = 0, y0 = 0, bh = 0, i0 = 0, j_next = 0;
      const int32_t* list = p.col_idx;
      UnionWalk walk(bits, bits, 0);
      const int32_t unit = p.in_raster ? 1 : BT;
      auto rows = [&](uint32_t tile, uint32_t b, const CUtensorMap* map, const Stage& t) {   // K or V of a stage
        mbar_arrive_expect_tx(b, C::kKTile);
        if (p.in_raster) {
#pragma unroll 1
          for (int h = 0; h < C::NBOX; ++h) {
            const uint32_t dst = tile + h * C::kKBox;
            const int4 c1 = p.rbox.at(t.bh, t.r1);
            tma_load_5d(dst, map, b, 64 * h, c1.x, c1.y, c1.z, c1.w);
            if (PAIR) {
              const int4 c2 = p.rbox.at(t.bh, t.r2);
              tma_load_5d(dst + C::kHalfBox, map, b, 64 * h, c2.x, c2.y, c2.z, c2.w);
            }
          }
        } else if (PAIR && C::NBOX == 2) {   // the two blocks' rows alternate by 64-column box
#pragma unroll
          for (int h = 0; h < C::NBOX; ++h) {
            tma_load_3d(tile + h * C::kKBox, map, b, 0, t.r1, h);
            tma_load_3d(tile + h * C::kKBox + C::kHalfBox, map, b, 0, t.r2, h);
          }
        } else {                             // both boxes of d = 128 in one copy
          tma_load_3d(tile, map, b, 0, t.r1, 0);
          if (PAIR) tma_load_3d(tile + C::kHalfBox, map, b, 0, t.r2, 0);
        }
      };
      for (;;) {
        // the next item; one that is not ready is waited for only when nothing else is left to do
        while (e >= len && !end) {
          const uint32_t full = bar(I_FULL + ri);
          if (some && !mbar_test_wait(full, ip)) break;
          if (!(ok = wait(full, ip, g))) break;
          const int32_t item = ring[ri].x;
          len = ring[ri].y;
          e = 0;
          end = len == -2;
          if (len > 0) {
            bh = item / nbp;
            i0 = item - bh * nbp;
            if (PAIR) {
              i0 *= 2;
              walk = UnionWalk(bits + ri * 2 * C::MAXW, bits + ri * 2 * C::MAXW + C::MAXW, words);
            } else {
              list = p.col_idx + p.row_ptr[item];
              j_next = *list;
            }
            y0 = p.in_raster ? 0 : (int32_t)(bh * p.N);
          } else {
            mbar_arrive(bar(I_EMPTY + ri));
          }
          if (++ri == C::NI) ri = 0, ip ^= 1u;
        }
        if (!ok) break;
        const bool more = e < len;
        Stage next{0, 0, bh, -1, -1};
        if (more) {
          int32_t j1, j2;
          if constexpr (PAIR) {
            j1 = walk.next();
            j2 = walk.next();
            if (j2 < 0) j2 = j1;   // a lone last block: loaded twice, its second half masked
          } else {
            j1 = j2 = j_next;
            if (e + 1 < len) j_next = list[e + 1];
          }
          if (!dcheck(j1 >= 0 && j1 < nb && j2 >= 0 && j2 < nb, p.d_status)) j1 = j2 = 0;
          next.r1 = y0 + j1 * unit;
          next.r2 = y0 + j2 * unit;
          if (e == 0) next.first = i0;
          if (++e == len) next.slot = (int32_t)(ri == 0 ? C::NI - 1 : ri - 1);
          if (!(ok = wait(bar(K_EMPTY + ks), kp, g))) break;
          rows(sK + ks * C::kKTile, bar(K_FULL + ks), &tk, next);
          ++k_fill;
          if (++ks == C::NK) ks = 0, kp ^= 1u;
        } else if (!some && end) {
          break;
        }
        if (some) {
          if (now.first >= 0) {
            if (!(ok = wait(bar(Q_EMPTY), qp, g))) break;
            mbar_arrive_expect_tx(bar(Q_FULL), C::kQTile);
            if (p.in_raster) {   // the item's block(s), one 5-D box each
#pragma unroll 1
              for (int h = 0; h < C::NBOX; ++h) {
                const int4 c = p.rbox.at(now.bh, now.first);
                tma_load_5d(sQ + h * C::kQBox, &tq, bar(Q_FULL), 64 * h, c.x, c.y, c.z, c.w);
                if (PAIR) {   // a head's last pair of an odd nb loads its first block twice (never stored)
                  const int4 c2 = p.rbox.at(now.bh, now.first + 1 < nb ? now.first + 1 : now.first);
                  tma_load_5d(sQ + h * C::kQBox + C::kHalfBox, &tq, bar(Q_FULL), 64 * h, c2.x, c2.y, c2.z, c2.w);
                }
              }
            } else {
              tma_load_3d(sQ, &tq, bar(Q_FULL), 0, (int32_t)(now.bh * p.N) + now.first * BT, 0);
            }
            qp ^= 1u;
            ++q_fill;
          }
          if (!(ok = wait(bar(V_EMPTY + vs), vp, g))) break;
          rows(sV + vs * C::kKTile, bar(V_FULL + vs), &tv, now);
          ++v_fill;
          if (++vs == C::NV) vs = 0, vp ^= 1u;
          if (now.slot >= 0) mbar_arrive(bar(I_EMPTY + now.slot));   // the item's lists have been walked
        }
        some = more;
        now = next;
      }
      if (*abort_flag) {
        // drain copies still in flight before the shared memory goes away
        if (q_fill) wait_raw(bar(Q_FULL), (q_fill - 1) & 1u, kDrainNs);
        for (uint32_t s = 0; s < C::NK; ++s)
          if (k_fill > s) wait_raw(bar(K_FULL + s), ((k_fill - 1 - s) / C::NK) & 1u, kDrainNs);
        for (uint32_t s = 0; s < C::NV; ++s)
          if (v_fill > s) wait_raw(bar(V_FULL + s), ((v_fill - 1 - s) / C::NV) & 1u, kDrainNs);
      }
    }
    __syncwarp();
  } else if (C::DUO && warp == C::W_S) {
    // ------------------------------------------------------------ S and PV from one warp (DUO)
    // Per item: S(0), then S(e) before PV(e-1) for e = 1 .. len-1, then PV(len-1).
    // S(e) waits for the softmax to have loaded S(e-1) (one S buffer) and PV(e-1)
    // for P(e-1); the softmax releases S(e-1) before it writes P(e-1), so neither
    // wait holds back the other stream, and S(e) runs under the softmax of e-1.
    constexpr uint32_t idS = idesc_bf16(128, C::KR, 0, 0);
    constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
    uint32_t it_use = 0, q_use = 0, k_use = 0, v_use = 0, s_issue = 0, pv = 0, o_items = 0;
    bool issued_any = false, ok = true;
    for (;;) {
      const int ri = (int)(it_use % C::NI);
      if (!(ok = wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g))) break;
      const int len = ring[ri].y;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(I_EMPTY + ri));
      ++it_use;
      if (len == -2) break;
      if (len <= 0) continue;
      if (!(ok = wait_warp(bar(Q_FULL), q_use & 1u, g))) break;
      ++q_use;
      for (int e = 0; e <= len && ok; ++e) {
        if (e < len) {
          const uint32_t ks = k_use % C::NK;
          if (!(ok = wait_warp(bar(S_FREE), (s_issue & 1u) ^ 1u, g))) break;
          if (!(ok = wait_warp(bar(K_FULL + ks), (k_use / C::NK) & 1u, g))) break;
          fence_after();
          const uint32_t kb = sK + ks * C::kKTile;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t offq = (uint32_t)(kk >> 2) * C::kQBox + (uint32_t)(kk & 3) * 32u;
              const uint32_t offk = (uint32_t)(kk >> 2) * C::kKBox + (uint32_t)(kk & 3) * 32u;
              mma_ss(tmem + C::kColS, smem_desc(sQ + offq, 16, 1024, kSwizzle128B),
                     smem_desc(kb + offk, 16, 1024, kSwizzle128B), idS, kk > 0 ? 1u : 0u);
            }
            commit(bar(S_FULL));
            commit(bar(K_EMPTY + ks));
            if (e + 1 == len) commit(bar(Q_EMPTY));
          }
          __syncwarp();
          ++s_issue;
          ++k_use;
          issued_any = true;
        }
        if (e == 0) continue;
        // O += P(e-1) V(e-1)
        const uint32_t vs = v_use % C::NV;
        if (!(ok = wait_warp(bar(V_FULL + vs), (v_use / C::NV) & 1u, g))) break;
        if (!(ok = wait_warp(bar(P_FULL), pv & 1u, g))) break;
        if (e == 1 && !(ok = wait_warp(bar(O_EMPTY), (o_items & 1u) ^ 1u, g))) break;
        fence_after();
        const uint32_t vb = sV + vs * C::kKTile;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < C::KR / 16; ++kk)
            mma_ts(tmem + C::kColO, tmem + C::kColP + (uint32_t)kk * 8u,
                   smem_desc(vb + (uint32_t)kk * 2048u, C::kKBox, 1024, kSwizzle128B), idO,
                   (e > 1 || kk > 0) ? 1u : 0u);
          commit(bar(V_EMPTY + vs));
          commit(bar(PV_DONE));
          if (e == len) commit(bar(O_FULL));
        }
        __syncwarp();
        ++v_use;
        ++pv;
      }
      if (!ok) break;
      ++o_items;
    }
    if (*abort_flag && issued_any) {
      if (elect_one()) commit(bar(TEAR));
      __syncwarp();
      wait_raw(bar(TEAR), 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == C::W_S) {
    // ------------------------------------------------------------ S = Q K^T issuer
    constexpr uint32_t idS = idesc_bf16(128, C::KR, 0, 0);
    uint32_t it_use = 0, q_use = 0, k_use = 0, s_issue = 0;
    bool issued_any = false;
    for (;;) {
      const int ri = (int)(it_use % C::NI);
      if (!wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g)) break;
      const int len = ring[ri].y;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(I_EMPTY + ri));
      ++it_use;
      if (len == -2) break;
      if (len <= 0) continue;
      if (!wait_warp(bar(Q_FULL), q_use & 1u, g)) break;
      ++q_use;
      bool ok = true;
      for (int e = 0; e < len; ++e) {
        const uint32_t b = s_issue % C::NSB, ks = k_use % C::NK;
        // FAST: the buffer held P until its PV was done
        if (!(ok = wait_warp(bar((C::FAST ? C::B_PV : S_FREE) + b), ((s_issue / C::NSB) & 1u) ^ 1u, g))) break;
        if (!(ok = wait_warp(bar(K_FULL + ks), (k_use / C::NK) & 1u, g))) break;
        fence_after();
        const uint32_t kb = sK + ks * C::kKTile;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            // k-step kk: 16 columns = 32 bytes into the row, in box kk / 4
            const uint32_t offq = (uint32_t)(kk >> 2) * C::kQBox + (uint32_t)(kk & 3) * 32u;
            const uint32_t offk = (uint32_t)(kk >> 2) * C::kKBox + (uint32_t)(kk & 3) * 32u;
            mma_ss(tmem + C::kColS + b * 128u, smem_desc(sQ + offq, 16, 1024, kSwizzle128B),
                   smem_desc(kb + offk, 16, 1024, kSwizzle128B), idS, kk > 0 ? 1u : 0u);
          }
          commit(bar(C::B_S + b));
          commit(bar(K_EMPTY + ks));
          if (e + 1 == len) commit(bar(Q_EMPTY));   // every S of this item is issued
        }
        __syncwarp();
        ++s_issue;
        ++k_use;
        issued_any = true;
      }
      if (!ok) break;
    }
    if (*abort_flag && issued_any) {
      if (elect_one()) commit(bar(TEAR));
      __syncwarp();
      wait_raw(bar(TEAR), 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == C::W_PV) {
    // ------------------------------------------------------------ O += P V issuer
    constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
    uint32_t it_use = 0, v_use = 0, pv = 0, o_items = 0;
    bool issued_any = false;
    for (;;) {
      const int ri = (int)(it_use % C::NI);
      if (!wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g)) break;
      const int len = ring[ri].y;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(I_EMPTY + ri));
      ++it_use;
      if (len == -2) break;
      if (len <= 0) continue;
      bool ok = true;
      for (int e = 0; e < len; ++e) {
        const uint32_t b = pv % C::NPB, vs = v_use % C::NV;
        if (!(ok = wait_warp(bar(V_FULL + vs), (v_use / C::NV) & 1u, g))) break;
        if (!(ok = wait_warp(bar(C::B_P + b), (pv / C::NPB) & 1u, g))) break;
        if (e == 0 && !(ok = wait_warp(bar(O_EMPTY), (o_items & 1u) ^ 1u, g))) break;
        fence_after();
        const uint32_t vb = sV + vs * C::kKTile;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < C::KR / 16; ++kk)
            mma_ts(tmem + C::kColO,
                   C::FAST ? tmem + C::kColS + b * 128u + (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u
                           : tmem + C::kColP + b * 64u + (uint32_t)kk * 8u,
                   smem_desc(vb + (uint32_t)kk * 2048u, C::kKBox, 1024, kSwizzle128B), idO,
                   (e > 0 || kk > 0) ? 1u : 0u);
          commit(bar(V_EMPTY + vs));
          commit(bar(C::B_PV + b));
          if (e + 1 == len) commit(bar(O_FULL));
        }
        __syncwarp();
        ++v_use;
        ++pv;
        issued_any = true;
      }
      if (!ok) break;
      ++o_items;
    }
    if (*abort_flag && issued_any) {
      if (elect_one()) commit(bar(TEAR_PV));
      __syncwarp();
      wait_raw(bar(TEAR_PV), 0, kDrainNs);
    }
    __syncwarp();
  }
  } else if constexpr (C::FAST) {
    // ------------------------------------------------------------ softmax + epilogue with a mask or a cap
    // No running maximum: P = exp2(y - c0) with one constant c0 for every row. With a
    // cap of at most kFixedCap the scores cannot leave the range of that; else
    // c0 = 0 and an item with a row whose sum left [2^-60, 2^80], or whose O is not
    // finite or too small beside its sum, goes on the list of items that the general kernel
    // does after this one (scores of more than 55, or all below -42: a softmax that is one key).
    // So stages do not depend on one another and nothing is rescaled. Two groups of
    // eight warps take the stages in turn, two warps per 32 rows with 64 columns each, so
    // that the waits and loads of some run under the arithmetic of others; three S / P
    // buffers, so that neither group waits for its next S. A warp goes through TMEM 32 columns at
    // a time in a loop that is not unrolled: unrolled, its variants do not stay
    // in the instruction cache. At the end of an item the parts of the row sum
    // meet in shared memory and group 0 writes O and LSE while group 1 goes on.
    // Measured: 65,536 tokens, 24 heads of 128, clips: 3.35 ms (the kernel without a mask
    // 3.27 ms on the same blocks), the tensor pipe issuing 70% of the time; 30,720
    // tokens, 40 heads of 128, frames and cap: 5.5 to 5.8 ms, the fp32 pipe 48% and the
    // tensor pipe 54% busy; 8,192 tokens, 12 heads of 64, clips: 211 us, of it 25 us the other
    // launches and 20 us the uneven ends of 768 items on 152 SMs; a stage takes there as
    // long as its chain S, 64 columns per warp, P V. Four warps with a running maximum
    // took 381 us there, two S buffers and two of P 220.
    const int grp = warp >> 3, hh = (warp >> 2) & 1, rw = warp & 3, t = (int)(threadIdx.x & 127);
    const uint32_t t_row = tmem + ((uint32_t)(rw * 32) << 16);
    float* part = reinterpret_cast<float*>(gbase + C::kOffEx);   // [4][128] parts of the row sums
    uint32_t it_use = 0, o_items = 0, stages_before = 0;         // stages of this CTA
    const int half = PAIR ? t >> 6 : 0;   // with pairs, rows 0-63 are query block 2p and rows 64-127 block 2p + 1
    auto arrive = [&](uint32_t bar_) {   // for the whole warp
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_);
    };
    for (;;) {
      const int ri = (int)(it_use % C::NI);
      if (!wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g)) break;
      const int64_t item = ring[ri].x;
      const int len = ring[ri].y;
      const int badbits = ring[ri].z;
      ++it_use;
      if (len < 0) {
        arrive(bar(I_EMPTY + ri));
        if (len == -2) break;
        continue;
      }
      const int64_t bh = item / nbp;
      const int i = PAIR ? 2 * (int)(item % nbp) + half : (int)(item % nb);   // this thread's query block
      const int o = PAIR ? t & 63 : t;                                        // its token in the block
      const int64_t row = bh * p.N + (int64_t)i * BT + o;
      bool stores = grp == 0 && i < nb && !((badbits >> half) & 1);
      int64_t orow_idx = row;
      if (p.raster && stores) orow_idx = p.rm.row(bh, i, o);
      if (stores) stores = dcheck(row < p.rows_total && orow_idx >= 0 && orow_idx < p.rows_total, p.d_status);
      uint4* orow = reinterpret_cast<uint4*>(p.o + orow_idx * D) + hh * (D / 16);   // this thread's half of the row
      if (len == 0) {
        if (stores) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) orow[c] = make_uint4(0, 0, 0, 0);
          if (hh == 0) p.lse[row] = -INFINITY;
        }
        arrive(bar(I_EMPTY + ri));
        continue;
      }
      const uint32_t* mk = masks + ri * C::kMaskWords;
      uint32_t ilo = 0u, ilen = 0u;      // this row's interval
      const int32_t* pos0 = p.mask.pos;
      RowGroups groups{};
      if (p.mask.pos != nullptr) {
        const int64_t tok0 = bh / p.rm.H * p.N;   // this batch element's first token
        pos0 += tok0 + lane;
        if (i < nb) {
          ilo = (uint32_t)__ldg(p.mask.lo + tok0 + (int64_t)i * BT + o);
          ilen = __ldg(p.mask.len + tok0 + (int64_t)i * BT + o);
        }
        groups.make(ilo, ilen, lane);
      }
      UnionSeek seek(bits + ri * 2 * C::MAXW, bits + ri * 2 * C::MAXW + C::MAXW, PAIR ? words : 0);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t any = 0u;   // this row has seen a key
      bool ok = true;
      for (int e = (grp ^ (int)(stages_before & 1u)); e < len; e += 2) {
        // did the row block select this half's key block, does the mask cut it, and the
        // columns this row sees then
        bool has = true, cut;
        if constexpr (PAIR) {
          const uint32_t code = reinterpret_cast<const uint8_t*>(mk)[e] >> (4 * hh + half);   // bit 0: selected; 2: cut
          has = code & 1u;
          cut = has && ((code >> 2) & 1u);
        } else {
          cut = (mk[e >> 5] >> (e & 31)) & 1u;
        }
        uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;
        if (cut) {
          const int64_t j = PAIR ? seek.at(2 * e + hh) : __ldg(p.col_idx + p.row_ptr[item] + e);
          const int32_t* kp = pos0 + j * BT + (PAIR ? 0 : 64 * hh);
          query_bits(groups, ilo, ilen, __ldg(kp), __ldg(kp + 32), lane, see0, see1);
        }
        const uint32_t n = stages_before + (uint32_t)e, buf = n % 3u;   // stage of the CTA, its buffer
        const uint32_t tS = t_row + C::kColS + buf * 128u + hh * 64u;   // this warp's scores, and its P over them
        if (!(ok = wait_warp(bar(C::B_S + buf), (n / 3u) & 1u, g))) break;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const uint32_t w = c == 0 ? see0 : see1;
          uint32_t pk[16];
          // columns no row of the warp sees (or of a block the row block did not select)
          if (!has || !__any_sync(0xffffffffu, w != 0u)) {
#pragma unroll
            for (int x = 0; x < 16; ++x) pk[x] = 0u;
            tmem_st16(tS + 16u * c, pk);
            continue;
          }
          uint32_t s[32];
          float most = 0.f;   // the largest score of this row's chunk
          if constexpr (MOD == 2) most = tmem_ld32_most(tS + 32u * c, s);
          else tmem_ld32(tS + 32u * c, s);
          wait_ld();
          any |= w;
          auto probs = [&](auto form_c, auto cut_c) {   // form of the cap: near, within, any, none, any and large
            constexpr int FORM = decltype(form_c)::value;
            constexpr bool CUT = decltype(cut_c)::value;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float s0 = __uint_as_float(s[2 * x]), s1 = __uint_as_float(s[2 * x + 1]);
              float y0, y1;
              if constexpr (FORM == 0) {
                near_cap_x2(p.near, s0, s1, -p.c0, y0, y1);
              } else if constexpr (FORM == 1) {
                tanh_poly_x2(s0, s1, p.inv_cap, y0, y1);
                fma_x2(y0, y1, p.cap2, -p.c0, y0, y1);
              } else if constexpr (FORM == 2) {
                y0 = cap_exp(s0 * p.c1, p.cap2) - p.c0;
                y1 = cap_exp(s1 * p.c1, p.cap2) - p.c0;
              } else if constexpr (FORM == 4) {
                y0 = fmaf(tanh_any(s0 * p.inv_cap, s0 * p.c1), p.cap2, -p.c0);
                y1 = fmaf(tanh_any(s1 * p.inv_cap, s1 * p.c1), p.cap2, -p.c0);
              } else {
                mul_x2(s0, s1, p.scale_log2, p.scale_log2, y0, y1);
              }
              float p0 = ex2f(y0), p1 = ex2f(y1);
              if constexpr (CUT) {
                if (!((w >> (2 * x)) & 1u)) p0 = 0.f;
                if (!((w >> (2 * x + 1)) & 1u)) p1 = 0.f;
              }
              add_x2(sum[x & 1].x, sum[x & 1].y, p0, p1);
              pk[x] = pack2(p0, p1);
            }
          };
          using std::integral_constant;
          if constexpr (MOD == 1) {
            if (cut) probs(integral_constant<int, 3>{}, std::true_type{});
            else probs(integral_constant<int, 3>{}, std::false_type{});
          } else {
            // the largest score of the warp's chunk says which form of the cap holds
            if (__all_sync(0xffffffffu, most <= p.near.limit)) {
              if (cut) probs(integral_constant<int, 0>{}, std::true_type{});
              else probs(integral_constant<int, 0>{}, std::false_type{});
            } else if (__all_sync(0xffffffffu, most * p.inv_cap <= 1.f)) {
              probs(integral_constant<int, 1>{}, std::true_type{});
            } else if (p.exp_cap) {
              probs(integral_constant<int, 2>{}, std::true_type{});
            } else {
              probs(integral_constant<int, 4>{}, std::true_type{});
            }
          }
          tmem_st16(tS + 16u * c, pk);
        }
        wait_st();
        fence_before();
        arrive(bar(C::B_P + buf));
      }
      if (!ok) break;
      arrive(bar(I_EMPTY + ri));
      stages_before += (uint32_t)len;
      float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (any != 0u && l < 1.2e-38f) l = 1.2e-38f;   // 0 is for a row that has seen no key; NaN stays NaN
      if (!wait_warp(bar(EXCH + 4 + rw), (o_items & 1u) ^ 1u, g)) break;   // the last item's parts were read
      part[(2 * grp + hh) * 128 + t] = l;
      arrive(bar(EXCH + rw));
      if (grp == 1) {
        ++o_items;
        continue;
      }
      if (!wait_warp(bar(EXCH + rw), o_items & 1u, g)) break;
      l = (part[t] + part[128 + t]) + (part[256 + t] + part[384 + t]);
      arrive(bar(EXCH + 4 + rw));
      if (!wait_warp(bar(O_FULL), o_items & 1u, g)) break;
      ++o_items;
      fence_after();
      const float inv = l > 0.f ? 1.0f / l : 0.f;   // 0: the row saw no key
      // (NaN compares false: such a row goes to the general kernel as well)
      bool good = p.fix_items == nullptr || l == 0.f || (l > 8.7e-19f && l < 1.2e24f);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t ov[32];
        tmem_ld32(t_row + C::kColO + hh * (D / 2) + c * 32u, ov);
        wait_ld();
        if (p.fix_items != nullptr) {
          // sums of products beyond fp32 of both signs are infinite here, not NaN (measured); a maximum
          // that passes NaN on does not rest on that
          float top[2] = {0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 32; x += 2)
            top[(x >> 1) & 1] = max_nan(max_nan(top[(x >> 1) & 1], fabsf(__uint_as_float(ov[x]))),
                                        fabsf(__uint_as_float(ov[x + 1])));
          const float most = max_nan(top[0], top[1]);
          // A small sum may belong to probabilities whose products with small values leave fp32 at
          // the lower end: 2^19 products lost below 2^-126 are 2^-17 of a largest sum of 2^-90, and, with a
          // row sum above 2^-20 (scores above -14), 2^-87 in O.
          good = good && most < INFINITY && (l == 0.f || l > 9.6e-7f || most > 8.1e-28f);
        }
        if (!stores) continue;
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x)
          w[x] = pack2(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
#pragma unroll
        for (int x = 0; x < 4; ++x) orow[c * 4 + x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
      }
      fence_before();
      arrive(bar(O_EMPTY));
      if (stores && hh == 0) p.lse[row] = l == 0.f ? -INFINITY : (p.c0 + log2f(l)) * 0.69314718055994531f;   // NaN of NaN
      // one entry per item however many of its warps ask for it
      if (p.fix_items != nullptr && __any_sync(0xffffffffu, stores && !good) && lane == 0 &&
          atomicExch(&p.fix_mark[item], 1) == 0)
        p.fix_items[atomicAdd(p.fix_count, 1)] = (int32_t)item;
    }
  } else if constexpr (MOD != 0) {
    if constexpr (C::DUO) regs_increase<C::kRegSoftmax>();
    // ------------------------------------------------------------ softmax + epilogue of any scores with a mask or a cap
    const uint32_t t_row = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t it_use = 0, s_use = 0, o_items = 0;
    uint64_t blocks_done = 0;
    const float sl2 = p.scale_log2;
    const int half = PAIR ? (int)(threadIdx.x >> 6) : 0;   // rows 0-63: query block 2p, rows 64-127: block 2p + 1
    bool ok = true;
    auto arrive = [&](uint32_t bar_) {   // for the whole warp
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_);
    };
    for (;;) {
      const int ri = (int)(it_use % C::NI);
      if (!wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g)) break;
      const int64_t item = ring[ri].x;
      const int len = ring[ri].y;
      const int badbits = ring[ri].z;
      // the item's masks are read until it ends; release the slot then
      auto release = [&]() { arrive(bar(I_EMPTY + ri)); };
      ++it_use;
      if (len < 0) {
        release();
        if (len == -2) break;
        continue;
      }
      const int64_t bh = item / nbp;
      const int i = PAIR ? 2 * (int)(item % nbp) + half : (int)(item % nb);   // this thread's query block
      const int o = PAIR ? (int)(threadIdx.x & 63) : (int)threadIdx.x;       // its token in the block
      const int64_t row = bh * p.N + (int64_t)i * BT + o;
      bool stores = i < nb && !((badbits >> half) & 1);
      int64_t orow_idx = row;
      if (p.raster && stores) orow_idx = p.rm.row(bh, i, o);
      if (stores) stores = dcheck(row < p.rows_total && orow_idx >= 0 && orow_idx < p.rows_total, p.d_status);
      uint4* orow = reinterpret_cast<uint4*>(p.o + orow_idx * D);
      if (len == 0) {
        if (stores) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0, 0, 0, 0);
          p.lse[row] = -INFINITY;
        }
        release();
        continue;
      }
      const uint32_t* mk = masks + ri * C::kMaskWords;
      // this row's interval, and of the next stage which halves the row block selected,
      // which of them the mask cuts, and there the positions of this lane's columns
      uint32_t ilo = 0u, ilen = 0u;
      const int32_t* pos0 = p.mask.pos;
      int32_t kpos[4];
      bool has1 = true, has2 = true, cut1 = false, cut2 = false;
      RowGroups groups{};
      UnionSeek seek(bits + ri * 2 * C::MAXW, bits + ri * 2 * C::MAXW + C::MAXW, PAIR ? words : 0);
      auto next = [&](int e) {
        if constexpr (PAIR) {
          const uint32_t code = reinterpret_cast<const uint8_t*>(mk)[e] >> half;   // bits 0, 4: selected; 2, 6: cut
          has1 = code & 1u;
          has2 = (code >> 4) & 1u;
          cut1 = has1 && ((code >> 2) & 1u);
          cut2 = has2 && ((code >> 6) & 1u);
        } else {
          has1 = has2 = true;
          cut1 = cut2 = (mk[e >> 5] >> (e & 31)) & 1u;
        }
        if (!cut1 && !cut2) return;
        int64_t j1, j2;
        if constexpr (PAIR) {
          j1 = seek.at(2 * e);
          j2 = cut2 ? seek.at(2 * e + 1) : j1;
        } else {
          j1 = j2 = __ldg(p.col_idx + p.row_ptr[item] + e);
        }
        kpos[0] = __ldg(pos0 + j1 * BT);
        kpos[1] = __ldg(pos0 + j1 * BT + 32);
        kpos[2] = __ldg(pos0 + j2 * BT + (PAIR ? 0 : 64));
        kpos[3] = __ldg(pos0 + j2 * BT + (PAIR ? 32 : 96));
      };
      if (p.mask.pos != nullptr) {
        const int64_t tok0 = bh / p.rm.H * p.N;   // this batch element's first token
        pos0 += tok0 + lane;
        if (i < nb) {
          ilo = (uint32_t)__ldg(p.mask.lo + tok0 + (int64_t)i * BT + o);
          ilen = __ldg(p.mask.len + tok0 + (int64_t)i * BT + o);
        }
        groups.make(ilo, ilen, lane);
      }
      next(0);
      float m = -INFINITY, l = 0.f;
      // O *= f; O must not change under the PV of block g - 1 (g = global block index)
      auto rescale = [&](uint64_t gb, float f) -> bool {
        const uint64_t gp = gb - 1;
        if (!wait_warp(bar(PV_DONE + (uint32_t)(gp % C::NPB)), (uint32_t)((gp / C::NPB) & 1u), g)) return false;
        fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(t_row + C::kColO + c * 32u, ov);
          wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * f);
          tmem_st32(t_row + C::kColO + c * 32u, ov);
        }
        return true;
      };
      for (int e = 0; e < len; ++e) {
        const uint32_t b = s_use % C::NSB;
        const uint64_t gb = blocks_done + e;
        // A stage goes half by half through TMEM in a loop that is not unrolled, against
        // the maximum of the stages before; when that is outgrown by more than the
        // threshold it starts over with the stage's own.
        auto stage_mod = [&]() -> bool {
          // bit c of see[w]: this row sees column 32 w + c; a half that no row of the
          // warp sees counts as not selected
          uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
          if (cut1) {
            query_bits(groups, ilo, ilen, kpos[0], kpos[1], lane, see[0], see[1]);
            has1 = __any_sync(0xffffffffu, (see[0] | see[1]) != 0u);
          }
          if (cut2) {
            query_bits(groups, ilo, ilen, kpos[2], kpos[3], lane, see[2], see[3]);
            has2 = __any_sync(0xffffffffu, (see[2] | see[3]) != 0u);
          }
          if (!wait_warp(bar(S_FULL + b), (s_use / C::NSB) & 1u, g)) return false;
          fence_after();
          if (gb >= (uint64_t)C::NPB) {
            if (!wait_warp(bar(PV_DONE + b), (uint32_t)(((gb - C::NPB) / C::NPB) & 1u), g)) return false;
            fence_after();
          }
          // a half's scores (masked ones -inf) and their maximum in log2 units, capped
          uint32_t s[64];
          auto load_half = [&](int hh) -> float {
            const uint32_t ts = t_row + C::kColS + b * 128u + hh * 64u;
            tmem_ld32(ts, s);
            tmem_ld32(ts + 32u, s + 32);
            wait_ld();
            const uint32_t w0 = hh ? see[2] : see[0], w1 = hh ? see[3] : see[1];
            float mw[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const uint32_t w = c < 32 ? w0 : w1;
              if (MOD == 3) {   // -inf stands for a masked score below; one that is seen is -cap
                s[c] = __float_as_uint(max_nan(__uint_as_float(s[c]), -3.402823466e38f));
                s[c + 1] = __float_as_uint(max_nan(__uint_as_float(s[c + 1]), -3.402823466e38f));
              }
              if (!((w >> (c & 31)) & 1u)) s[c] = 0xff800000u;
              if (!((w >> ((c + 1) & 31)) & 1u)) s[c + 1] = 0xff800000u;
              mw[(c >> 1) & 1] = fmaxf(fmaxf(mw[(c >> 1) & 1], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
            }
            const float mx = fmaxf(mw[0], mw[1]);
            if (MOD != 3) return mx * sl2;
            return mx == -INFINITY ? mx : tanh_any(mx * p.inv_cap, mx * p.c1) * p.cap2;
          };
          bool known = false, resc = false;
          float f = 1.f;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int hh = 0; hh < 2;) {
            uint32_t pk[32];
            if (!(hh == 0 ? has1 : has2)) {
#pragma unroll
              for (int c = 0; c < 32; ++c) pk[c] = 0u;
              tmem_st32(t_row + C::kColP + b * 64u + 32u * hh, pk);
              ++hh;
              continue;
            }
            const float mx = load_half(hh);
            if (!known && __any_sync(0xffffffffu, mx > m + kRescaleThreshold)) {
              float m_new = fmaxf(m, mx);
              if (hh == 0 ? has2 : has1) m_new = fmaxf(m_new, load_half(hh ^ 1));
              known = true;
              resc = e > 0;
              f = m_new == -INFINITY ? 1.f : ex2f(m - m_new);
              m = m_new;
              sum[0] = sum[1] = make_float2(0.f, 0.f);
              hh = 0;
              continue;
            }
            // a row that has seen no key yet: every exponent is -inf against 0
            const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float s0 = __uint_as_float(s[2 * c]), s1 = __uint_as_float(s[2 * c + 1]);
              float x0, x1;
              if constexpr (MOD != 3) {
                fma_x2(s0, s1, sl2, -mr, x0, x1);
              } else {   // the cap would bring a masked score back
                x0 = s0 == -INFINITY ? s0 : fmaf(tanh_any(s0 * p.inv_cap, s0 * p.c1), p.cap2, -mr);
                x1 = s1 == -INFINITY ? s1 : fmaf(tanh_any(s1 * p.inv_cap, s1 * p.c1), p.cap2, -mr);
              }
              const float p0 = ex2f(x0), p1 = ex2f(x1);
              add_x2(sum[c & 1].x, sum[c & 1].y, p0, p1);
              pk[c] = pack2(p0, p1);
            }
            tmem_st32(t_row + C::kColP + b * 64u + 32u * hh, pk);
            ++hh;
          }
          fence_before();
          arrive(bar(S_FREE + b));
          ++s_use;
          if (resc) {
            if (!rescale(gb, f)) return false;
            l *= f;
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          return true;
        };
        if (!(ok = stage_mod())) break;
        wait_st();
        fence_before();
        arrive(bar(P_FULL + b));
        if (e + 1 < len) next(e + 1);
      }
      release();
      if (!ok) break;
      blocks_done += (uint64_t)len;
      if (!(ok = wait_warp(bar(O_FULL), o_items & 1u, g))) break;
      ++o_items;
      fence_after();
      const float inv = l > 0.f ? 1.0f / l : 0.f;   // 0: the row saw no key
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(t_row + C::kColO + c * 32u, ov);
        wait_ld();
        if (!stores) continue;
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x)
          w[x] = pack2(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
#pragma unroll
        for (int x = 0; x < 4; ++x) orow[c * 4 + x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
      }
      fence_before();
      arrive(bar(O_EMPTY));
      if (stores) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;   // NaN of NaN
    }
  } else {
    if constexpr (C::DUO) regs_increase<C::kRegSoftmax>();
    {
    // ------------------------------------------------------------ softmax + epilogue
      const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
      const uint32_t t_row = tmem + lane_base;
      uint32_t it_use = 0, s_use = 0, o_items = 0;
      uint64_t blocks_done = 0;
      const float sl2 = p.scale_log2;
      // with pairs, rows 0-63 are query block 2p and rows 64-127 block 2p + 1
      const int half = PAIR ? (int)(threadIdx.x >> 6) : 0;
      bool ok = true;
      for (;;) {
        const int ri = (int)(it_use % C::NI);
        if (!wait_warp(bar(I_FULL + ri), (it_use / C::NI) & 1u, g)) break;
        const int64_t item = ring[ri].x;
        const int len = ring[ri].y;
        const int badbits = ring[ri].z;
        __syncwarp();
        // pairs read the item's bitmaps until the item ends; release the slot then
        auto release = [&]() {
          if (lane == 0) mbar_arrive(bar(I_EMPTY + ri));
        };
        if (!PAIR) release();
        ++it_use;
        if (len == -2) {
          if (PAIR) release();
          break;
        }
        if (len == -1) {
          if (PAIR) release();
          continue;
        }
        const int64_t bh = item / nbp;
        const int i = PAIR ? 2 * (int)(item % nbp) + half : (int)(item % nb);   // this thread's query block
        const int o = PAIR ? (int)(threadIdx.x & 63) : (int)threadIdx.x;       // its token in the block
        const int64_t row = bh * p.N + (int64_t)i * BT + o;
        // rows past the block (or past the last block of a pair) are computed, never stored
        bool stores = o < BT && i < nb && !((badbits >> half) & 1);
        int64_t orow_idx = row;
        if (p.raster && stores) orow_idx = p.rm.row(bh, i, o);
        if (stores) stores = dcheck(row < p.rows_total && orow_idx >= 0 && orow_idx < p.rows_total, p.d_status);
        uint4* orow = reinterpret_cast<uint4*>(p.o + orow_idx * D);
        if (len == 0) {
          if (stores) {
  #pragma unroll
            for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0, 0, 0, 0);
            p.lse[row] = -INFINITY;
          }
          if (PAIR) release();
          continue;
        }
        const uint32_t* mk = masks + ri * C::kMaskWords;
        float m = -INFINITY, l = 0.f;
        for (int e = 0; e < len; ++e) {
          // which halves of this stage's 128 columns this row attends to (warp-uniform)
          bool has1 = true, has2 = true;
          if constexpr (PAIR && C::MASK_BYTES) {
            const uint32_t st = reinterpret_cast<const uint16_t*>(mk)[e];   // bytes 2e, 2e + 1
            has1 = (st >> half) & 1u;
            has2 = (st >> (8 + half)) & 1u;
          } else if constexpr (PAIR) {
            const uint32_t nib = mk[e >> 3] >> (4 * (e & 7));   // stage e's two blocks, two rows
            has1 = (nib >> half) & 1u;
            has2 = (nib >> (2 + half)) & 1u;
          }
          const uint32_t b = s_use % C::NSB;
          if (!(ok = wait_warp(bar(S_FULL + b), (s_use / C::NSB) & 1u, g))) break;
          fence_after();
          {
          uint32_t s[C::KR];
          float cm[C::KR / 32];   // the maximum of each 32-column load (exact, as any order of max)
  #pragma unroll
          for (int c = 0; c < C::KR / 32; ++c)
            cm[c] = tmem_ld32_max(t_row + C::kColS + b * 128u + c * 32u, s + 32 * c);
          wait_ld();
          fence_before();
          mbar_arrive(bar(S_FREE + b));
          ++s_use;
          if (!has1) cm[0] = cm[1] = -INFINITY;
          if (!has2) cm[2] = cm[3] = -INFINITY;
          float mx = cm[0];
  #pragma unroll
          for (int c = 1; c < C::KR / 32; ++c) mx = fmaxf(mx, cm[c]);
          const float m_new = fmaxf(m, mx * sl2);
          // a rescale of O (by f) is applied after P is written, when the S row is
          // no longer held in registers
          bool resc = false;
          float f = 1.f;
          if (e == 0) {
            m = m_new;
          } else if (__any_sync(0xffffffffu, m_new > m + kRescaleThreshold)) {
            resc = true;
            f = ex2f(m - m_new);
            m = m_new;
          }
          uint32_t pk[C::KR / 2];
          float rs[8];
  #pragma unroll
          for (int u = 0; u < 8; ++u) rs[u] = 0.f;
  #pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            // columns [64*hh, 64*hh + 64): one key block of a pair (both halves of
            // one block otherwise)
            if (hh == 0 ? has1 : has2) {
              // two columns per instruction for the scale-and-subtract and the sums
              // (packed fp32 pairs: eight running sums, even and odd columns)
  #pragma unroll
              for (int c = 32 * hh; c < 32 * hh + 32; ++c) {
                float x0, x1;
                fma_x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]), sl2, -m, x0, x1);
                const float p0 = ex2f(x0), p1 = ex2f(x1);
                add_x2(rs[2 * (c & 3)], rs[2 * (c & 3) + 1], p0, p1);
                pk[c] = pack2(p0, p1);
              }
            } else {
  #pragma unroll
              for (int c = 32 * hh; c < 32 * hh + 32; ++c) pk[c] = 0u;
            }
          }
          // P buffer b was last read by the PV of block g - NPB
          const uint64_t gb = blocks_done + e;
          if (gb >= (uint64_t)C::NPB) {
            if (!(ok = wait_warp(bar(PV_DONE + b), (uint32_t)(((gb - C::NPB) / C::NPB) & 1u), g))) break;
            fence_after();
          }
  #pragma unroll
          for (int c = 0; c < C::KR / 64; ++c) tmem_st32(t_row + C::kColP + b * 64u + 32u * c, pk + 32 * c);
          if (resc) {
            // O must not change under the PV of block g-1 (g = global block index)
            const uint64_t gp = gb - 1;
            if (!(ok = wait_warp(bar(PV_DONE + (uint32_t)(gp % C::NPB)), (uint32_t)((gp / C::NPB) & 1u), g))) break;
            fence_after();
  #pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32(t_row + C::kColO + c * 32u, ov);
              wait_ld();
  #pragma unroll
              for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * f);
              tmem_st32(t_row + C::kColO + c * 32u, ov);
            }
            l *= f;
          }
          l += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
          wait_st();
          fence_before();
          mbar_arrive(bar(P_FULL + b));
          }
        }
        if (PAIR) release();
        if (!ok) break;
        blocks_done += (uint64_t)len;
        if (!(ok = wait_warp(bar(O_FULL), o_items & 1u, g))) break;
        ++o_items;
        fence_after();
        // a row that attended to no key (its block's own row is empty in a pair) has l = 0
        const float inv = l > 0.f ? 1.0f / l : 0.f;
  #pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(t_row + C::kColO + c * 32u, ov);
          wait_ld();
          if (!stores) continue;
          uint32_t w[16];
  #pragma unroll
          for (int x = 0; x < 16; ++x)
            w[x] = pack2(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
  #pragma unroll
          for (int x = 0; x < 4; ++x) orow[c * 4 + x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        }
        fence_before();
        mbar_arrive(bar(O_EMPTY));
        if (stores) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == C::W_S) tmem_dealloc(tmem, C::kTmemCols);
  if (p.prof != nullptr && threadIdx.x == 0)
    atomicAdd((unsigned long long*)&p.prof[smid() % SPARSP_PROF_SLOTS],
              (unsigned long long)(globaltimer_ns() - t_start));
}

template <int BT, int D, int MOD>
sparsp_status_t go_fwd(const Dims& s, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const Params& prm, cudaStream_t st) {
  using C = Cfg<BT, D, MOD>;
  auto kern = attn_fwd_tc_kernel<BT, D, MOD>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  // all of the SM's memory as shared memory: one CTA of ~225 KB, or two of ~100 KB
  if (cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    return SPARSP_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return SPARSP_ERR_CUDA;
  const int64_t grid = cap_grid(s, (int64_t)sms * C::kMinCtas, prm.n_items);
  kern<<<(unsigned)grid, C::THREADS, C::kSmemBytes, st>>>(tq, tk, tv, prm);
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

template <int MOD>
sparsp_status_t launch_fwd_mod(const Dims& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                               const __nv_bfloat16* v, const int32_t* row_ptr, const int32_t* col_idx, float scale,
                               __nv_bfloat16* o, float* lse, bool raster, bool in_raster, const int32_t* items,
                               int32_t* counter, uint64_t* prof, int32_t* d_status, const MaskView& mask, float cap,
                               const FixList& fix, cudaStream_t st) {
  const uint64_t rows = (uint64_t)s.B * s.H * s.N;
  CUtensorMap tq, tk, tv;
  if (in_raster) {
    // raster inputs: one block per 5-D box (two boxes for a pair's query tile)
    if (!make_tmap_bf16_raster(&tq, q, s) || !make_tmap_bf16_raster(&tk, k, s) || !make_tmap_bf16_raster(&tv, v, s))
      return SPARSP_ERR_CUDA;
  } else if (MOD == 1 || MOD == 2) {   // the loader's: all columns of 128 query rows, or of one block
    const uint32_t kv_boxes = s.Bt == 64 ? 1 : (uint32_t)s.d / 64;   // pairs' blocks alternate by column box
    if (!make_tmap_bf16_boxes(&tq, q, rows, (uint64_t)s.d, 128, (uint32_t)s.d / 64) ||
        !make_tmap_bf16_boxes(&tk, k, rows, (uint64_t)s.d, (uint32_t)s.Bt, kv_boxes) ||
        !make_tmap_bf16_boxes(&tv, v, rows, (uint64_t)s.d, (uint32_t)s.Bt, kv_boxes))
      return SPARSP_ERR_CUDA;
  } else if (!make_tmap_bf16_rows(&tq, q, rows, (uint64_t)s.d, 128) ||   // Q boxes: the MMA's 128 rows
             !make_tmap_bf16_rows(&tk, k, rows, (uint64_t)s.d, (uint32_t)s.Bt) ||   // K, V: one block
             !make_tmap_bf16_rows(&tv, v, rows, (uint64_t)s.d, (uint32_t)s.Bt)) {
    return SPARSP_ERR_CUDA;
  }
  // 64-token blocks: items are pairs of query blocks, ordered by the caller
  // over the pair rows (attn_fwd_tc_items)
  const int nbp = attn_fwd_tc_items_per_head(s);
  constexpr float kLog2e = 1.4426950408889634f;
  Params prm{row_ptr, col_idx, s.N, s.nb, nbp, (int64_t)s.B * s.H * nbp, (int64_t)rows, scale * kLog2e, o, lse,
             raster ? 1 : 0, raster_map(s), in_raster ? 1 : 0, raster_box(s), items, counter, prof, d_status,
             mask, MOD == 2 || MOD == 3 ? 2.f * scale * kLog2e / cap : 0.f, cap * kLog2e,
             MOD == 2 || MOD == 3 ? scale / cap : 0.f,
             MOD == 2 ? near_cap(scale, cap) : NearCap{}, cap <= kExpCap,
             MOD == 2 && cap <= kFixedCap ? fmaxf(cap * kLog2e - 20.f, 0.f) : 0.f, fix.items, fix.count, fix.mark};
  if (s.Bt == 128 && s.d == 128) return go_fwd<128, 128, MOD>(s, tq, tk, tv, prm, st);
  if (s.Bt == 128 && s.d == 64) return go_fwd<128, 64, MOD>(s, tq, tk, tv, prm, st);
  if (s.Bt == 64 && s.d == 128) return go_fwd<64, 128, MOD>(s, tq, tk, tv, prm, st);
  if (s.Bt == 64 && s.d == 64) return go_fwd<64, 64, MOD>(s, tq, tk, tv, prm, st);
  return SPARSP_ERR_UNSUPPORTED;
}

}  // namespace

}  // namespace sparsp
