// Token masks of attention: the plan (tile order and block ranges), block
// scores without the pairs nobody sees, and the CSR without them. All three
// read a few bytes per block pair or token and are bound by latency: 4 us the plan of
// 1,024 tokens, about 10 us the CSR's count, scan and fill (8,192 tokens, 12 heads, where
// they save attention 30 us).
#include "mask.cuh"

namespace sparsp {
namespace {

// One warp per block: its tokens in tile order, and the block's ranges.
__global__ void __launch_bounds__(256)
mask_plan_kernel(const int32_t* __restrict__ pos, const int32_t* __restrict__ lo, const int32_t* __restrict__ hi,
                 const RasterMap rm, int Bt, int nb, int64_t blocks, int32_t* __restrict__ opos,
                 int32_t* __restrict__ olo, uint32_t* __restrict__ olen, int2* __restrict__ krange,
                 int2* __restrict__ qrange, int2* __restrict__ qhull) {
  const int64_t blk = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (blk >= blocks) return;
  const int64_t b = blk / nb;
  const int j = (int)(blk % nb);
  int kmin = INT32_MAX, kmax = INT32_MIN, lomax = INT32_MIN, himin = INT32_MAX, lomin = INT32_MAX, himax = INT32_MIN;
  for (int o = lane; o < Bt; o += 32) {
    // the raster row of a one-head tensor is the token's index
    const RasterMap r1{rm.N, 1, rm.Y, rm.X, rm.ta, rm.tb, rm.tc, rm.nY, rm.nX};
    const int64_t n = r1.row(b, j, o), at = b * rm.N + (int64_t)j * Bt + o;
    const int32_t p = pos[n], l = lo[n], h = hi[n];
    opos[at] = p;
    olo[at] = l;
    olen[at] = h > l ? (uint32_t)h - (uint32_t)l : 0u;
    kmin = min(kmin, p);
    kmax = max(kmax, p);
    lomax = max(lomax, l);
    himin = min(himin, h);
    if (h > l) {
      lomin = min(lomin, l);
      himax = max(himax, h);
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  lomax = __reduce_max_sync(0xffffffffu, lomax);
  himin = __reduce_min_sync(0xffffffffu, himin);
  lomin = __reduce_min_sync(0xffffffffu, lomin);
  himax = __reduce_max_sync(0xffffffffu, himax);
  if (lane == 0) {
    krange[blk] = make_int2(kmin, kmax);
    qrange[blk] = make_int2(lomax, himin);
    qhull[blk] = make_int2(lomin, himax);
  }
}

__global__ void __launch_bounds__(256)
mask_scores_kernel(const MaskView m, int H, int nb, float* __restrict__ scores) {
  const int64_t row = blockIdx.x;                 // (b*H + h)*nb + i
  const int64_t b = row / ((int64_t)H * nb);
  const int2 q = m.qhull[b * nb + row % nb];
  for (int j = threadIdx.x; j < nb; j += blockDim.x)
    if (!blocks_meet(q, m.krange[b * nb + j])) scores[row * nb + j] = SPARSP_MASKED_SCORE;
}

// One warp per CSR row. FILL = false counts the kept blocks (a malformed row
// keeps none), FILL = true writes them at out_ptr[row] in their order.
template <bool FILL>
__global__ void __launch_bounds__(256)
mask_csr_kernel(const MaskView m, int H, int nb, int64_t rows, const int32_t* __restrict__ row_ptr,
                const int32_t* __restrict__ col_idx, int32_t* __restrict__ out_ptr, int32_t* __restrict__ out_idx,
                int32_t* d_status) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int32_t a = row_ptr[row], e1 = row_ptr[row + 1];
  bool bad = e1 < a || (int64_t)e1 - a > nb;
  const int64_t b = row / ((int64_t)H * nb);
  const int2 q = m.qhull[b * nb + row % nb];
  int kept = 0;
  const int32_t at = FILL ? out_ptr[row] : 0;
  if (FILL && out_ptr[row + 1] == at) return;   // nothing kept, or malformed
  for (int32_t e = a; e < e1 && !bad; e += 32) {
    const bool in = e + lane < e1;
    const int32_t j = in ? col_idx[e + lane] : 0;
    bad = __any_sync(0xffffffffu, j < 0 || j >= nb);
    if (bad) break;
    const bool keep = in && blocks_meet(q, m.krange[b * nb + j]);
    const unsigned vote = __ballot_sync(0xffffffffu, keep);
    if (FILL && keep) out_idx[at + kept + __popc(vote & ((1u << lane) - 1u))] = j;
    kept += __popc(vote);
  }
  if (!FILL && lane == 0) {
    if (bad) report(d_status, SPARSP_ERR_DATA);
    out_ptr[row] = bad ? 0 : kept;
  }
}

// The work order of a small problem in one CTA: items (rows, or pairs of rows of a
// head) by their number of blocks, the longest first, equal ones in any order (the
// results do not depend on it); the pull counter and `n_zero` further words are
// cleared. A counting sort in shared memory; the lanes of a warp with equal costs count
// together, as one counter hit by all items one by one takes longer than the sort
// (ranks by comparing all pairs of 768 items: 15 us more).
constexpr int kOrderThreads = 1024, kOrderMaxBlocks = 1024, kOrderItems = 4096;
__global__ void __launch_bounds__(kOrderThreads)
order_items_kernel(const int32_t* __restrict__ row_ptr, int nb, int per_head, int n, int32_t* __restrict__ items,
                   int32_t* __restrict__ counter, int32_t* __restrict__ zero, int n_zero) {
  __shared__ int32_t place[2 * kOrderMaxBlocks + 1];   // items per cost, then the next slot of each
  __shared__ int32_t warp_sum[32];
  const int t = threadIdx.x, lane = t & 31, top = 2 * nb, step = per_head == nb ? 1 : 2;
  // adds the warp's items to their costs' counters; an item's place among them
  auto take = [&](int item, int32_t& c) {
    c = -1;
    if (item < n) {
      const int h = item / per_head, r = (item - h * per_head) * step;
      c = row_ptr[(int64_t)h * nb + min(r + step, nb)] - row_ptr[(int64_t)h * nb + r];
      c = min(max(c, 0), top);
    }
    const unsigned same = __match_any_sync(0xffffffffu, c);
    const int lead = __ffs(same) - 1;
    int32_t at = 0;
    if (lane == lead && c >= 0) at = atomicAdd(&place[c], __popc(same));
    return __shfl_sync(0xffffffffu, at, lead) + __popc(same & ((1u << lane) - 1u));
  };
  for (int c = t; c <= top; c += kOrderThreads) place[c] = 0;
  for (int i = t; i < n_zero; i += kOrderThreads) zero[i] = 0;
  if (t == 0) *counter = 0;
  __syncthreads();
  int32_t c;
  for (int i = t; i - lane < n; i += kOrderThreads) take(i, c);
  __syncthreads();
  // items with a larger cost: each thread some costs from the top down, then over the threads
  constexpr int kPer = (2 * kOrderMaxBlocks + kOrderThreads) / kOrderThreads;
  int32_t mine[kPer], sum = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int k = top - (t * kPer + u);
    mine[u] = k >= 0 ? place[k] : 0;
    sum += mine[u];
  }
  int32_t incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sum[t >> 5] = incl;
  __syncthreads();
  int32_t run = incl - sum;
  for (int w = 0; w < (t >> 5); ++w) run += warp_sum[w];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int k = top - (t * kPer + u);
    if (k >= 0) place[k] = run;
    run += mine[u];
  }
  __syncthreads();
  for (int i = t; i - lane < n; i += kOrderThreads) {
    const int32_t slot = take(i, c);
    if (i < n) items[slot] = i;
  }
}

}  // namespace

bool order_items_fits(const Dims& s, int per_head, bool uneven) {
  const int64_t n = (int64_t)s.B * s.H * per_head, kv_bytes = (int64_t)s.B * s.H * s.N * s.d * s.elem * 2;
  if (s.nb > kOrderMaxBlocks || n > kOrderItems) return false;
  return n <= device_sm_count() || (uneven && kv_bytes <= (int64_t)64 << 20);
}

sparsp_status_t launch_order_items(const Dims& s, int per_head, const int32_t* row_ptr, int32_t* items,
                                   int32_t* counter, int32_t* zero, int n_zero, cudaStream_t st) {
  order_items_kernel<<<1, kOrderThreads, 0, st>>>(row_ptr, s.nb, per_head, s.B * s.H * per_head, items, counter, zero,
                                                  n_zero);
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_mask_plan(const Dims& s, const int32_t* pos, const int32_t* lo, const int32_t* hi, void* plan,
                                 cudaStream_t st) {
  const MaskPlan l = mask_plan_layout(s);
  uint8_t* p = (uint8_t*)plan;
  const int64_t blocks = (int64_t)s.B * s.nb;
  mask_plan_kernel<<<(unsigned)((blocks + 7) / 8), 256, 0, st>>>(
      pos, lo, hi, raster_map(s), s.Bt, s.nb, blocks, (int32_t*)(p + l.pos), (int32_t*)(p + l.lo),
      (uint32_t*)(p + l.len), (int2*)(p + l.krange), (int2*)(p + l.qrange), (int2*)(p + l.qhull));
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_mask_scores(const Dims& s, const MaskView& m, float* scores, cudaStream_t st) {
  mask_scores_kernel<<<(unsigned)s.rows(), 256, 0, st>>>(m, s.H, s.nb, scores);
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

sparsp_status_t launch_mask_csr(const Dims& s, const MaskView& m, const int32_t* row_ptr, const int32_t* col_idx,
                                int32_t* out_ptr, int32_t* out_idx, int32_t* d_status, cudaStream_t st) {
  const unsigned grid = (unsigned)((s.rows() + 7) / 8);
  mask_csr_kernel<false><<<grid, 256, 0, st>>>(m, s.H, s.nb, s.rows(), row_ptr, col_idx, out_ptr, nullptr, d_status);
  SPARSP_LAUNCH_CHECK();
  const sparsp_status_t r = launch_scan_counts(out_ptr, s.rows(), st);
  if (r != SPARSP_OK) return r;
  mask_csr_kernel<true><<<grid, 256, 0, st>>>(m, s.H, s.nb, s.rows(), row_ptr, col_idx, out_ptr, out_idx, d_status);
  SPARSP_LAUNCH_CHECK();
  return SPARSP_OK;
}

}  // namespace sparsp
