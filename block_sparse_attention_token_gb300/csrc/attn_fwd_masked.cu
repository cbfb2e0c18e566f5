// The tcgen05 forward with a token mask and, in a variant of its own, a score
// cap (attn_fwd_tc.cuh).
#include "attn_fwd_tc.cuh"

namespace sparsp {

sparsp_status_t launch_attn_fwd_masked(const Dims& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                       const __nv_bfloat16* v, const int32_t* row_ptr, const int32_t* col_idx,
                                       float scale, float cap, const MaskView& mask, __nv_bfloat16* o, float* lse,
                                       bool raster, bool in_raster, const int32_t* items, int32_t* counter,
                                       uint64_t* prof, int32_t* d_status, cudaStream_t st) {
  if (cap > kFixedCap)
    return launch_fwd_mod<3>(s, q, k, v, row_ptr, col_idx, scale, o, lse, raster, in_raster, items, counter, prof,
                             d_status, mask, cap, st);
  if (cap > 0.f)
    return launch_fwd_mod<2>(s, q, k, v, row_ptr, col_idx, scale, o, lse, raster, in_raster, items, counter, prof,
                             d_status, mask, cap, st);
  return launch_fwd_mod<1>(s, q, k, v, row_ptr, col_idx, scale, o, lse, raster, in_raster, items, counter, prof,
                           d_status, mask, cap, st);
}

}  // namespace sparsp
