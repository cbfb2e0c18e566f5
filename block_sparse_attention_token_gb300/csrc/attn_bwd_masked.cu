// The tcgen05 backward with the forward's token mask and score cap
// (attn_bwd_tc.cuh).
#include "attn_bwd_tc.cuh"

namespace sparsp {

sparsp_status_t launch_attn_bwd_masked(const Dims& s, int mode, const __nv_bfloat16* q,
                                   const __nv_bfloat16* k, const __nv_bfloat16* v,
                                   const __nv_bfloat16* dout, const float* lse2,
                                   const float* delta, const int32_t* ptr, const int32_t* idx,
                                   float scale, __nv_bfloat16* out, __nv_bfloat16* out2,
                                   const int32_t* items, int32_t* counter, uint64_t* prof, int32_t* d_status,
                                   bool raster, const MaskView& mask, float cap, cudaStream_t st) {
  if (cap > 0.f)
    return launch_bwd_mod<2>(s, mode, q, k, v, dout, lse2, delta, ptr, idx, scale, out, out2, items, counter, prof,
                             d_status, raster, mask, cap, st);
  return launch_bwd_mod<1>(s, mode, q, k, v, dout, lse2, delta, ptr, idx, scale, out, out2, items, counter, prof,
                           d_status, raster, mask, cap, st);
}

}  // namespace sparsp
