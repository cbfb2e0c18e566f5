// The tcgen05 backward over the selected blocks alone (attn_bwd_tc.cuh).
#include "attn_bwd_tc.cuh"

namespace sparsp {

bool attn_bwd_tc_supported(const Dims& s) {
  if (s.d != 128 && s.d != 64) return false;
  // 64-token blocks run as pairs; an item slot holds the pair's two lists as bitmaps
  if (s.Bt == 64 && s.nb > 32 * (s.d == 64 ? BCfg<64, 64>::MAXW : BCfg<128, 64>::MAXW)) return false;
  return (s.Bt == 128 || s.Bt == 64) && attn_fwd_tc_supported(s);
}

int attn_bwd_tc_items_per_head(const Dims& s) { return s.Bt == 64 ? (s.nb + 1) / 2 : s.nb; }

sparsp_status_t launch_attn_bwd_tc(const Dims& s, int mode, const __nv_bfloat16* q,
                                   const __nv_bfloat16* k, const __nv_bfloat16* v,
                                   const __nv_bfloat16* dout, const float* lse2,
                                   const float* delta, const int32_t* ptr, const int32_t* idx,
                                   float scale, __nv_bfloat16* out, __nv_bfloat16* out2,
                                   const int32_t* items, int32_t* counter, uint64_t* prof, int32_t* d_status,
                                   bool raster, cudaStream_t st) {
  return launch_bwd_mod<0>(s, mode, q, k, v, dout, lse2, delta, ptr, idx, scale, out, out2, items, counter, prof,
                           d_status, raster, MaskView{}, 0.f, st);
}

}  // namespace sparsp
