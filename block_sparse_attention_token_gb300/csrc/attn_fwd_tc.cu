// The tcgen05 forward over the selected blocks alone (attn_fwd_tc.cuh).
#include "attn_fwd_tc.cuh"

namespace sparsp {

int attn_fwd_tc_items_per_head(const Dims& s) { return s.Bt == 64 ? (s.nb + 1) / 2 : s.nb; }

bool attn_fwd_tc_supported(const Dims& s) {
  if (s.dtype != SPARSP_BF16 || (s.Bt != 64 && s.Bt != 128) || (s.d != 64 && s.d != 128)) return false;
  if (s.Bt == 64 && s.nb > 32 * (s.d == 64 ? Cfg<64, 64>::MAXW : Cfg<64, 128>::MAXW)) return false;
  if ((int64_t)s.B * s.H * s.N >= (int64_t)1 << 31) return false;
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return false;
  return major == 10;
}

sparsp_status_t launch_attn_fwd_tc(const Dims& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                   const __nv_bfloat16* v, const int32_t* row_ptr,
                                   const int32_t* col_idx, float scale, __nv_bfloat16* o,
                                   float* lse, bool raster, bool in_raster, const int32_t* items,
                                   int32_t* counter, uint64_t* prof, int32_t* d_status, cudaStream_t st) {
  return launch_fwd_mod<0>(s, q, k, v, row_ptr, col_idx, scale, o, lse, raster, in_raster, items, counter, prof,
                           d_status, MaskView{}, 0.f, FixList{}, st);
}

}  // namespace sparsp
