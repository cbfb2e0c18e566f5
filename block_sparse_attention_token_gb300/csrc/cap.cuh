// The score cap y = cap tanh(x), x = scale s / cap, in log2 units (cap2 = cap
// log2 e), for the tcgen05 attention kernels. By its definition a score costs an
// exponential and a reciprocal beside the softmax's exponential, all three on one unit;
// polynomials put it on the fp32 pipe, two scores per instruction.
// Which form holds is decided per warp and 32 columns by the largest score there (forward
// of 30,720 tokens, 40 heads of 128, frames, cap 30: 5.7 ms with all scores within 0.6 of the
// cap, 6.9 ms with some beyond, 8.1 ms with most beyond the cap).
#pragma once

#include <math.h>

#include "tc_helpers.cuh"

namespace sparsp {
namespace tc {

__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) / x on |x| <= 1 as a polynomial of degree 6 in x^2: least squares on
// Chebyshev points, reweighted until the largest relative error is flat
// (Lawson's iteration); 5e-8 in exact arithmetic, 1.7e-7 evaluated in fp32.
// Seven multiply-adds, against an exponential and a reciprocal on the unit that
// already has the softmax's exponentials to do.
__device__ constexpr float tanh_coef(int k) {
  return k == 0   ? 0.9999999403953552f
         : k == 1 ? -0.33332839608192444f
         : k == 2 ? 0.13325203955173492f
         : k == 3 ? -0.05345702916383743f
         : k == 4 ? 0.020289979875087738f
         : k == 5 ? -0.006203378085047007f
                  : 0.001041022245772183f;
}

// tanh of a pair of scores, x = s inv_cap, by the polynomial
__device__ __forceinline__ void tanh_poly_x2(float s0, float s1, float inv_cap, float& t0, float& t1) {
  float x0, x1, u0, u1, q0, q1;
  mul_x2(s0, s1, inv_cap, inv_cap, x0, x1);
  mul_x2(x0, x1, x0, x1, u0, u1);
  fma_x2(u0, u1, tanh_coef(6), tanh_coef(5), q0, q1);
#pragma unroll
  for (int k = 4; k >= 0; --k) fma2_x2(q0, q1, u0, u1, tanh_coef(k), q0, q1);
  mul_x2(x0, x1, q0, q1, t0, t1);
}
// cap2 tanh by its definition, t = 2 x log2(e): 1 - 2 / (1 + exp(2 x)), for any x. Good to
// a few 2^-24 of the cap, in small scores too, and so used up to kExpCap only.
constexpr float kExpCap = 256.0f;
__device__ __forceinline__ float cap_exp(float t, float cap2) {
  return fmaf(rcpf(1.f + exp2_approx(t)), -2.f * cap2, cap2);
}
// tanh for any x and any cap: by the polynomial where |x| <= 1, else by its definition
// (in place of cap_exp at every cap: 1.14 ms against 0.51 for the forward of 8,192 tokens
// in 64-token blocks, scores beyond the cap).
__device__ __forceinline__ float tanh_any(float x, float t) {
  const float u = x * x;
  float q = tanh_coef(6);
#pragma unroll
  for (int k = 5; k >= 0; --k) q = fmaf(q, u, tanh_coef(k));
  return fabsf(x) <= 1.f ? x * q : fmaf(rcpf(1.f + exp2_approx(t)), -2.f, 1.f);
}

// Where all |x| <= kNearCap a polynomial of degree 4 in s^2 does (the same fit, 1.7e-7
// evaluated in fp32), with the powers of scale / cap and the factor cap2 folded into
// its coefficients: six multiply-adds from the score to y. `limit` is the largest
// |s| it is for; all is 0 where the folded coefficients would leave fp32's range.
constexpr float kNearCap = 0.6f;
struct NearCap {
  float c[5];
  float limit;
};
inline NearCap near_cap(double scale, double cap) {
  NearCap n{};
  const double a = scale / cap;
  if (!(a >= 1.0 / 16384 && a <= 16384.0)) return n;
  const double t[5] = {0.9999999403953552, -0.33332309126853943, 0.13310173153877258, -0.05210147798061371,
                       0.01547542680054903};
  double f = cap * 1.4426950408889634 * a;
  for (int k = 0; k < 5; ++k, f *= a * a) {
    n.c[k] = (float)(t[k] * f);
    if (isinf(n.c[k])) return NearCap{};   // a chunk of zeros is within any limit, and 0 times infinity is not 0
  }
  n.limit = (float)(kNearCap / a);
  return n;
}
// The backward rounds everything it makes of tanh to bf16: degree 3 (2.3e-6) will do
// there, and tanh itself is what it needs twice (c[4] is not used). The error counts
// times the score in the exponent, so that above a cap of 100 (where it could pass
// 2e-4) the fit is that of |x| <= 0.25 (5e-9). Its largest coefficient is 0.05 * 16384^7.
inline NearCap near_cap_backward(double scale, double cap) {
  NearCap n{};
  const double a = scale / cap;
  if (!(a >= 1.0 / 16384 && a <= 16384.0)) return n;
  const double wide[4] = {0.9999978542327881, -0.33314040303230286, 0.13057856261730194, -0.04092942178249359};
  const double narrow[4] = {1.0, -0.3333320617675781, 0.13323132693767548, -0.051327724009752274};
  const bool large = cap > 100.0;
  double f = a;
  for (int k = 0; k < 4; ++k, f *= a * a) n.c[k] = (float)((large ? narrow : wide)[k] * f);
  n.limit = (float)((large ? 0.25 : (double)kNearCap) / a);
  return n;
}
// tanh of a pair of scores from the backward's coefficients
__device__ __forceinline__ void near_tanh_x2(const NearCap& n, float s0, float s1, float& t0, float& t1) {
  float u0, u1, q0, q1;
  mul_x2(s0, s1, s0, s1, u0, u1);
  fma_x2(u0, u1, n.c[3], n.c[2], q0, q1);
  fma2_x2(q0, q1, u0, u1, n.c[1], q0, q1);
  fma2_x2(q0, q1, u0, u1, n.c[0], q0, q1);
  mul_x2(s0, s1, q0, q1, t0, t1);
}
// y + add of a pair of scores
__device__ __forceinline__ void near_cap_x2(const NearCap& n, float s0, float s1, float add, float& y0, float& y1) {
  float u0, u1, q0, q1;
  mul_x2(s0, s1, s0, s1, u0, u1);
  fma_x2(u0, u1, n.c[4], n.c[3], q0, q1);
#pragma unroll
  for (int k = 2; k >= 0; --k) fma2_x2(q0, q1, u0, u1, n.c[k], q0, q1);
  fma2_x2(s0, s1, q0, q1, add, y0, y1);
}

}  // namespace tc
}  // namespace sparsp
