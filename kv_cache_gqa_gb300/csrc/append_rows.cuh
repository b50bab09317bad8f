// Steps of a q or K row that the quantising and the paged append share: the rotation's angles and products of pairs.  (Their
// norms differ: the quantising one's sum is strided over a copy in shared memory, the paged one's is over the lanes' registers.)
#pragma once

#include "common.cuh"

namespace kva {
namespace {

// cos and sin of the angle p * inv (inv = ih + il) in float32, off by at most 3.5e-8 (half an ulp below 1 is
// 3.0e-8; 1 in 400 is not the correctly rounded value).  For |p| < 2^20 the angle is a pair of floats, brought
// to r = rh + rl about within pi/4 by subtracting k pi/2 in three parts (Cody and Waite); the series of
// cos and sin carry their first terms as pairs (Dekker's sums and products), the rest, below 0.016, in
// float32.  Larger positions take float64 up to the reduced angle, whose product p * inv is rounded first:
// up to 1.2e-7 more near 2^31.
__device__ __forceinline__ void rotation(int32_t p, float ih, float il, double inv, float* c, float* s) {
  float rh, rl;
  int k;
  if (p > -(1 << 20) && p < (1 << 20)) {
    const float pf = (float)p, hi = __fmul_rn(pf, ih);
    const float lo = fmaf(pf, il, fmaf(pf, ih, -hi));
    const float kf = rintf(hi * 0.636619772f);
    k = (int)kf;
    constexpr float A = 1.570796012878418f, B = 3.1391647e-07f, C = 5.390303e-15f;   // pi/2 = A + B + C; A has 22 bits
    const float t = fmaf(-kf, A, hi);                      // exact
    const float d = __fmul_rn(kf, B), de = fmaf(kf, B, -d);
    const float u = __fsub_rn(t, d), z = __fsub_rn(u, t);  // u + ue = t - d
    const float ue = __fsub_rn(__fsub_rn(t, __fsub_rn(u, z)), __fadd_rn(d, z));
    const float e = __fadd_rn(__fsub_rn(ue, de), fmaf(-kf, C, lo));
    rh = __fadd_rn(u, e);
    rl = __fadd_rn(__fsub_rn(u, rh), e);
  } else {
    const double a = (double)p * inv, kd = rint(a * 0.63661977236758134);
    const double r = fma(-kd, 6.123233995736766e-17, fma(-kd, 1.5707963267948966, a));
    k = (int)((int64_t)kd & 3);
    rh = (float)r;
    rl = (float)(r - (double)rh);
  }
  const float uh = __fmul_rn(rh, rh), ul = fmaf(2.0f * rh, rl, fmaf(rh, rh, -uh));     // r^2
  // cos r = 1 - r^2/2 + r^4 (1/24 - r^2/720 + ...)
  const float pc = fmaf(fmaf(fmaf(-2.75573192e-7f, uh, 2.48015873e-5f), uh, -1.38888889e-3f), uh, 4.16666667e-2f);
  const float h = 0.5f * uh, w = __fsub_rn(1.0f, h), we = __fsub_rn(__fsub_rn(1.0f, w), h);
  const float co = __fadd_rn(w, fmaf(__fmul_rn(uh, uh), pc, fmaf(-0.5f, ul, we)));
  // sin r = r - r^3/6 + r^5 (1/120 - r^2/5040 + ...)
  const float ps = fmaf(fmaf(fmaf(-2.50521084e-8f, uh, 2.75573192e-6f), uh, -1.98412698e-4f), uh, 8.33333333e-3f);
  const float vh = __fmul_rn(uh, rh), vl = fmaf(ul, rh, fmaf(uh, rl, fmaf(uh, rh, -vh)));   // r^3
  constexpr float SIXTH = 1.0f / 6.0f, SIXTH_REST = -4.9670538e-9f;
  const float th = __fmul_rn(vh, SIXTH), tl = fmaf(vh, SIXTH_REST, fmaf(vl, SIXTH, fmaf(vh, SIXTH, -th)));
  const float y = __fsub_rn(rh, th), ye = __fsub_rn(__fsub_rn(rh, y), th);
  const float si = __fadd_rn(y, fmaf(__fmul_rn(vh, uh), ps, __fadd_rn(__fsub_rn(ye, tl), rl)));
  const float a = k & 1 ? si : co, b = k & 1 ? co : si;
  *c = (k + 1) & 2 ? -a : a;
  *s = k & 2 ? -b : b;
}

// a b + c d of both elements, products and sum rounded apart
__device__ __forceinline__ uint64_t sum_of_products(uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  return pack_f32x2(__fadd_rn(__fmul_rn(f32x2_lo(a), f32x2_lo(b)), __fmul_rn(f32x2_lo(c), f32x2_lo(d))),
                    __fadd_rn(__fmul_rn(f32x2_hi(a), f32x2_hi(b)), __fmul_rn(f32x2_hi(c), f32x2_hi(d))));
}
__device__ __forceinline__ void unpack_pairs(const uint64_t (&x)[4], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) { y[2 * i] = f32x2_lo(x[i]); y[2 * i + 1] = f32x2_hi(x[i]); }
}
// 4 pairs of shared memory
__device__ __forceinline__ void shared_pairs(const float* p, uint64_t (&x)[4]) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

}  // namespace
}  // namespace kva
