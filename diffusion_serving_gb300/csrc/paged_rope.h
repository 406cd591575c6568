// One component a b - c d of a rotated pair (a, c of the store type, b, d fp32 table entries), so
// that rounding the returned fp32 value to the store type gives the exact value rounded once to
// nearest-even (finite inputs).
//
// 16-bit stores.  In fp32: p = c d, its exact error e = fma(c, d, -p) (exact while |c d| >= 2^-100,
// or c or d zero), r = fma(a, b, -p), r2 = r - e.  With |p| <= 2^20 |r2| the error of r2 is at most
// 1.5 ulps, so r2 rounds as the exact value does unless it lies within 2 ulps of a rounding
// midpoint of the store type, which its low bits show.  The rest (less than one in 400 of N(0, 1)
// data) goes through fp64: both products are exact there, their difference is a rounded sum plus
// its exact rest (Knuth's TwoSum), and rounding that to odd in fp32 leaves one rounding to come.
// fp32 stores: both products and their errors, and the errors of the sums, in fp32; the result stands
// if moving the last of them by a bound on what is neglected does not change its rounding (all but
// some 2^-22 of the cases).  The rest goes through fp64, whose sum rounds right except on an fp32
// midpoint, where its own rest decides.  (fp64 for every element would take some twenty times as long
// as the copy.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

__device__ __forceinline__ double pg_two_prod_diff(float a, float b, float c, float d, double* rest) {
  const double x = (double)a * (double)b, y = -((double)c * (double)d);
  const double s = x + y, t = s - x;
  *rest = (x - (s - t)) + (y - t);
  return s;
}

__device__ __noinline__ float pg_rot_odd(float a, float b, float c, float d) {
  double rest;
  const double s = pg_two_prod_diff(a, b, c, d, &rest);
  const float t = __double2float_rz(s);
  uint32_t u = __float_as_uint(t);
  if ((double)t == s) {
    if (rest == 0.0) return t;                     // exact
    if ((rest > 0.0) != (s > 0.0)) u -= 1;         // the exact value lies just inside t
  }
  return __uint_as_float(u | 1u);
}

// r is more than 2 fp32 ulps from every midpoint of the type
__device__ __forceinline__ bool pg_clear(float r, const __nv_bfloat16*) {
  return (__float_as_uint(r) & 0xFFFFu) - 0x7FFEu > 4u;
}
__device__ __forceinline__ bool pg_clear(float r, const __half*) {
  const float m = fabsf(r);
  if (m >= 65536.f) return true;                   // rounds to infinity
  return m >= 0x1p-14f && (__float_as_uint(r) & 0x1FFFu) - 0x0FFEu > 4u;
}

template <typename T>
__device__ __forceinline__ float pg_rot(float a, float b, float c, float d, const T* type) {
  const float p = __fmul_rn(c, d);
  const float e = __fmaf_rn(c, d, -p);
  const float r2 = __fsub_rn(__fmaf_rn(a, b, -p), e);
  const float m = fabsf(p);
  const bool ok = ((m >= 0x1p-100f && m <= fabsf(r2) * 0x1p20f) || (m == 0.f && (c == 0.f || d == 0.f))) &&
                  pg_clear(r2, type);
  return ok ? r2 : pg_rot_odd(a, b, c, d);
}
__device__ __noinline__ float pg_rot_f32(float a, float b, float c, float d) {
  double rest;
  const double s = pg_two_prod_diff(a, b, c, d, &rest);
  const float f = __double2float_rn(s);
  if (rest == 0.0) return f;
  const float lo = __double2float_rd(s), hi = __double2float_ru(s);
  if (lo == hi) return f;
  const double up = isinf(hi) ? copysign(0x1p128, (double)hi) : (double)hi;
  const double down = isinf(lo) ? copysign(0x1p128, (double)lo) : (double)lo;
  if (s != 0.5 * (up + down)) return f;
  return rest > 0.0 ? hi : lo;
}
__device__ __forceinline__ float pg_two_sum(float x, float y, float* err) {
  const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
  *err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t));
  return s;
}
__device__ __forceinline__ float pg_rot(float a, float b, float c, float d, const float*) {
  const float p = __fmul_rn(a, b), ep = __fmaf_rn(a, b, -p);
  const float q = __fmul_rn(c, d), eq = __fmaf_rn(c, d, -q);
  float es, e;
  const float s = pg_two_sum(p, -q, &es);
  const float u = __fsub_rn(ep, eq);                  // a b - c d = s + es + u, but for u's rounding
  const float r = pg_two_sum(s, __fadd_rn(es, u), &e);
  const float slack = (fabsf(es) + fabsf(ep) + fabsf(eq)) * 0x1p-22f;   // bounds that and the sum's own rounding
  const float m = fminf(fabsf(p), fabsf(q));
  const bool ok = m >= 0x1p-100f && fabsf(r) >= 0x1p-100f && fabsf(r) <= 0x1p126f &&
                  __fadd_rn(r, __fadd_rn(e, slack)) == r && __fadd_rn(r, __fsub_rn(e, slack)) == r;
  return ok ? r : pg_rot_f32(a, b, c, d);
}
