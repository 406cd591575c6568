// Internal declarations of the 4-bit paged store (include/kvc_paged4.h).
#pragma once

#include "../../include/kvc_paged4.h"
#include "paged_internal.h"

struct kvc_paged4 {
  kvc_paged_config cfg;
  int ps_log2;
  int sub, Gv, Hv;      // as kvc_paged's
  float scale;
  uint8_t* pages;
  const int32_t* table;
  const int32_t* kv_len;
  uint8_t* ws;
  int device;
  uint64_t debug_stall_ns;
};

// Workspace, in bytes from its start.
struct kvc_pg4_layout {
  size_t tickets;       // int32 per block: blocks that have left their part of a split item
  size_t warp_tickets;  // the same per softmax warp of the tensor-core kernel
  size_t zeroed;        // end of what has to start at zero (and is left at zero)
  size_t parts;         // split partials
  size_t total;
};

// Bytes of a record: a page's slots of one kv head.
__host__ __device__ inline int64_t kvc_pg4_record(int D, int ps_log2) { return (int64_t)(D + D / 16) << ps_log2; }

cudaError_t kvc_pg4_launch_append(kvc_paged4* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                                  int64_t q_stride, void* q_out, int n_tokens, const int32_t* cu, const float* rope,
                                  int rope_positions, const kvc_rope_axes* axes, const int32_t* positions, bool half,
                                  cudaStream_t s);
cudaError_t kvc_pg4_launch_read(kvc_paged4* c, void* k_out, void* v_out, int n_tokens, const int32_t* cu, cudaStream_t s);
cudaError_t kvc_pg4_launch_decode(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s);
cudaError_t kvc_pg4_launch_tc(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s);
// Shared-memory opt-ins of the kernels a handle may launch, once per handle.
cudaError_t kvc_pg4_prepare_decode(const kvc_paged4* c);
cudaError_t kvc_pg4_prepare_tc(const kvc_paged4* c);

#ifdef __CUDACC__
#include <cuda_fp16.h>
#include <cuda_bf16.h>

// Held values are (c - 8) s.  A code moved into a mantissa reads 64 + c (fp16, under an exponent of 64) or 128 + c (bf16), and
// one fused multiply-add makes it (64 + c) s - 72 s: 72 s has 8 significant bits at most, 136 s too (17 times four bits), and the
// result 7, so all of it is exact in either 16-bit type.
template <typename T>
struct kvc_pg4_type;
template <>
struct kvc_pg4_type<__half> {
  static constexpr uint32_t kMask = 0x00F000F0u, kBase = 0x54005400u, kOff = 0xD480D480u;    // 64, -72
  static constexpr int kAt = 4;
};
template <>
struct kvc_pg4_type<__nv_bfloat16> {
  static constexpr uint32_t kMask = 0x000F000Fu, kBase = 0x43004300u, kOff = 0xC308C308u;    // 128, -136
  static constexpr int kAt = 0;
};

// What a pair of values is made with: s and -72 s (-136 s).
struct kvc_pg4_scale {
  uint32_t s, o;
};
__device__ __forceinline__ uint32_t pg4_mul(uint32_t a, uint32_t b, const __half*) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pg4_mul(uint32_t a, uint32_t b, const __nv_bfloat16*) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pg4_fma(uint32_t a, uint32_t b, uint32_t c, const __half*) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pg4_fma(uint32_t a, uint32_t b, uint32_t c, const __nv_bfloat16*) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Two e4m3 (low byte, high byte) as a pair of T (exact).
__device__ __forceinline__ uint32_t pg4_e4m3x2(uint32_t two, const __half*) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}
__device__ __forceinline__ uint32_t pg4_e4m3x2(uint32_t two, const __nv_bfloat16*) {
  const uint32_t h = pg4_e4m3x2(two, (const __half*)nullptr);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(f.y), "f"(f.x));
  return d;
}
template <typename T>
__device__ __forceinline__ kvc_pg4_scale pg4_scale(uint32_t s) {
  return {s, pg4_mul(s, kvc_pg4_type<T>::kOff, (const T*)nullptr)};
}
// Pair i of a word of codes (dims 2 i and 2 i + 1 of the word's eight).  `base`: kBase, in a register (a constant known to the
// compiler would cost a second logic operation: an instruction takes one immediate).
template <typename T, int i>
__device__ __forceinline__ uint32_t pg4_pair(uint32_t word, const kvc_pg4_scale& sc, uint32_t base) {
  constexpr int kDown = 4 * i - kvc_pg4_type<T>::kAt;
  const uint32_t x = ((kDown < 0 ? word << (kDown < 0 ? -kDown : 0) : word >> (kDown > 0 ? kDown : 0)) & kvc_pg4_type<T>::kMask) | base;
  return pg4_fma(x, sc.s, sc.o, (const T*)nullptr);
}

// The same as fp16 at fewer instructions, up to a power of 2: codes 0 and 1 of each half stand in the mantissa's bits 0 .. 3 and
// 4 .. 7 as they are, codes 2 and 3 once the word is shifted by 8; under an exponent of 64 they read 64 + c / 16 and 64 + c.
// So pairs 0 and 2 come out as (c - 8) s / 16, pairs 1 and 3 as (c - 8) s, and whoever multiplies makes up for it.  64.5 s and
// 72 s have 11 significant bits at most (129 times four bits; 9 times four), so all of it is exact.
struct kvc_pg4_fast_scale {
  uint32_t s, o0, o1;     // s, -64.5 s, -72 s
};
__device__ __forceinline__ kvc_pg4_fast_scale pg4_fast_scale(uint32_t two_e4m3) {
  const __half* t = nullptr;
  const uint32_t s = pg4_e4m3x2(two_e4m3, t);
  return {s, pg4_mul(s, 0xD408D408u, t), pg4_mul(s, 0xD480D480u, t)};
}
// `sixty_four`: kvc_pg4_type<__half>::kBase, in a register (as pg4_pair's).  d[i]: dims 2 i and 2 i + 1 (of K), or the ith codes of the word's halves.
__device__ __forceinline__ void pg4_fast_pairs(uint32_t word, const kvc_pg4_fast_scale& sc, uint32_t sixty_four, uint32_t* d) {
  const __half* t = nullptr;
  const uint32_t b = word >> 8;
  d[0] = pg4_fma((word & 0x000F000Fu) | sixty_four, sc.s, sc.o0, t);
  d[1] = pg4_fma((word & 0x00F000F0u) | sixty_four, sc.s, sc.o1, t);
  d[2] = pg4_fma((b & 0x000F000Fu) | sixty_four, sc.s, sc.o0, t);
  d[3] = pg4_fma((b & 0x00F000F0u) | sixty_four, sc.s, sc.o1, t);
}

// ---- queries for such pairs ----
// A row of queries as fp16, times a power of 2 that brings its largest element to 2^10 .. 2^11, and 16 times that at the dims of
// pairs 0 and 2, whose keys come out too small.  Elements are exact down to 2^-25 of the largest, and below it off by 2^-36 of
// it at most; held magnitudes span less than 2^21, so a score is off by less than 2^-15 of the sum of its terms' magnitudes, at
// queries and keys made for it.  (A row whose largest element is below 2^-110 is brought up by 2^120 and no more.)
__device__ __forceinline__ uint32_t pg4_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 pg4_floats(uint32_t w, const __half*) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ float2 pg4_floats(uint32_t w, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ float pg4_query_top(const uint4& v, float top) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pg4_floats(w[i], (const T*)nullptr);
    top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
  }
  return top;
}
// The factor of a row whose largest magnitude is `top`, and what undoes it.  (An infinity stays one; both are within fp32's range.)
__device__ __forceinline__ float pg4_query_factor(float top, float* undo) {
  const int e = (int)(__float_as_uint(top) >> 23) - 127;       // top is 2^e .. 2^(e + 1)
  const int up = e == 128 ? 0 : min(10 - e, 120);
  *undo = __uint_as_float((uint32_t)(127 - up) << 23);
  return __uint_as_float((uint32_t)(127 + up) << 23);
}
// What takes a row's scores to log2 units.  (Never 0, which would make NaN of a masked score: a scale that is less than fp32's normal
// range leaves scores, 2^31 at most, that no weight shows.)
__device__ __forceinline__ float pg4_score_scale(float undo, float scale_log2) { return fmaxf(undo * scale_log2, 0x1p-126f); }
template <typename T>
__device__ __forceinline__ void pg4_query_vec(uint4& v, float f) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pg4_floats(w[i], (const T*)nullptr);
    const float y = i & 1 ? f : 16.f * f;
    w[i] = pg4_pack(x.x * y, x.y * y);
  }
}
#endif  // __CUDACC__
