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
// Shared-memory opt-ins of the kernels a handle may launch, once per handle.
cudaError_t kvc_pg4_prepare_decode(const kvc_paged4* c);

#ifdef __CUDACC__
#include <cuda_fp16.h>
#include <cuda_bf16.h>

// Held values are (c - 8) s.  A code moved into the mantissa of 16 reads 16 + c, and one fused multiply-add makes it
// (16 + c) s - 24 s: 24 s has 6 significant bits and the result 7 at most, so all of it is exact in either 16-bit type.
template <typename T>
struct kvc_pg4_type;
template <>
struct kvc_pg4_type<__half> {
  static constexpr uint32_t kMask = 0x03C003C0u, kSixteen = 0x4C004C00u;
  static constexpr int kAt = 6;         // the mantissa's top four bits
};
template <>
struct kvc_pg4_type<__nv_bfloat16> {
  static constexpr uint32_t kMask = 0x00780078u, kSixteen = 0x41804180u;
  static constexpr int kAt = 3;
};

// A scale pair for a pair of values: (s, -24 s) in T.
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
  constexpr uint32_t kM24 = sizeof(T) == 2 && kvc_pg4_type<T>::kAt == 6 ? 0xCE00CE00u : 0xC1C0C1C0u;
  return {s, pg4_mul(s, kM24, (const T*)nullptr)};
}
// Pair i of a word of codes (dims 2 i and 2 i + 1 of the word's eight).
template <typename T, int i>
__device__ __forceinline__ uint32_t pg4_pair(uint32_t word, const kvc_pg4_scale& sc) {
  using P = kvc_pg4_type<T>;
  constexpr int kUp = P::kAt - 4 * i;
  const uint32_t x = ((kUp >= 0 ? word << (kUp >= 0 ? kUp : 0) : word >> (kUp < 0 ? -kUp : 0)) & P::kMask) | P::kSixteen;
  return pg4_fma(x, sc.s, sc.o, (const T*)nullptr);
}

// Halves of held values as pairs of fp16, (c - 8) s / 2, at fewer instructions: a word shifted left by 2 has codes 0 and 1
// of each half in the mantissa's bits 2 .. 5 and 6 .. 9, one shifted right by 6 codes 2 and 3; under exponents of 128 and 8 they
// read 128 + c / 2 and 8 + c / 2.  132 s and 12 s have 9 and 6 significant bits; 132 s is finite where 264 s would not be.
struct kvc_pg4_half_scale {
  uint32_t s, lo, hi;     // s, -132 s, -12 s
};
__device__ __forceinline__ kvc_pg4_half_scale pg4_half_scale(uint32_t two_e4m3) {
  const __half* t = nullptr;
  const uint32_t s = pg4_e4m3x2(two_e4m3, t);
  return {s, pg4_mul(s, 0xD820D820u, t), pg4_mul(s, 0xCA00CA00u, t)};
}
// The four pairs of a word: d[i] is dims 2 i and 2 i + 1 (of K), or the ith codes of the word's halves.
__device__ __forceinline__ void pg4_half_pairs(uint32_t word, const kvc_pg4_half_scale& sc, uint32_t* d) {
  const __half* t = nullptr;
  const uint32_t a = word << 2, b = word >> 6;
  d[0] = pg4_fma((a & 0x003C003Cu) | 0x58005800u, sc.s, sc.lo, t);
  d[1] = pg4_fma((a & 0x03C003C0u) | 0x48004800u, sc.s, sc.hi, t);
  d[2] = pg4_fma((b & 0x003C003Cu) | 0x58005800u, sc.s, sc.lo, t);
  d[3] = pg4_fma((b & 0x03C003C0u) | 0x48004800u, sc.s, sc.hi, t);
}
#endif  // __CUDACC__
