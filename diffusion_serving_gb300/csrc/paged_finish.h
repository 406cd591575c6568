// States of the paged attentions: O (unnormalised), the running maximum m in the exp2 domain and the
// sum l of a query row's weights over some of its keys.  States over disjoint keys join as
//   O = sum_c 2^(m_c - M) O_c,  L = sum_c 2^(m_c - M) l_c,  M = max_c m_c.
#pragma once

#include "paged_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

__device__ __forceinline__ float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void pg_store4(float* p, const float4& x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void pg_store4(__half* p, const float4& x) {
  const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void pg_store4(__nv_bfloat16* p, const float4& x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void pg_acc4(float4& a, float w, const float4& x) {
  a.x = fmaf(w, x.x, a.x);
  a.y = fmaf(w, x.y, a.y);
  a.z = fmaf(w, x.z, a.z);
  a.w = fmaf(w, x.w, a.w);
}
// weight of a part with maximum m against M (M finite wherever a part has keys)
__device__ __forceinline__ float pg_weight(float m, float M) { return m == -INFINITY ? 0.f : pg_ex2(m - M); }

// Joins `n` states into (M, L, x), eight loads in flight: get(i, &ml, &o) gives state i's (m, l) and four dims of O.
template <typename Get>
__device__ __forceinline__ void pg_join(int n, float& M, float& L, float4& x, Get get) {
  for (int i0 = 0; i0 < n; i0 += 8) {
    float2 ml[8];
    float4 y[8];
    float top = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < n) get(i0 + i, &ml[i], &y[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
    const float w0 = pg_weight(M, top);
    x.x *= w0, x.y *= w0, x.z *= w0, x.w *= w0;
    L *= w0;
    M = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = pg_weight(ml[i].x, M);
      L = fmaf(w, ml[i].y, L);
      if (w != 0.f) pg_acc4(x, w, y[i]);         // (a state without keys may hold anything)
    }
  }
}

// One more state.
__device__ __forceinline__ void pg_join1(float& M, float& L, float4& x, float2 ml, const float4& y) {
  const float top = fmaxf(M, ml.x);
  const float w0 = pg_weight(M, top), w = pg_weight(ml.x, top);
  x.x *= w0, x.y *= w0, x.z *= w0, x.w *= w0;
  L = fmaf(w, ml.y, L * w0);
  M = top;
  if (w != 0.f) pg_acc4(x, w, y);
}

// Partials of R rows: slot i of a buffer, row r.  What the tensor-core kernel leaves of rows' own slots (`by8`) has 8 dims of
// all rows together, whoever joins it: that kernel, with a row to a thread, or k_paged_join; its stores, and its own loads, are then
// whole lines (1302 tokens over 8000 slots, 40 heads: 155 us, and 180 with a row's dims together).  All others have a row's dims
// together: a shared prefix's, which k_paged_join_prefix reads with a warp to a row (4096 slots, 8 rows: 28.0 us, and 33.6 with
// 8 dims together), and the streaming and FMA kernels'.
template <int R, int D, bool by8 = false>
__device__ __forceinline__ void pg_load_part(const float* buf, int64_t i, int r, int d, float2* ml, float4* y) {
  const float* p = buf + i * (int64_t)(R * (D + 2));
  *ml = __ldcg(reinterpret_cast<const float2*>(p + R * D + 2 * r));
  *y = __ldcg(reinterpret_cast<const float4*>(p + (by8 ? ((d >> 3) * R + r) * 8 + (d & 7) : r * D + d)));
}

// Four dims d .. d + 3 of one token and head, from its joined state.
template <typename T, int D>
__device__ __forceinline__ void pg_emit(const kvc_pg_args& a, T* out, int64_t at, int d, float M, float L, const float4& x) {
  const float inv = L != 0.f ? 1.f / L : 0.f;          // no visible slot: out 0 (a NaN goes on)
  pg_store4(out + at * D + d, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  if (d == 0 && a.lse != nullptr) a.lse[at] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// What the end of an item needs to know of it.
struct kvc_pg_end {
  int rows;              // real query rows
  int c0, c1;            // the blocks it spans
  int slot;              // where this block leaves its state, if it does
  bool left;             // it does: the item spans blocks, or phase 1 leaves it for kvc_pg_launch_join_prefix
};
template <int R, int TS, bool kW>
__device__ __forceinline__ kvc_pg_end pg_end(const kvc_pg_args& a, const kvc_pg_sched<R, TS, kW>& sch, const kvc_pg_item& it) {
  kvc_pg_end e;
  e.rows = min(sch.T, it.r.n - it.k * sch.T) * a.Gv;
  sch.span(it, &e.c0, &e.c1);
  e.left = a.phase == 1 || e.c0 != e.c1;
  // phase 1: item + block (item and block borders only move forward, so no two collide); else the block's second
  // slot for the item that begins in it, its first for one that goes on
  e.slot = a.phase == 1 ? it.vh * ((it.r.n + sch.T - 1) / sch.T) + it.k + (int)blockIdx.x
                        : 2 * (int)blockIdx.x + ((int)blockIdx.x == e.c0 ? 1 : 0);
  return e;
}
// Row of the outputs [n_tokens * H] for query row r of an item.
template <int R, int TS, bool kW>
__device__ __forceinline__ int64_t pg_at(const kvc_pg_args& a, const kvc_pg_sched<R, TS, kW>& sch, const kvc_pg_item& it, int r) {
  const int i = r / a.Gv;
  return (int64_t)(it.r.t0 + it.k * sch.T + i) * a.H + it.vh * a.Gv + r - i * a.Gv;
}

// The end of an item: this block's state own(r, d, &M, &L) -> O's four dims, for the item's real rows, goes straight
// out to row at(r), or is left as a partial.  The block that leaves last joins the partials, in their order on the
// line whichever block it is, so the result does not depend on timing.  Behind a shared prefix, pre(r, d, &ml, &o) is
// the prefix's state.
// `threads` threads call it (tid 0 .. threads - 1); bar() separates them; s_flag is an int they share.
template <typename T, int D, int R, typename Own, typename Pre, typename At, typename Bar>
__device__ __forceinline__ void pg_finish(const kvc_pg_args& a, const kvc_pg_end& e, T* out, int* s_flag, int tid,
                                          int threads, bool prefix, Own own, Pre pre, At at, Bar bar) {
  float* mine = (a.phase == 1 ? a.pre : a.part) + (int64_t)e.slot * (R * (D + 2));
  for (int v = tid; v < e.rows * (D / 4); v += threads) {
    const int r = v / (D / 4), d = 4 * (v % (D / 4));
    float M, L;
    float4 x = own(r, d, &M, &L);
    if (e.left) {
      *reinterpret_cast<float4*>(mine + r * D + d) = x;
      if (d == 0) *reinterpret_cast<float2*>(mine + R * D + 2 * r) = make_float2(M, L);
      continue;
    }
    if (prefix) {
      float2 ml;
      float4 y;
      pre(r, d, &ml, &y);
      pg_join1(M, L, x, ml, y);
    }
    pg_emit<T, D>(a, out, at(r), d, M, L, x);
  }
  if (!e.left || a.phase == 1) return;
  // the partial's stores precede thread 0's release (barrier, then a cumulative release); the last block's loads
  // follow its acquire
  bar();
  if (tid == 0) {
    int prev;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + e.c0) : "memory");
    const int last = prev == e.c1 - e.c0;
    if (last) a.tickets[e.c0] = 0;     // every block of the item is past it
    *s_flag = last;
  }
  bar();
  if (!*s_flag) return;
  for (int v = tid; v < e.rows * (D / 4); v += threads) {
    const int r = v / (D / 4), d = 4 * (v % (D / 4));
    float M = -INFINITY, L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (prefix) {
      float2 ml;
      float4 y;
      pre(r, d, &ml, &y);
      pg_join1(M, L, x, ml, y);
    }
    pg_join(e.c1 - e.c0 + 1, M, L, x,
            [&](int i, float2* ml, float4* y) { pg_load_part<R, D>(a.part, 2 * (e.c0 + i) + (i == 0 ? 1 : 0), r, d, ml, y); });
    pg_emit<T, D>(a, out, at(r), d, M, L, x);
  }
}
// The state that a shared prefix left for one token and head (in global memory).
template <int D>
__device__ __forceinline__ void pg_load_prefix(const kvc_pg_args& a, int64_t at, int d, float2* ml, float4* y) {
  *ml = __ldcg(a.pre_ml + at);
  *y = __ldcg(reinterpret_cast<const float4*>(a.pre_o + at * D + d));
}
