// How an item of the paged attentions ends: its block's state (O unnormalised, running max m in
// the exp2 domain, sum l) is written out at once, or left as a partial and joined by the block
// that leaves last, or left for the launch that attends what follows a shared prefix.
//   O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c,  M = max_c m_c,
// over the item's own parts and, behind a shared prefix, the prefix's.  The parts are added in
// their order on the line, whichever block does it, so the result does not depend on timing.
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

// One state: O rows of D floats, and (m, l) per row.
struct kvc_pg_state {
  const float* o;
  const float* ml;
};
// Slot `i` of a buffer of partials with R rows.
template <int R, int D>
__device__ __forceinline__ kvc_pg_state pg_part(const float* buf, int64_t i) {
  const float* p = buf + i * (int64_t)(R * (D + 2));
  return {p, p + R * D};
}

// `threads` threads (tid 0 .. threads - 1, all of a named set that bar() separates) end an item.
// own_o [R][D] and own_ml [R][2]: this block's state, in shared memory.  s_flag, s_row: shared scratch
// (one int; 2 R floats).  bar(): a barrier of the set.  rows: the item's real rows.
template <typename T, int D, int R, int TS, typename Bar>
__device__ __forceinline__ void pg_finish(const kvc_pg_args& a, const kvc_pg_sched<R, TS>& sch, const kvc_pg_item& it,
                                          const float* own_o, const float* own_ml, T* out, int* s_flag, float* s_row,
                                          int tid, int threads, Bar bar) {
  const int n_tok = min(sch.T, it.r.n - it.k * sch.T);
  const int rows = n_tok * a.Gv;
  const int c0 = it.start / sch.per, c1 = (it.start + it.tiles - 1) / sch.per;
  const int cta = blockIdx.x;
  if (a.phase == 1 || c0 != c1) {
    // leave the state: phase 1 in slot item + block, a split item in its block's first or second slot
    const int m = (it.r.n + sch.T - 1) / sch.T;
    float* dst = a.phase == 1 ? a.pre + (int64_t)(it.vh * m + it.k + cta) * (R * (D + 2))
                              : a.part + (int64_t)(2 * cta + (cta == c0 ? 1 : 0)) * (R * (D + 2));
    for (int v = tid; v < rows * (D / 4); v += threads)
      reinterpret_cast<float4*>(dst)[v] = reinterpret_cast<const float4*>(own_o)[v];
    for (int v = tid; v < rows * 2; v += threads) dst[R * D + v] = own_ml[v];
    if (a.phase == 1) return;
    // the partial's stores precede thread 0's release (barrier, then a cumulative release); the last
    // block's loads follow its acquire
    bar();
    if (tid == 0) {
      int prev;
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + c0) : "memory");
      const int last = prev == c1 - c0;
      if (last) a.tickets[c0] = 0;       // every block of the item is past it
      *s_flag = last;
    }
    bar();
    if (!*s_flag) return;
  }
  const int prefix = a.phase == 2 ? max(0, *a.prefix_len) : 0;
  const bool split = c0 != c1;
  auto own = [&](int c) { return split ? pg_part<R, D>(a.part, 2 * c + (c == c0 ? 1 : 0)) : kvc_pg_state{own_o, own_ml}; };
  // maximum and sum of each row: one warp per row, its lanes over the parts
  const int warp = tid >> 5, lane = tid & 31;
  for (int r = warp; r < rows; r += threads >> 5) {
    const int t = it.r.t0 + it.k * sch.T + r / a.Gv, g = r % a.Gv;
    kvc_pg_prefix_parts pp{0, 0, 0};
    if (prefix > 0) pp = pg_prefix_parts(a, prefix, t, it.vh, g);
    auto ml_of = [&](int i) {            // part i: the prefix's first, then the item's own
      const float* p;
      if (i < pp.count) p = a.pre + (int64_t)(pp.first + i) * (a.pre_rows * (D + 2)) + a.pre_rows * D + 2 * pp.row;
      else p = own(c0 + i - pp.count).ml + 2 * r;
      return *reinterpret_cast<const float2*>(p);
    };
    const int n_parts = pp.count + c1 - c0 + 1;
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < n_parts; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int i = lane; i < n_parts; i += 32) {
      const float2 x = ml_of(i);
      L = fmaf(pg_weight(x.x, M), x.y, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) {
      s_row[2 * r] = M;
      s_row[2 * r + 1] = L != 0.f ? 1.f / L : 0.f;   // no visible slot: out 0 (a NaN goes on)
      if (a.lse != nullptr)
        a.lse[(int64_t)t * a.H + it.vh * a.Gv + g] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
  }
  bar();
  for (int v = tid; v < rows * (D / 4); v += threads) {
    const int r = v / (D / 4), d = 4 * (v % (D / 4));
    const int t = it.r.t0 + it.k * sch.T + r / a.Gv, g = r % a.Gv;
    const float M = s_row[2 * r], inv = s_row[2 * r + 1];
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (inv != 0.f) {
      if (prefix > 0) {
        const kvc_pg_prefix_parts pp = pg_prefix_parts(a, prefix, t, it.vh, g);
#pragma unroll 4
        for (int i = 0; i < pp.count; ++i) {
          const float* p = a.pre + (int64_t)(pp.first + i) * (a.pre_rows * (D + 2));
          const float m = p[a.pre_rows * D + 2 * pp.row];
          pg_acc4(x, pg_weight(m, M), *reinterpret_cast<const float4*>(p + pp.row * D + d));
        }
      }
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const kvc_pg_state st = own(c);
        pg_acc4(x, pg_weight(st.ml[2 * r], M), *reinterpret_cast<const float4*>(st.o + r * D + d));
      }
    }
    pg_store4(out + ((int64_t)t * a.H + it.vh * a.Gv + g) * D + d, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  }
}
