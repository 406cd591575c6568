// Append to a paged store: keys turned by RoPE at their positions and values into the pages of
// their rows, queries turned beside them, and the key bounds of the pages kept.
//
// HBM-bound for prompts (each input read once, each output written once), latency-bound for a
// decode step's few tokens.  A block takes one run: the new tokens of one row that fall into one
// page, so the row, the page number and the bounds are dealt with once per page.  A lane owns two
// 16-byte vectors of a token's row, D/2 apart in one head: both halves of the pairs (x[j],
// x[j + D/2]), or two vectors of pairs (x[2j], x[2j+1]).  A block's warps are divided between columns
// (32 such lanes' worth of the keys' and values' heads, or of the queries') and tokens: few tokens to
// a run, and all of them are on columns; many, and each takes every eighth token, some four in all,
// so that a long page does not become a long chain.  One token of a warp is in flight, all its loads together, the next one's
// on their way to L2 (eight 16-byte ones a lane, and 32 warps an SM: 6.4 TB/s for prompts, 0.94 of a copy; a decode step of 32 rows takes
// 3.3 us replayed, of which the loads that wait for the page number, though only the stores need it, are a part).
// Keys that are stored as they come (kTurn false) have instances of their own, without the rotation's registers and without the
// prefetch, which only helps where arithmetic stands between the loads: 8 prompts of 8 heads, fp16, 7.9 us (9.2 in the instance
// that can turn; with bounds 11.0 and 15.2), a step of 32 rows 2.0 (2.2).
// A run's keys, after rounding, give the page's maximum and minimum in registers: no second pass, no
// atomics.
//
// With positions of several axes (kAxes) each pair takes its angles from the row of its axis: by the same 16-byte loads where a
// lane's pairs of a vector go by one axis (sections side by side), else pair by pair.  Two frames of 1560 tokens, 40 heads of 128:
// 39.4 us, 4.9 TB/s, where slots as positions take 34.3: a position is loaded before its angles (eight tokens' at a time), and the
// shuffles that hand positions on keep warps whole.  More registers to a thread, for no spills, cost more in warps (65 us where this
// took 49); query warps that went through the keys' loop as well, to no end, cost 3.6 us.
#include "paged_append.h"

namespace {

// (a NaN goes on: the page's bounds show it wherever in the page it stands)
__device__ __forceinline__ float pick_max(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ __half pick_max(__half a, __half b) { return __hmax_nan(a, b); }
__device__ __forceinline__ __nv_bfloat16 pick_max(__nv_bfloat16 a, __nv_bfloat16 b) { return __hmax_nan(a, b); }
__device__ __forceinline__ float pick_min(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ __half pick_min(__half a, __half b) { return __hmin_nan(a, b); }
__device__ __forceinline__ __nv_bfloat16 pick_min(__nv_bfloat16 a, __nv_bfloat16 b) { return __hmin_nan(a, b); }

template <typename T, int D, bool kBounds, bool kTurn, int kAxes>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
k_paged_append(const T* k, const T* v, const T* q, T* __restrict__ kp, T* __restrict__ vp,
               T* q_out, T* __restrict__ bounds, ArgsOf<T, kAxes> a) {
  constexpr int VL = Vec<T>::N;
  constexpr int PH = D / 2 / VL;          // vector pairs of a head
  __shared__ uint4 s_red[kBounds ? kWarps : 1][4][32];
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = 1 << a.ps_log2;
  int b, j;
  if (!find_run(a, b, j)) return;
  const Row r = row_of(a, b);
  if (!r.ok || r.n == 0) return;
  const int p0 = r.len - r.n;                       // position of the row's first new token
  const int column = (p0 >> a.ps_log2) + j;
  const int lo = max(p0, column << a.ps_log2), hi = min(r.len, (column + 1) << a.ps_log2);
  if (lo >= hi) return;
  const int end = !kAxes && kTurn ? min(hi, a.rope_positions) : hi;
  if (end < hi && threadIdx.x == 0) atomicOr(a.err, KVC_DEV_BAD_POS);
  const int gw = a.groups_y;                        // column groups this block's warps divide into
  const int group = (int)blockIdx.y * gw + warp % gw;
  const int stride = kWarps / gw;
  if (kTurn && group >= a.kv_groups)
    append_queries<T, D, kAxes>(a, r, q, q_out, group - a.kv_groups, lo + warp / gw, end, stride, p0);
  // ---- keys and values ----
  const int page = a.table[(int64_t)b * a.max_pages + column];
  if (page < 0 || page >= a.n_pages) {              // (the same for the whole block)
    if (threadIdx.x == 0) atomicOr(a.err, KVC_DEV_BAD_PAGE);
    return;
  }
  const int col = group * 32 + lane;
  const bool have = group < a.kv_groups && col < a.kv_cols;
  const int head = have ? col / PH : 0, c = have ? col % PH : 0;
  const int64_t src0 = (int64_t)head * D + c * VL;
  const int64_t dst_row = (int64_t)a.Hkv * D;
  Vec<T> mx0, mx1, mn0, mn1;
  bool any = false;
  if (kAxes ? group < a.kv_groups : have) {         // (with axes a warp stays whole; those of queries alone leave the keys out)
    uint32_t axes = 0;
    if constexpr (kAxes != kSlots) axes = lane_axes<T, D>(a, c, a.half);
    Places places;
    for (int p = lo + warp / gw; p < end; p += stride) {
      Vec<T> x, y, vx, vy;
      Turn<T> cs;
      const int64_t off = (int64_t)(r.t0 + p - p0) * a.kv_stride + src0;
      x.u = pg_ld(reinterpret_cast<const uint4*>(k + off));
      y.u = pg_ld(reinterpret_cast<const uint4*>(k + off + D / 2));
      if (kTurn && p + stride < end) {
        const int64_t next = off + stride * a.kv_stride;
        ahead(k + next);
        ahead(k + next + D / 2);
        ahead(v + next);
        ahead(v + next + D / 2);
      }
      if constexpr (kAxes != kSlots) {
        if (!places.next(a, r.t0 + p - p0, stride, r.t0 + end - p0)) continue;
        load_turn_axes<T, D, kAxes>(cs, a.rope, places, axes, c, a.half);
        if (!have) continue;
      } else if (kTurn) {
        load_turn<T, D>(cs, a.rope + (int64_t)p * (D / 2), c, a.half);
      }
      vx.u = pg_ld(reinterpret_cast<const uint4*>(v + off));
      vy.u = pg_ld(reinterpret_cast<const uint4*>(v + off + D / 2));
      const int64_t dst = (((int64_t)page << a.ps_log2) + (p & (ps - 1))) * dst_row + src0;
      *reinterpret_cast<uint4*>(vp + dst) = vx.u;
      *reinterpret_cast<uint4*>(vp + dst + D / 2) = vy.u;
      if (kTurn) turn<T>(x, y, cs, a.half);
      *reinterpret_cast<uint4*>(kp + dst) = x.u;
      *reinterpret_cast<uint4*>(kp + dst + D / 2) = y.u;
      if (kBounds) {
        if (!any) {
          mx0.u = mn0.u = x.u;
          mx1.u = mn1.u = y.u;
          any = true;
        } else {
#pragma unroll
          for (int i = 0; i < VL; ++i) {
            mx0.e[i] = pick_max(mx0.e[i], x.e[i]);
            mn0.e[i] = pick_min(mn0.e[i], x.e[i]);
            mx1.e[i] = pick_max(mx1.e[i], y.e[i]);
            mn1.e[i] = pick_min(mn1.e[i], y.e[i]);
          }
        }
      }
    }
  }
  if (!kBounds || end <= lo) return;                // (uniform per block)
  // warps of the same columns, then what the page held before
  if (kAxes && !any) {                              // (tokens may have been left out)
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      from_f(mx0.e[i], -INFINITY);
      from_f(mn0.e[i], INFINITY);
    }
    mx1.u = mx0.u;
    mn1.u = mn0.u;
  }
  s_red[warp][0][lane] = mx0.u;
  s_red[warp][1][lane] = mx1.u;
  s_red[warp][2][lane] = mn0.u;
  s_red[warp][3][lane] = mn1.u;
  if (kAxes) {
    if (!__syncthreads_or(any)) return;             // nothing written to this page
  } else {
    __syncthreads();
  }
  if (warp >= gw || !have) return;                  // the warp of the run's first token has one for sure
  auto widen = [&](const uint4& a0, const uint4& a1, const uint4& i0, const uint4& i1) {
    Vec<T> u0, u1, w0, w1;
    u0.u = a0;
    u1.u = a1;
    w0.u = i0;
    w1.u = i1;
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      mx0.e[i] = pick_max(mx0.e[i], u0.e[i]);
      mx1.e[i] = pick_max(mx1.e[i], u1.e[i]);
      mn0.e[i] = pick_min(mn0.e[i], w0.e[i]);
      mn1.e[i] = pick_min(mn1.e[i], w1.e[i]);
    }
  };
  for (int w = warp + gw, t = 1; t < stride; w += gw, ++t)
    if (lo + t < end) widen(s_red[w][0][lane], s_red[w][1][lane], s_red[w][2][lane], s_red[w][3][lane]);
  T* bd = bounds + (((int64_t)page * a.Hkv + head) * 2) * D + c * VL;
  if (lo & (ps - 1))
    widen(*reinterpret_cast<const uint4*>(bd), *reinterpret_cast<const uint4*>(bd + D / 2),
          *reinterpret_cast<const uint4*>(bd + D), *reinterpret_cast<const uint4*>(bd + D + D / 2));
  *reinterpret_cast<uint4*>(bd) = mx0.u;
  *reinterpret_cast<uint4*>(bd + D / 2) = mx1.u;
  *reinterpret_cast<uint4*>(bd + D) = mn0.u;
  *reinterpret_cast<uint4*>(bd + D + D / 2) = mn1.u;
}

template <typename T, int D>
cudaError_t launch(kvc_paged* c, const void* k, const void* v, const void* q, void* q_out, AxesArgs a,
                   cudaStream_t s) {
  constexpr int VL = Vec<T>::N;
  a.kv_cols = a.Hkv * (D / 2 / VL);
  a.q_cols = q != nullptr ? a.H * (D / 2 / VL) : 0;
  a.kv_groups = (a.kv_cols + 31) / 32;
  const int groups = a.kv_groups + (a.q_cols + 31) / 32;
  const dim3 grid = run_grid(a, groups);
  auto go = [&](auto kernel) {
    return kvc_launch_pdl(kernel, grid, dim3(kThreads), 0, s, (const T*)k, (const T*)v, (const T*)q, (T*)c->k, (T*)c->v,
                          (T*)q_out, (T*)c->bounds, a);
  };
  const bool bounds = c->bounds != nullptr;
  if (a.rope == nullptr) return bounds ? go(k_paged_append<T, D, true, false, kSlots>) : go(k_paged_append<T, D, false, false, kSlots>);
  switch (axes_kind(a, D, VL)) {
    case kSlots: return bounds ? go(k_paged_append<T, D, true, true, kSlots>) : go(k_paged_append<T, D, false, true, kSlots>);
    case kFlat: return bounds ? go(k_paged_append<T, D, true, true, kFlat>) : go(k_paged_append<T, D, false, true, kFlat>);
    default: return bounds ? go(k_paged_append<T, D, true, true, kAny>) : go(k_paged_append<T, D, false, true, kAny>);
  }
}

}  // namespace

cudaError_t kvc_pg_launch_append(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                                 int64_t q_stride, void* q_out, int n_tokens, const int32_t* cu, const float* rope,
                                 int rope_positions, const kvc_rope_axes* axes, const int32_t* positions, bool half,
                                 cudaStream_t s) {
  const kvc_paged_config& g = c->cfg;
  AxesArgs a{};
  a.table = c->table;
  a.kv_len = c->kv_len;
  a.cu = cu;
  a.err = reinterpret_cast<int32_t*>(c->ws);
  a.rope = reinterpret_cast<const float2*>(rope);
  a.rope_positions = rope_positions;
  a.B = g.batch;
  a.n_tokens = n_tokens;
  a.ps_log2 = c->ps_log2;
  a.n_pages = g.n_pages;
  a.max_pages = g.max_pages;
  a.kv_stride = kv_stride;
  a.q_stride = q_stride;
  a.H = g.heads;
  a.Hkv = g.kv_heads;
  a.half = half;
  if (axes != nullptr) set_axes(a, *axes, positions, g.head_dim);
  const bool d64 = g.head_dim == 64;
  switch (g.dtype) {
    case KVC_F32: return d64 ? launch<float, 64>(c, k, v, q, q_out, a, s) : launch<float, 128>(c, k, v, q, q_out, a, s);
    case KVC_F16: return d64 ? launch<__half, 64>(c, k, v, q, q_out, a, s) : launch<__half, 128>(c, k, v, q, q_out, a, s);
    default:
      return d64 ? launch<__nv_bfloat16, 64>(c, k, v, q, q_out, a, s) : launch<__nv_bfloat16, 128>(c, k, v, q, q_out, a, s);
  }
}
