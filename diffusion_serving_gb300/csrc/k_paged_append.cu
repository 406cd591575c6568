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
// so that a long page does not become a long chain.  One token of a warp is in flight, all its loads together
// (eight 16-byte ones a lane, and 32 warps an SM: 5.2 TB/s for prompts, 0.77 of a copy; a decode step of 32 rows takes
// 5 us replayed, of which the loads that wait for the page number, though only the stores need it, are a part).
// A run's keys, after rounding, give the page's maximum and minimum in registers: no second pass, no
// atomics.
//
// With positions of several axes (kAxes) each pair takes its angles from the row of its axis: two neighbouring pairs of
// one axis by one 16-byte load, as before, others by two of 8 bytes.
#include "paged_internal.h"
#include "paged_rope.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
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

template <typename T>
union Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 u;
  T e[16 / sizeof(T)];
  __device__ Vec() {}
};

struct AppendArgs {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  int32_t* err;
  const float2* rope;
  int rope_positions;
  int B, n_tokens, ps_log2, n_pages, max_pages;
  int groups_y;               // column groups per block
  int64_t kv_stride, q_stride;
  int kv_cols, q_cols;        // vector pairs of a key / query row
  int kv_groups;              // column groups of the keys; those of the queries follow
  int H, Hkv;
  int half;
  const int32_t* pos;         // [n_tokens][n_axes], with axes
  int n_axes;
  uint32_t pair_axis[4];      // two bits a pair
};

// Turns the two vectors x (elements c VL ..) and y (D/2 further) of a head by the row `cs` of the table.
template <typename T>
struct Turn {
  float4 t[2][Vec<T>::N / 4];
};
// The entries of VL / 2 pairs each: of the two halves' elements w VL/2 .., or of vector w.
template <typename T, int D>
__device__ __forceinline__ void load_turn(Turn<T>& t, const float2* cs, int c, bool half) {
  constexpr int VL = Vec<T>::N;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = half ? c * VL + w * (VL / 2) : (w * (D / 2) + c * VL) / 2;
#pragma unroll
    for (int i = 0; i < VL / 4; ++i) t.t[w][i] = pg_ld(reinterpret_cast<const float4*>(cs + first) + i);
  }
}
// A token's positions, one per axis (those that there are not repeat the last).
struct Place {
  int p[4];
  __device__ __forceinline__ int of(int axis) const {
    return axis & 2 ? (axis & 1 ? p[3] : p[2]) : (axis & 1 ? p[1] : p[0]);
  }
};
__device__ __forceinline__ bool load_place(const AppendArgs& a, int64_t token, Place& at) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    at.p[i] = i < a.n_axes ? pg_ld(a.pos + token * a.n_axes + i) : at.p[i > 0 ? i - 1 : 0];
    ok = ok && at.p[i] >= 0 && at.p[i] < a.rope_positions;
  }
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(a.err, KVC_DEV_BAD_POS);
  return ok;
}
// The axes of a lane's pairs, two bits each: VL / 2 pairs from `first`, for both w.
template <typename T, int D>
__device__ __forceinline__ uint32_t lane_axes(const AppendArgs& a, int c, bool half) {
  constexpr int VL = Vec<T>::N;
  uint32_t bits = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = half ? c * VL + w * (VL / 2) : (w * (D / 2) + c * VL) / 2;
#pragma unroll
    for (int i = 0; i < VL / 2; ++i) {
      const int j = first + i, word = j >> 4;
      const uint32_t x = word & 2 ? (word & 1 ? a.pair_axis[3] : a.pair_axis[2]) : (word & 1 ? a.pair_axis[1] : a.pair_axis[0]);
      bits |= (x >> (2 * (j & 15)) & 3) << (2 * (w * (VL / 2) + i));
    }
  }
  return bits;
}
template <typename T, int D>
__device__ __forceinline__ void load_turn_axes(Turn<T>& t, const float2* rope, const Place& at, uint32_t axes, int c, bool half) {
  constexpr int VL = Vec<T>::N;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = half ? c * VL + w * (VL / 2) : (w * (D / 2) + c * VL) / 2;
#pragma unroll
    for (int i = 0; i < VL / 4; ++i) {
      const int sh = 2 * (w * (VL / 2) + 2 * i), j = first + 2 * i;
      const int p0 = at.of(axes >> sh & 3), p1 = at.of(axes >> (sh + 2) & 3);
      const float2* r0 = rope + (int64_t)p0 * (D / 2) + j;
      if (p0 == p1) {
        t.t[w][i] = pg_ld(reinterpret_cast<const float4*>(r0));
      } else {
        const uint2 x = pg_ld(reinterpret_cast<const uint2*>(r0));
        const uint2 y = pg_ld(reinterpret_cast<const uint2*>(rope + (int64_t)p1 * (D / 2) + j + 1));
        t.t[w][i] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(y.x), __uint_as_float(y.y));
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void turn(Vec<T>& x, Vec<T>& y, const Turn<T>& cs, bool half) {
  constexpr int VL = Vec<T>::N;
  const T* type = nullptr;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float4* t = cs.t[w];
#pragma unroll
    for (int i = 0; i < VL / 2; ++i) {
      const float co = i & 1 ? t[i / 2].z : t[i / 2].x, si = i & 1 ? t[i / 2].w : t[i / 2].y;
      T& e0 = half ? x.e[w * (VL / 2) + i] : (w ? y : x).e[2 * i];
      T& e1 = half ? y.e[w * (VL / 2) + i] : (w ? y : x).e[2 * i + 1];
      const float a = to_f(e0), b = to_f(e1);
      from_f(e0, pg_rot(a, co, b, si, type));
      from_f(e1, pg_rot(a, si, b, -co, type));
    }
  }
}

// Row b's tokens and length, checked (the error bits are set by the first block alone).
struct Row {
  int t0, n, len;
  bool ok;
};
__device__ __forceinline__ Row row_of(const AppendArgs& a, int b) {
  Row r;
  if (a.cu == nullptr) {
    r.n = a.n_tokens / a.B;
    r.t0 = b * r.n;
    r.ok = true;
  } else {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    r.t0 = lo;
    r.n = hi - lo;
    r.ok = lo >= 0 && hi >= lo && hi <= a.n_tokens;
  }
  r.len = a.kv_len[b];
  const bool len_ok = r.len >= 0 && r.len <= (a.max_pages << a.ps_log2) && (!r.ok || r.len >= r.n);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (!r.ok) atomicOr(a.err, KVC_DEV_BAD_CUSEQ);
    if (!len_ok) atomicOr(a.err, KVC_DEV_BAD_KVLEN);
  }
  r.ok = r.ok && len_ok;
  return r;
}

// The last b in [0, B) with f(b) <= x, by a whole warp: 32 probes a step.
template <typename F>
__device__ __forceinline__ int search(int B, long long x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
#pragma unroll 1
  for (int step = 0; step < 3 && n > 1; ++step) {
    const int w = (n + 31) / 32;
    const int b = lo + lane * w;
    const unsigned hit = __ballot_sync(0xffffffffu, lane * w < n && f(b) <= x);
    const int last = hit ? 31 - __clz(hit) : 0;
    lo += last * w;
    n = min(w, n - last * w);
  }
  return lo;
}

template <typename T, int D, bool kBounds, bool kAxes>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
k_paged_append(const T* k, const T* v, const T* q, T* __restrict__ kp, T* __restrict__ vp,
               T* q_out, T* __restrict__ bounds, AppendArgs a) {
  constexpr int VL = Vec<T>::N;
  constexpr int PH = D / 2 / VL;          // vector pairs of a head
  __shared__ uint4 s_red[kBounds ? kWarps : 1][4][32];
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = 1 << a.ps_log2;
  if (blockIdx.x == 0 && blockIdx.y == 0)      // every row is checked once, whether or not a block comes to it
    for (int b = threadIdx.x; b < a.B; b += kThreads) row_of(a, b);

  // ---- the run of this block ----
  // Runs are numbered with room to spare: row b's start at cu[b] / page_size + 2 b, which leaves each
  // row at least as many numbers as its tokens can touch pages.
  int b, j;
  if (a.cu == nullptr) {
    const int most = (a.n_tokens / a.B + ps - 2) / ps + 1;
    b = blockIdx.x / most;
    j = blockIdx.x % most;
  } else {
    auto start = [&](int i) { return (long long)(a.cu[i] >> a.ps_log2) + 2 * i; };
    b = search(a.B, blockIdx.x, start);
    const long long jj = (long long)blockIdx.x - start(b);
    if (jj < 0 || jj > a.max_pages) return;
    j = (int)jj;
  }
  const Row r = row_of(a, b);
  if (!r.ok || r.n == 0) return;
  const int p0 = r.len - r.n;                       // position of the row's first new token
  const int column = (p0 >> a.ps_log2) + j;
  const int lo = max(p0, column << a.ps_log2), hi = min(r.len, (column + 1) << a.ps_log2);
  if (lo >= hi) return;
  const int end = !kAxes && a.rope != nullptr ? min(hi, a.rope_positions) : hi;
  if (end < hi && threadIdx.x == 0) atomicOr(a.err, KVC_DEV_BAD_POS);
  const int gw = a.groups_y;                        // column groups this block's warps divide into
  const int group = (int)blockIdx.y * gw + warp % gw;
  const int stride = kWarps / gw;
  if (group >= a.kv_groups) {
    // ---- queries ----
    const int col = (group - a.kv_groups) * 32 + lane;
    if (col < a.q_cols) {
      const int64_t off = (int64_t)(col / PH) * D + (col % PH) * VL;
      const uint32_t axes = kAxes ? lane_axes<T, D>(a, col % PH, a.half) : 0;
      for (int p = lo + warp / gw; p < end; p += stride) {
        Vec<T> x, y;
        Turn<T> cs;
        Place at;
        if (kAxes && !load_place(a, r.t0 + p - p0, at)) continue;
        const T* src = q + (int64_t)(r.t0 + p - p0) * a.q_stride + off;
        x.u = *reinterpret_cast<const uint4*>(src);
        y.u = *reinterpret_cast<const uint4*>(src + D / 2);
        if (kAxes) load_turn_axes<T, D>(cs, a.rope, at, axes, col % PH, a.half);
        else load_turn<T, D>(cs, a.rope + (int64_t)p * (D / 2), col % PH, a.half);
        turn<T>(x, y, cs, a.half);
        T* dst = q_out + (int64_t)(r.t0 + p - p0) * a.H * D + off;
        *reinterpret_cast<uint4*>(dst) = x.u;
        *reinterpret_cast<uint4*>(dst + D / 2) = y.u;
      }
    }
  }
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
  if (have) {
    const uint32_t axes = kAxes ? lane_axes<T, D>(a, c, a.half) : 0;
    for (int p = lo + warp / gw; p < end; p += stride) {
      Vec<T> x, y, vx, vy;
      Turn<T> cs;
      Place at;
      if (kAxes && !load_place(a, r.t0 + p - p0, at)) continue;
      const int64_t off = (int64_t)(r.t0 + p - p0) * a.kv_stride + src0;
      x.u = pg_ld(reinterpret_cast<const uint4*>(k + off));
      y.u = pg_ld(reinterpret_cast<const uint4*>(k + off + D / 2));
      if (kAxes) load_turn_axes<T, D>(cs, a.rope, at, axes, c, a.half);
      else if (a.rope != nullptr) load_turn<T, D>(cs, a.rope + (int64_t)p * (D / 2), c, a.half);
      vx.u = pg_ld(reinterpret_cast<const uint4*>(v + off));
      vy.u = pg_ld(reinterpret_cast<const uint4*>(v + off + D / 2));
      const int64_t dst = (((int64_t)page << a.ps_log2) + (p & (ps - 1))) * dst_row + src0;
      *reinterpret_cast<uint4*>(vp + dst) = vx.u;
      *reinterpret_cast<uint4*>(vp + dst + D / 2) = vy.u;
      if (kAxes || a.rope != nullptr) turn<T>(x, y, cs, a.half);
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
cudaError_t launch(kvc_paged* c, const void* k, const void* v, const void* q, void* q_out, AppendArgs a,
                   cudaStream_t s) {
  constexpr int VL = Vec<T>::N;
  a.kv_cols = a.Hkv * (D / 2 / VL);
  a.q_cols = q != nullptr ? a.H * (D / 2 / VL) : 0;
  a.kv_groups = (a.kv_cols + 31) / 32;
  const int groups = a.kv_groups + (a.q_cols + 31) / 32;
  // a warp takes about four tokens of a run: one warp of a column for runs of up to 4 tokens, ... 8 for more than 16
  const int ps = 1 << a.ps_log2;
  const int mean = (a.n_tokens + a.B - 1) / a.B, run = mean < ps ? mean : ps;
  const int on_tokens = run <= 4 ? 1 : run <= 8 ? 2 : run <= 16 ? 4 : 8;
  a.groups_y = kWarps / on_tokens;
  const int gy = (groups + a.groups_y - 1) / a.groups_y;
  const int64_t runs = a.cu == nullptr ? (int64_t)a.B * ((a.n_tokens / a.B + ps - 2) / ps + 1)
                                       : (int64_t)a.n_tokens / ps + 2 * (int64_t)a.B;
  const dim3 grid((unsigned)runs, gy);
  auto go = [&](auto kernel) {
    return kvc_launch_pdl(kernel, grid, dim3(kThreads), 0, s, (const T*)k, (const T*)v, (const T*)q, (T*)c->k, (T*)c->v,
                          (T*)q_out, (T*)c->bounds, a);
  };
  if (a.pos != nullptr) return c->bounds != nullptr ? go(k_paged_append<T, D, true, true>) : go(k_paged_append<T, D, false, true>);
  return c->bounds != nullptr ? go(k_paged_append<T, D, true, false>) : go(k_paged_append<T, D, false, false>);
}

}  // namespace

cudaError_t kvc_pg_launch_append(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                                 int64_t q_stride, void* q_out, int n_tokens, const int32_t* cu, const float* rope,
                                 int rope_positions, const kvc_rope_axes* axes, const int32_t* positions, bool half,
                                 cudaStream_t s) {
  const kvc_paged_config& g = c->cfg;
  AppendArgs a{};
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
  if (axes != nullptr) {
    a.pos = positions;
    a.n_axes = axes->n_axes;
    for (int j = 0; j < g.head_dim / 2; ++j) a.pair_axis[j >> 4] |= (uint32_t)axes->pair_axis[j] << (2 * (j & 15));
  }
  const bool d64 = g.head_dim == 64;
  switch (g.dtype) {
    case KVC_F32: return d64 ? launch<float, 64>(c, k, v, q, q_out, a, s) : launch<float, 128>(c, k, v, q, q_out, a, s);
    case KVC_F16: return d64 ? launch<__half, 64>(c, k, v, q, q_out, a, s) : launch<__half, 128>(c, k, v, q, q_out, a, s);
    default:
      return d64 ? launch<__nv_bfloat16, 64>(c, k, v, q, q_out, a, s) : launch<__nv_bfloat16, 128>(c, k, v, q, q_out, a, s);
  }
}
