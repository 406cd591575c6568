// What the appends to paged stores of 16, 32 and 4 bits share: the runs that blocks take, vectors of a token's row, the
// rotation of pairs at one position or at several axes' positions.
#pragma once

#include "paged_internal.h"
#include "paged_rope.h"

#include <type_traits>

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
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
};
// With positions of several axes.
struct AxesArgs : AppendArgs {
  const int32_t* pos;         // [n_tokens][n_axes]; null: slots are the positions
  int n_axes;
  uint32_t pair_axis[4];      // two bits a pair
};
// How positions are given: slots; several axes, with each lane's VL / 2 pairs of a vector on one of them (kFlat: sections side by
// side); several axes in any order.
enum { kSlots = 0, kFlat = 1, kAny = 2 };
// What a kernel is told.  Launch parameters that it has no use for cost an fp32 step of 32 rows 0.1 us (2.64 and 2.76 us replayed, with
// bounds 3.15 and 3.28) and 8 prompts 1 %.  16-bit rotations are short of registers and get them all the same: with fewer parameters the
// compiler keeps more of them in registers and spills 12 to 24 bytes more (8 prompts into 4 bits 79.9 and 81.5 us, 40 heads, a step 3.2 and 3.0).
template <typename T, int kAxes>
using ArgsOf = std::conditional_t<kAxes != kSlots || sizeof(T) == 2, AxesArgs, AppendArgs>;

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
// Positions of a warp's tokens, eight at a time, four axes of a token in neighbouring lanes (those that there are not repeat the
// last): the angles' loads wait for one load of positions in eight tokens, not for one each.
struct Places {
  int v, i;
  unsigned bad;
  __device__ __forceinline__ Places() : v(0), i(-1), bad(0) {}
  // The next token's, `token` of the call; its warp's others follow it `stride` apart and end before `end`.  A whole warp calls it;
  // false, and the error bit, if one is outside the table.
  __device__ __forceinline__ bool next(const AxesArgs& a, int token, int stride, int end) {
    const int lane = threadIdx.x & 31;
    if ((++i & 7) == 0) {
      const int t = token + (lane >> 2) * stride;
      v = t < end ? pg_ld(a.pos + (int64_t)t * a.n_axes + min(lane & 3, a.n_axes - 1)) : 0;
      bad = __ballot_sync(0xffffffffu, v < 0 || v >= a.rope_positions);
    }
    const bool ok = (bad >> (4 * (i & 7)) & 15) == 0;
    if (!ok && lane == 0) atomicOr(a.err, KVC_DEV_BAD_POS);
    return ok;
  }
  // The token's position on an axis of the lane's own.
  __device__ __forceinline__ int of(int axis) const { return __shfl_sync(0xffffffffu, v, 4 * (i & 7) + axis); }
};
// The axes of a lane's pairs, two bits each: VL / 2 pairs from `first`, for both w.
template <typename T, int D>
__device__ __forceinline__ uint32_t lane_axes(const AxesArgs& a, int c, bool half) {
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
// (A whole warp calls it.)
template <typename T, int D, int kAxes>
__device__ __forceinline__ void load_turn_axes(Turn<T>& t, const float2* rope, const Places& at, uint32_t axes, int c, bool half) {
  constexpr int VL = Vec<T>::N;
  if constexpr (kAxes == kFlat) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int first = half ? c * VL + w * (VL / 2) : (w * (D / 2) + c * VL) / 2;
      const float2* row = rope + (int64_t)at.of(axes >> (w * VL) & 3) * (D / 2) + first;
#pragma unroll
      for (int i = 0; i < VL / 4; ++i) t.t[w][i] = pg_ld(reinterpret_cast<const float4*>(row) + i);
    }
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int first = half ? c * VL + w * (VL / 2) : (w * (D / 2) + c * VL) / 2;
#pragma unroll
      for (int i = 0; i < VL / 4; ++i) {
        const int sh = 2 * (w * (VL / 2) + 2 * i), j = first + 2 * i;
        const int p0 = at.of(axes >> sh & 3), p1 = at.of(axes >> (sh + 2) & 3);
        const uint2 x = pg_ld(reinterpret_cast<const uint2*>(rope + (int64_t)p0 * (D / 2) + j));
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
      float u, v;
      pg_rot_pair(to_f(e0), to_f(e1), co, si, &u, &v, type);
      from_f(e0, u);
      from_f(e1, v);
    }
  }
}

// The lines that the warp's next token will load.
__device__ __forceinline__ void ahead(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

// The run of this block: row b's jth page of new tokens; false if there is none.  Every row is checked once, by the first
// block, whether or not a block comes to it.
// Runs are numbered with room to spare: row b's start at cu[b] / page_size + 2 b, which leaves each
// row at least as many numbers as its tokens can touch pages.
__device__ __forceinline__ bool find_run(const AppendArgs& a, int& b, int& j) {
  const int ps = 1 << a.ps_log2;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.B; i += kThreads) row_of(a, i);
  if (a.cu == nullptr) {
    const int most = (a.n_tokens / a.B + ps - 2) / ps + 1;
    b = blockIdx.x / most;
    j = blockIdx.x % most;
    return true;
  }
  auto start = [&](int i) { return (long long)(a.cu[i] >> a.ps_log2) + 2 * i; };
  b = search(a.B, blockIdx.x, start);
  const long long jj = (long long)blockIdx.x - start(b);
  if (jj < 0 || jj > a.max_pages) return false;
  j = (int)jj;
  return true;
}

// Column group `group` of the queries of tokens at slots [p, end), every `stride`th.
template <typename T, int D, int kAxes>
__device__ __forceinline__ void append_queries(const ArgsOf<T, kAxes>& a, const Row& r, const T* q, T* q_out, int group, int p, int end,
                                               int stride, int p0) {
  constexpr int VL = Vec<T>::N;
  constexpr int PH = D / 2 / VL;          // vector pairs of a head
  const int col = group * 32 + (threadIdx.x & 31);
  const bool have = col < a.q_cols;
  if (!kAxes && !have) return;            // (with axes a warp stays whole)
  const int64_t off = (int64_t)(col / PH) * D + (col % PH) * VL;
  uint32_t axes = 0;
  if constexpr (kAxes != kSlots) axes = lane_axes<T, D>(a, col % PH, a.half);
  Places places;
  for (; p < end; p += stride) {
    Vec<T> x, y;
    Turn<T> cs;
    const T* src = q + (int64_t)(r.t0 + p - p0) * a.q_stride + off;
    if (have) {
      x.u = *reinterpret_cast<const uint4*>(src);
      y.u = *reinterpret_cast<const uint4*>(src + D / 2);
      if (p + stride < end) {
        ahead(src + stride * a.q_stride);
        ahead(src + stride * a.q_stride + D / 2);
      }
    }
    if constexpr (kAxes != kSlots) {
      if (!places.next(a, r.t0 + p - p0, stride, r.t0 + end - p0)) continue;
      load_turn_axes<T, D, kAxes>(cs, a.rope, places, axes, col % PH, a.half);
      if (!have) continue;
    } else {
      load_turn<T, D>(cs, a.rope + (int64_t)p * (D / 2), col % PH, a.half);
    }
    turn<T>(x, y, cs, a.half);
    T* dst = q_out + (int64_t)(r.t0 + p - p0) * a.H * D + off;
    *reinterpret_cast<uint4*>(dst) = x.u;
    *reinterpret_cast<uint4*>(dst + D / 2) = y.u;
  }
}

// Host: the grid for `groups` column groups; sets a.groups_y.  A warp takes about four tokens of a run: one warp of a column
// for runs of up to 4 tokens, ... 8 for more than 16.
inline dim3 run_grid(AppendArgs& a, int groups) {
  const int ps = 1 << a.ps_log2;
  const int mean = (a.n_tokens + a.B - 1) / a.B, run = mean < ps ? mean : ps;
  const int on_tokens = run <= 4 ? 1 : run <= 8 ? 2 : run <= 16 ? 4 : 8;
  a.groups_y = kWarps / on_tokens;
  const int gy = (groups + a.groups_y - 1) / a.groups_y;
  const int64_t runs = a.cu == nullptr ? (int64_t)a.B * ((a.n_tokens / a.B + ps - 2) / ps + 1)
                                       : (int64_t)a.n_tokens / ps + 2 * (int64_t)a.B;
  return dim3((unsigned)runs, gy);
}
inline void set_axes(AxesArgs& a, const kvc_rope_axes& axes, const int32_t* positions, int head_dim) {
  a.pos = positions;
  a.n_axes = axes.n_axes;
  for (int j = 0; j < head_dim / 2; ++j) a.pair_axis[j >> 4] |= (uint32_t)axes.pair_axis[j] << (2 * (j & 15));
}
// The kind of an append: kSlots, kFlat or kAny, for vectors of `vl` elements.
inline int axes_kind(const AxesArgs& a, int head_dim, int vl) {
  if (a.pos == nullptr) return kSlots;
  auto axis = [&](int j) { return a.pair_axis[j >> 4] >> (2 * (j & 15)) & 3; };
  for (int j = 0; j < head_dim / 2; ++j)
    if (axis(j) != axis(j - j % (vl / 2))) return kAny;
  return kFlat;
}

}  // namespace
