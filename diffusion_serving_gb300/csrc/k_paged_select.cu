// Which pages a token attends: scores from the pages' key bounds, then the n_select best.
//
//   U(page) = max over the group's heads g of sum_d max(q_gd hi_d, q_gd lo_d)
//           = max over g of (q_g+ . hi + q_g- . lo),  q+ = max(q, 0), q- = min(q, 0),
// bounds every score q_g . k of the page's keys from above.
//
// k_paged_score_mma (16-bit stores) takes the second form: a product of [q+ q-] with a page's 2 D
// bounds, by warp-level MMAs, heads in M and pages in N.  It is HBM-bound: each page's bounds are
// read once, 1 / page_size of the bytes of its keys and values.  The order of the contraction is free,
// so a lane takes 8 dims of a page in one 16-byte load, and the queries are laid out to match.  A
// block's life is short (8 sets of 8 pages a warp), so its chain of loads counts: the row's length, page numbers and
// queries are asked for together, the first bounds before the queries are worked on.  16 rows of up to 2048 pages,
// 8 kv heads of 128 (83 MB): 22 us, 3.8 TB/s (33 with the loads one after another); 4.5 us for one row.
// k_paged_score does fp32 stores with FMAs, a warp per page.
//
// Bounds that are infinite or NaN.  The first pass's scores then say nothing (an infinity meets the zeroed half of q as
// 0 times infinity; max drops a NaN), so any of them makes the error bound of its (row, kv head) infinite: every page is
// scored again in fp64 by the definition, a query element of 0 adding 0, and a page whose score is NaN ranks first.
//
// k_paged_rank, a block per (row, kv head), takes the n_select largest.  Rounding could swap pages
// whose scores nearly agree, so it decides nothing: with |error| <= delta, a page more than 2 delta
// above the last one taken is in, one more than 2 delta below is out, and those between are scored
// again in twice fp32's precision (products and sums with their rounding errors; fp64 is some fifty
// times slower than fp32 here) and ranked by that, equal ones by column.  "The last one taken" need
// only be known to within a narrow interval: a histogram of 2048 equal steps between the least and
// the largest score gives one that mostly holds a few pages.  Where it does not serve (scores all but
// equal, or not finite), radix selection takes its place.  Bound by the latency of its eight or so
// phases between barriers: 8 us for one row of 2048 pages, 10 for 16.
#include "paged_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

struct SelArgs {
  const int32_t* table;
  const int32_t* kv_len;
  int32_t* err;
  int B, H, Hkv, G, ps_log2, n_pages, max_pages;
  double* scores;            // [B * Hkv][max_pages]; k_paged_score's fp32 stand in the first half of each part
  uint32_t* score_max;       // [B * Hkv] fp32 bits: largest sum of a score's |terms|; left at 0
  int n_sel, first, recent;
  int32_t* sel;
};

// pages of row b; -1 for a bad length
__device__ __forceinline__ int row_pages(const SelArgs& a, int b) {
  const int len = a.kv_len[b];
  if (len < 0 || len > (a.max_pages << a.ps_log2)) return -1;
  return (len + (1 << a.ps_log2) - 1) >> a.ps_log2;
}

constexpr int kScoreThreads = 256;
constexpr float kWide = 0x1p120f;          // sums of terms above it count as infinite (their fp32 sums could leave the range)

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads)
k_paged_score(const T* q, const T* bounds, SelArgs a) {
  constexpr int N = D / 32;
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int np = row_pages(a, b);
  if (np <= a.n_sel) return;                         // every page is taken: nothing to rank
  float* out = reinterpret_cast<float*>(a.scores + ((int64_t)b * a.Hkv + kvh) * a.max_pages);
  float terms = 0.f;
  for (int j = blockIdx.x * (kScoreThreads / 32) + warp; j < np; j += gridDim.x * (kScoreThreads / 32)) {
    const int page = a.table[(int64_t)b * a.max_pages + j];
    float best = -INFINITY;
    if (page >= 0 && page < a.n_pages) {             // (a bad page is reported by the attention that meets it)
      const T* bd = bounds + ((int64_t)page * a.Hkv + kvh) * 2 * D + lane * N;
      float hi[N], lo[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        hi[i] = to_f(bd[i]);
        lo[i] = to_f(bd[D + i]);
      }
      for (int g = 0; g < a.G; ++g) {
        const T* qp = q + ((int64_t)b * a.H + kvh * a.G + g) * D + lane * N;
        float u = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float x = to_f(qp[i]);
          u = fmaf(x, x > 0.f ? hi[i] : lo[i], u);
          t = fmaf(fabsf(x), fmaxf(fabsf(hi[i]), fabsf(lo[i])), t);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          u += __shfl_xor_sync(0xffffffffu, u, o);
          t += __shfl_xor_sync(0xffffffffu, t, o);
        }
        best = fmaxf(best, u);
        terms = t < kWide && u == u ? fmaxf(terms, t) : INFINITY;
      }
    }
    if (lane == 0) out[j] = best;
  }
  if (lane == 0 && terms > 0.f) atomicMax(a.score_max + b * a.Hkv + kvh, __float_as_uint(terms));
}

// ---- 16-bit stores --------------------------------------------------------------------
constexpr int kMmaWarps = 4;

template <typename T>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);   // A's rows 8..15 are zero
template <>
__device__ __forceinline__ void mma<__half>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(0u), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(0u), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float2 pair_f(uint32_t u, const __half*) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ float2 pair_f(uint32_t u, const __nv_bfloat16*) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, const __half*) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, const __nv_bfloat16*) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, const __half*) {
  const __half2 r = __hmin2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, const __nv_bfloat16*) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// the pair's positive (or negative) parts
__device__ __forceinline__ uint32_t part_of(uint32_t u, bool negative) {
  uint32_t neg;                                            // ffff where the half is negative
  asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(neg) : "r"(u));
  return negative ? u & neg : u & ~neg;
}

// A warp takes 8 pages at a time: lane (n, c) = (lane / 4, lane % 4) holds dims 32 v + 8 c .. + 7 of page n's bounds.
// The two k16 steps of a vector pair its dims as (0, 1 | 2, 3) and (4, 5 | 6, 7) where the MMA counts k = 2 c, 2 c + 1 |
// 2 c + 8, 2 c + 9; the queries' fragments hold the same dims, so the sum is the same.
template <typename T, int D>
__global__ void __launch_bounds__(kMmaWarps * 32)
k_paged_score_mma(const T* q, const T* bounds, SelArgs a) {
  constexpr int V = D / 32;                 // 16-byte vectors per lane of one bound
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int first = (blockIdx.x * kMmaWarps + warp) * 8, step = gridDim.x * kMmaWarps * 8;
  const T* type = nullptr;
  float* out = reinterpret_cast<float*>(a.scores + ((int64_t)b * a.Hkv + kvh) * a.max_pages);
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
  // the row's length, its first pages' numbers (used where the length says so) and the first queries, loaded together
  int page = first + n < a.max_pages ? pg_ld(table + first + n) : -1;
  uint4 qx[V];
  auto load_q = [&](int g0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      qx[v] = make_uint4(0, 0, 0, 0);
      if (g0 + n < a.G) qx[v] = pg_ld(reinterpret_cast<const uint4*>(q + ((int64_t)b * a.H + kvh * a.G + g0 + n) * D + 32 * v + 8 * c));
    }
  };
  load_q(0);
  const int np = row_pages(a, b);
  if (np <= a.n_sel) return;                // every page is taken: nothing to rank
  if (first >= np) return;
  float terms = 0.f;
  for (int g0 = 0; g0 < a.G; g0 += 8) {     // 8 heads a pass
    if (g0 > 0) {
      load_q(g0);
      page = first + n < np ? pg_ld(table + first + n) : -1;
    } else if (first + n >= np) {
      page = -1;
    }
    bool ok;
    uint4 x[2][V];
    auto load_x = [&] {                     // (a bad page is reported by the attention that meets it)
      ok = page >= 0 && page < a.n_pages;
      const uint4* bd = reinterpret_cast<const uint4*>(bounds + ((int64_t)(ok ? page : 0) * a.Hkv + kvh) * 2 * D);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < V; ++v) x[h][v] = ok ? pg_ld(bd + h * (D / 8) + 4 * v + c) : make_uint4(0, 0, 0, 0);
    };
    load_x();
    uint32_t qa[2][V][2][2];                // [hi, lo][vector][k16 step][k half]
    float l1 = 0.f;
    const bool real = g0 + n < a.G;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t w[4] = {qx[v].x, qx[v].y, qx[v].z, qx[v].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qa[0][v][i >> 1][i & 1] = part_of(w[i], false);
        qa[1][v][i >> 1][i & 1] = part_of(w[i], true);
        const float2 f = pair_f(w[i], type);
        l1 += fabsf(f.x) + fabsf(f.y);
      }
    }
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (!(l1 < INFINITY)) l1 = INFINITY;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l1 = fmaxf(l1, __shfl_xor_sync(0xffffffffu, l1, o));
    uint32_t top2 = 0u, low2 = 0u;          // largest upper and least lower bound (or 0), 16-bit pairs
    for (int j = first; j < np; j += step) {
      if (j > first) load_x();
      page = j + step + n < np ? pg_ld(table + j + step + n) : -1;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint32_t w[4] = {x[h][v].x, x[h][v].y, x[h][v].z, x[h][v].w};
          mma<T>(s[h], qa[h][v][0], w[0], w[1]);
          mma<T>(s[h], qa[h][v][1], w[2], w[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (h == 0) top2 = max2(top2, w[i], type);
            else low2 = min2(low2, w[i], type);
          }
        }
      // head g0 + n of this lane: pages j + 2 c, + 1
      const bool good = __shfl_sync(0xffffffffu, ok, 8 * c), good1 = __shfl_sync(0xffffffffu, ok, 8 * c + 4);
      float u0 = real && good ? s[0][0] + s[1][0] : -INFINITY, u1 = real && good1 ? s[0][1] + s[1][1] : -INFINITY;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, o));
        u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, o));
      }
      if (lane < 4) {
        const int i = j + 2 * lane;
        if (i < np) out[i] = g0 == 0 ? u0 : fmaxf(out[i], u0);
        if (i + 1 < np) out[i + 1] = g0 == 0 ? u1 : fmaxf(out[i + 1], u1);
      }
    }
    // no score's terms sum to more (an upper bound below 0 has a lower one further from it); NaN where one of these is
    const float2 top = pair_f(top2, type), low = pair_f(low2, type);
    const float t = l1 * fmaxf(fmaxf(top.x, top.y), -fminf(low.x, low.y));
    const bool finite = t < kWide && top.x == top.x && top.y == top.y && low.x == low.x && low.y == low.y;
    terms = finite ? fmaxf(terms, t) : INFINITY;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) terms = fmaxf(terms, __shfl_xor_sync(0xffffffffu, terms, o));
  if (lane == 0 && terms > 0.f) atomicMax(a.score_max + b * a.Hkv + kvh, __float_as_uint(terms));
}

// ---- ranking ----------------------------------------------------------------------------
constexpr int kRankThreads = 512, kRankWarps = kRankThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 512;                  // candidates ranked by comparing each with each

// order-preserving whole numbers
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {             // (in whole numbers: fp64 instructions are slow here)
  const uint64_t u = (uint64_t)__double_as_longlong(x), m = u << 1;
  if (m > 0xffe0000000000000ull) return ~0ull;       // NaN before all
  if (m == 0) return 0x8000000000000000ull;          // -0 counts as 0
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// Exclusive sum over the block's threads of `x`, and the total.
__device__ __forceinline__ int block_scan(int x, int* s_warp, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = y;
  __syncthreads();
  const int mine = lane < kRankThreads / 32 ? s_warp[lane] : 0;
  int sums = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += z;
  }
  *total = __shfl_sync(0xffffffffu, sums, 31);
  return __shfl_sync(0xffffffffu, sums - mine, warp) + y - x;
}

// The need-th largest (need >= 1) of key(i) over i in [0, n) with in(i), a byte a pass from the top.
template <typename K, typename Key, typename In>
__device__ __forceinline__ K radix_select(int n, int need, int* s_hist, int* s_pick, Key key, In in) {
  K prefix = 0, mask = 0;
#pragma unroll 1
  for (int shift = (int)sizeof(K) * 8 - 8; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kRankThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRankThreads) {
      if (!in(i)) continue;
      const K x = key(i);
      if ((x & mask) == prefix) atomicAdd(s_hist + (int)((x >> shift) & 255), 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l holds digits 255 - 8 l down to 248 - 8 l
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = s_hist[255 - 8 * (int)threadIdx.x - i];
        sum += c[i];
      }
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, above, o);
        if ((int)threadIdx.x >= o) above += z;
      }
      above -= sum;
      if (above < need && need <= above + sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < need && need <= above + c[i]) {
            s_pick[0] = 255 - 8 * (int)threadIdx.x - i;
            s_pick[1] = need - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix |= (K)s_pick[0] << shift;
    mask |= (K)255 << shift;
    need = s_pick[1];
  }
  return prefix;
}

// x + y and its rounding error
__device__ __forceinline__ float two_sum(float x, float y, float& err) {
  const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
  err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t));
  return s;
}

// Score of a page for one head, in twice fp32's precision, where no sum of terms leaves fp32's range; every lane of the warp
// returns it.
template <typename T, int D>
__device__ __forceinline__ double fine_score(const T* q, const T* bd, int lane) {
  float hi = 0.f, lo = 0.f;
  T qx[D / 32], up[D / 32], dn[D / 32];              // (both bounds: which one counts is known only with q)
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    qx[i] = q[lane + 32 * i];
    up[i] = bd[lane + 32 * i];
    dn[i] = bd[D + lane + 32 * i];
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const float x = to_f(qx[i]), y = to_f(x > 0.f ? up[i] : dn[i]);
    const float p = __fmul_rn(x, y), e = __fmaf_rn(x, y, -p);
    float r;
    hi = two_sum(hi, p, r);
    lo += r + e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    float r;
    const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
    // (the same on both sides of the exchange: the sum and its error, which is exact, are symmetric)
    hi = two_sum(hi, h, r);
    lo = (lo + l) + r;
  }
  return (double)hi + (double)lo;
}

// The same in fp64, for terms that leave that range, infinite bounds and NaN among them; a query element of 0 adds 0.
template <typename T, int D>
__device__ __forceinline__ double wide_score(const T* q, const T* bd, int lane) {
  double u = 0.0;
  for (int d = lane; d < D; d += 32) {
    const float x = to_f(q[d]);
    if (x != 0.f) u += (double)x * (double)to_f(x > 0.f ? bd[d] : bd[D + d]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRankThreads)
k_paged_rank(const T* q, const T* bounds, SelArgs a) {
  extern __shared__ float s_score[];                 // [np, rounded up to whole words of 32 pages]
  constexpr int kWords = KVC_PG_MAX_SCORED / 32;
  __shared__ int s_hist[kBins], s_pick[2], s_warp[kRankWarps], s_n[2];
  __shared__ int s_cand[kList];
  __shared__ unsigned long long s_key[kList];
  __shared__ uint32_t s_in[kWords], s_maybe[kWords]; // a bit per page: taken, candidate
  __shared__ float s_lo[kRankWarps], s_hi[kRankWarps];
  kvc_pdl_wait();
  kvc_pdl_release();
  const int kvh = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t pair = (int64_t)b * a.Hkv + kvh;
  int32_t* sel = a.sel + pair * a.n_sel;
  double* exact = a.scores + pair * a.max_pages;
  const float* approx = reinterpret_cast<const float*>(exact);
  const uint32_t max_bits = a.score_max[pair];
  const int np = row_pages(a, b);
  if (np < 0) {
    if (tid == 0) atomicOr(a.err, KVC_DEV_BAD_KVLEN);
    return;
  }
  if (np <= a.n_sel) {
    for (int i = tid; i < a.n_sel; i += kRankThreads) sel[i] = i < np ? i : -1;
    return;
  }
  const float delta = __uint_as_float(max_bits) * 0x1p-16f;
  const int last_others = np - a.recent;             // pages [first, last_others) are ranked, the others always taken
  auto forced = [&](int i) { return i < a.first || i >= last_others; };
  const int need = a.n_sel - a.first - a.recent;     // of those ranked (there are more than that)
  // the scores, their least and largest
  float lo = INFINITY, hi = -INFINITY;
  for (int i0 = tid; i0 < np; i0 += 4 * kRankThreads) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * kRankThreads < np) x[u] = approx[i0 + u * kRankThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kRankThreads;
      if (i >= np) continue;
      s_score[i] = x[u];
      if (!forced(i)) {
        lo = fminf(lo, x[u]);
        hi = fmaxf(hi, x[u]);
      }
    }
  }
  for (int i = tid; i < kBins; i += kRankThreads) s_hist[i] = 0;
  if (tid < kList) s_key[tid] = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
  }
  if (tid == 0) s_n[0] = s_n[1] = 0;
  __syncthreads();
  if (tid == 0) a.score_max[pair] = 0u;              // for the next call (every thread has read it)
  lo = s_lo[lane % kRankWarps];
  hi = s_hi[lane % kRankWarps];
#pragma unroll
  for (int o = kRankWarps / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  // the interval [t0, t1] that holds the last score taken
  float t0 = INFINITY, t1 = INFINITY;
  const float width = (hi - lo) / kBins;
  if (need > 0 && width > 1e-30f && width < INFINITY) {
    const float inv = 1.f / width;
    for (int i = tid; i < np; i += kRankThreads)
      if (!forced(i)) atomicAdd(s_hist + min(kBins - 1, max(0, (int)((s_score[i] - lo) * inv))), 1);
    __syncthreads();
    // thread t has four bins, from the top down; how many scores lie above them
    constexpr int kPer = kBins / kRankThreads;
    int c[kPer], sum = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = s_hist[kBins - 1 - kPer * tid - i];
      sum += c[i];
    }
    int above = block_scan(sum, s_warp, &all);
    if (above < need && need <= above + sum) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (above < need && need <= above + c[i]) s_pick[0] = kBins - 1 - kPer * tid - i;
        above += c[i];
      }
    }
    __syncthreads();
    // a step more on each side than the bin: its edges are rounded
    t0 = lo + (s_pick[0] - 1) * width;
    t1 = lo + (s_pick[0] + 2) * width;
  } else if (need > 0) {
    t0 = t1 = of_key(radix_select<uint32_t>(np, need, s_hist, s_pick, [&](int i) { return key_of(s_score[i]); },
                                            [&](int i) { return !forced(i); }));
  }
  // candidates: scores in [c_lo, c_hi]; above they are in, below out (need = 0: none is in)
  const float dd = delta == delta ? 2.f * delta : INFINITY;
  float c_lo = t0 - dd, c_hi = t1 + dd;
  if (!(c_lo == c_lo) || need <= 0) c_lo = need > 0 ? -INFINITY : INFINITY;     // (infinities in the scores)
  if (!(c_hi == c_hi) || need <= 0) c_hi = INFINITY;
  auto is_cand = [&](int i) { return need > 0 && !forced(i) && !(s_score[i] < c_lo) && !(s_score[i] > c_hi); };
  // a bit per page, a word per warp and step
  const int words = (np + 31) / 32;
  for (int w = warp; w < words; w += kRankWarps) {
    const int i = 32 * w + lane;
    const bool there = i < np;
    const bool cand = there && is_cand(i), in = there && (forced(i) || s_score[i] > c_hi);
    const uint32_t bits_in = __ballot_sync(0xffffffffu, in), bits_maybe = __ballot_sync(0xffffffffu, cand);
    const int n_in = __popc(__ballot_sync(0xffffffffu, in && !forced(i)));
    int at = 0;
    if (lane == 0) {
      s_in[w] = bits_in;
      s_maybe[w] = bits_maybe;
      if (n_in) atomicAdd(&s_n[1], n_in);
      if (bits_maybe) at = atomicAdd(&s_n[0], __popc(bits_maybe));
    }
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(bits_maybe & ((1u << lane) - 1));
    if (cand && at < kList) s_cand[at] = i;
  }
  __syncthreads();
  const int n_cand = s_n[0], rest = need - s_n[1];
  // candidates: none are taken, all, those that rank high in the list, or by radix selection (also where scores are in fp64)
  const bool wide = !(dd < INFINITY);
  const int take = rest <= 0 ? 0 : rest >= n_cand ? 1 : n_cand <= kList && !wide ? 2 : 3;
  auto score = [&](int i, int g, auto f) {
    const int page = a.table[(int64_t)b * a.max_pages + i];
    if (page < 0 || page >= a.n_pages) return -(double)INFINITY;
    return f(q + ((int64_t)b * a.H + kvh * a.G + g) * D, bounds + ((int64_t)page * a.Hkv + kvh) * 2 * D, lane);
  };
  int total;
  if (take == 2) {
    for (int e = warp; e < n_cand * a.G; e += kRankWarps) {
      const int f = e / a.G;
      const uint64_t key = key_of(score(s_cand[f], e - f * a.G, fine_score<T, D>));
      if (lane == 0) atomicMax(&s_key[f], (unsigned long long)key);
    }
    __syncthreads();
    for (int e = tid; e < n_cand; e += kRankThreads) {
      const unsigned long long x = s_key[e];
      const int i = s_cand[e];
      int better = 0;
      for (int f = 0; f < n_cand; ++f) better += s_key[f] > x || (s_key[f] == x && s_cand[f] < i);
      if (better < rest) atomicOr(s_in + (i >> 5), 1u << (i & 31));
    }
    __syncthreads();
  } else if (take == 3) {
    // the fine scores replace the others in the workspace
    for (int w = warp; w < words; w += kRankWarps)
      for (uint32_t left = s_maybe[w]; left; left &= left - 1) {
        const int i = 32 * w + __ffs(left) - 1;
        double best = -INFINITY;
        for (int g = 0; g < a.G; ++g) {
          const double u = wide ? score(i, g, wide_score<T, D>) : score(i, g, fine_score<T, D>);
          if (!(u <= best)) best = u;                // (a NaN comes in, and stays, below)
          if (u != u) break;
        }
        if (lane == 0) exact[i] = best;
      }
    __syncthreads();
    const uint64_t last = radix_select<uint64_t>(np, rest, s_hist, s_pick, [&](int i) { return key_of(exact[i]); }, is_cand);
    const int ties = s_pick[1];                      // of those equal to the last: how many, the lowest columns first
    const int stretch = (words + kRankThreads - 1) / kRankThreads;
    const int w0 = min(words, tid * stretch), w1 = min(words, w0 + stretch);
    int n_tie = 0;
    for (int w = w0; w < w1; ++w)
      for (uint32_t left = s_maybe[w]; left; left &= left - 1) n_tie += key_of(exact[32 * w + __ffs(left) - 1]) == last;
    int t = block_scan(n_tie, s_warp, &total);
    for (int w = w0; w < w1; ++w) {
      uint32_t won = 0;
      for (uint32_t left = s_maybe[w]; left; left &= left - 1) {
        const uint64_t x = key_of(exact[32 * w + __ffs(left) - 1]);
        if (x > last || (x == last && t++ < ties)) won |= left & -left;
      }
      s_in[w] |= won;
    }
    __syncthreads();
  }
  // columns in order: each thread's words, counted, then written a word per warp and step
  const int stretch = (words + kRankThreads - 1) / kRankThreads;
  const int w0 = min(words, tid * stretch), w1 = min(words, w0 + stretch);
  int n = 0;
  for (int w = w0; w < w1; ++w) {
    if (take == 1) s_in[w] |= s_maybe[w];
    n += __popc(s_in[w]);
  }
  int at = block_scan(n, s_warp, &total);
  for (int w = w0; w < w1; ++w) {
    s_maybe[w] = at;                                 // (where the word's first page goes)
    at += __popc(s_in[w]);
  }
  __syncthreads();
  for (int w = warp; w < words; w += kRankWarps) {
    const uint32_t in = s_in[w];
    const int to = (int)s_maybe[w] + __popc(in & ((1u << lane) - 1));
    if (((in >> lane) & 1) && to < a.n_sel) sel[to] = 32 * w + lane;
  }
  for (int i = total + tid; i < a.n_sel; i += kRankThreads) sel[i] = -1;
}

template <typename T, int D>
cudaError_t launch(const kvc_paged* c, const void* q, const SelArgs& a, cudaStream_t s, bool prepare) {
  if (prepare)
    return cudaFuncSetAttribute(k_paged_rank<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, KVC_PG_MAX_SCORED * 4);
  cudaError_t e = cudaSuccess;
  if (a.max_pages <= a.n_sel) {
    // no row has more pages than are taken: nothing to rank
  } else if constexpr (sizeof(T) == 2) {
    // 8 pages a warp; a warp takes four or eight such sets where that still leaves 16 warps an SM (16 rows of up to 2048
    // pages, 8 heads: 65.3 us with eight, 66.0 with four, 64.6 with sixteen, all three launches)
    const int64_t sets = ((int64_t)a.max_pages + 7) / 8 * a.Hkv * a.B;
    const int64_t warps = (int64_t)KVC_PG_GRID * 16;
    const int per_warp = sets >= warps * 8 ? 8 : sets >= warps * 4 ? 4 : 1;
    const int blocks = (a.max_pages + 8 * kMmaWarps * per_warp - 1) / (8 * kMmaWarps * per_warp);
    e = kvc_launch_pdl(k_paged_score_mma<T, D>, dim3(blocks, a.Hkv, a.B), dim3(kMmaWarps * 32), 0, s, (const T*)q,
                       (const T*)c->bounds, a);
  } else {
    const int blocks = (a.max_pages + 8 * 4 - 1) / (8 * 4);
    e = kvc_launch_pdl(k_paged_score<T, D>, dim3(blocks, a.Hkv, a.B), dim3(kScoreThreads), 0, s, (const T*)q,
                       (const T*)c->bounds, a);
  }
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)a.max_pages * 4;
  return kvc_launch_pdl(k_paged_rank<T, D>, dim3(a.Hkv, a.B), dim3(kRankThreads), smem, s, (const T*)q,
                        (const T*)c->bounds, a);
}

cudaError_t dispatch(const kvc_paged* c, const void* q, const SelArgs& a, cudaStream_t s, bool prep) {
  const bool d64 = c->cfg.head_dim == 64;
  switch (c->cfg.dtype) {
    case KVC_F32: return d64 ? launch<float, 64>(c, q, a, s, prep) : launch<float, 128>(c, q, a, s, prep);
    case KVC_F16: return d64 ? launch<__half, 64>(c, q, a, s, prep) : launch<__half, 128>(c, q, a, s, prep);
    default: return d64 ? launch<__nv_bfloat16, 64>(c, q, a, s, prep) : launch<__nv_bfloat16, 128>(c, q, a, s, prep);
  }
}

}  // namespace

cudaError_t kvc_pg_prepare_select(const kvc_paged* c) { return dispatch(c, nullptr, SelArgs{}, 0, true); }

cudaError_t kvc_pg_launch_select(kvc_paged* c, const void* q, int n_sel, int first, int recent, int32_t* sel,
                                 cudaStream_t s) {
  const kvc_paged_config& g = c->cfg;
  const kvc_pg_layout w = kvc_pg_workspace(g);
  SelArgs a{};
  a.table = c->table;
  a.kv_len = c->kv_len;
  a.err = reinterpret_cast<int32_t*>(c->ws);
  a.B = g.batch;
  a.H = g.heads;
  a.Hkv = g.kv_heads;
  a.G = g.heads / g.kv_heads;
  a.ps_log2 = c->ps_log2;
  a.n_pages = g.n_pages;
  a.max_pages = g.max_pages;
  a.scores = reinterpret_cast<double*>(c->ws + w.scores);
  a.score_max = reinterpret_cast<uint32_t*>(c->ws + w.score_max);
  a.n_sel = n_sel;
  a.first = first;
  a.recent = recent;
  a.sel = sel;
  return dispatch(c, q, a, s, false);
}
