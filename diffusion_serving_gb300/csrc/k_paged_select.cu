// Which pages a token attends: scores from the pages' key bounds, then the n_select best.
//
//   U(page) = max over the group's heads g of sum_d max(q_gd hi_d, q_gd lo_d)
// bounds every score q_g . k of the page's keys from above.
//
// k_paged_score writes U in fp32 for every (row, kv head, page): a warp per page.  HBM-bound: it
// reads each page's bounds once, 1 / page_size of the bytes of the keys and values themselves.
//
// k_paged_rank, a block per (row, kv head), finds the n_select largest by radix selection on the
// fp32 scores, a byte a pass.  Rounding could swap pages whose scores nearly agree, so it decides
// nothing: with |error| <= delta, a page more than 2 delta above the last one taken is in, one more
// than 2 delta below is out, and those between (mostly the last one alone, and then nothing is left
// to decide) are scored again in fp64 and ranked by that, equal ones by column.
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

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads)
k_paged_score(const T* __restrict__ q, const T* __restrict__ bounds, SelArgs a) {
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
        terms = fmaxf(terms, t);
      }
    }
    if (lane == 0) out[j] = best;
  }
  if (lane == 0 && terms > 0.f) atomicMax(a.score_max + b * a.Hkv + kvh, __float_as_uint(terms));
}

constexpr int kRankThreads = 512;

// order-preserving whole numbers
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);      // -0 counts as 0
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
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRankThreads / 32; ++w) {
    const int v = s_warp[w];
    before += w < warp ? v : 0;
    all += v;
  }
  *total = all;
  return before + y - x;
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

template <typename T, int D>
__global__ void __launch_bounds__(kRankThreads)
k_paged_rank(const T* __restrict__ q, const T* __restrict__ bounds, SelArgs a) {
  extern __shared__ uint32_t s_key[];                // [np]
  __shared__ int s_hist[256], s_pick[2], s_warp[kRankThreads / 32], s_n;
  __shared__ int s_cand[1024];
  kvc_pdl_wait();
  kvc_pdl_release();
  const int kvh = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t pair = (int64_t)b * a.Hkv + kvh;
  int32_t* sel = a.sel + pair * a.n_sel;
  const int np = row_pages(a, b);
  if (np < 0) {
    if (tid == 0) atomicOr(a.err, KVC_DEV_BAD_KVLEN);
    return;
  }
  if (np <= a.n_sel) {
    for (int i = tid; i < a.n_sel; i += kRankThreads) sel[i] = i < np ? i : -1;
    return;
  }
  double* exact = a.scores + pair * a.max_pages;
  const float* approx = reinterpret_cast<const float*>(exact);
  const float delta = __uint_as_float(a.score_max[pair]) * 0x1p-16f;
  for (int i = tid; i < np; i += kRankThreads) s_key[i] = key_of(approx[i]);
  __syncthreads();
  if (tid == 0) a.score_max[pair] = 0u;              // for the next call
  auto forced = [&](int i) { return i < a.first || i >= np - a.recent; };
  const int need = a.n_sel - a.first - a.recent;     // of the others
  uint32_t lo_key = 0xffffffffu, hi_key = 0xffffffffu;   // candidates: lo_key <= key <= hi_key
  uint64_t last = 0;                                 // in fp64: the last candidate taken
  int ties = 0;                                      // of candidates equal to it: how many
  int take = 0;                                      // 0: no candidate is taken, 1: all, 2: by fp64 score
  if (need > 0) {
    const float t = of_key(radix_select<uint32_t>(np, need, s_hist, s_pick, [&](int i) { return s_key[i]; },
                                                  [&](int i) { return !forced(i); }));
    const float dd = delta == delta ? 2.f * delta : INFINITY;
    const float lo_f = t - dd, hi_f = t + dd;
    lo_key = lo_f == lo_f ? key_of(lo_f) : 0u;
    hi_key = hi_f == hi_f ? key_of(hi_f) : 0xffffffffu;
    int sure = 0, cand = 0;
    for (int i = tid; i < np; i += kRankThreads) {
      if (forced(i)) continue;
      sure += s_key[i] > hi_key;
      cand += s_key[i] <= hi_key && s_key[i] >= lo_key;
    }
    int n_sure, n_cand;
    block_scan(sure, s_warp, &n_sure);
    block_scan(cand, s_warp, &n_cand);
    const int rest = need - n_sure;
    take = rest <= 0 ? 0 : rest >= n_cand ? 1 : 2;
    if (take == 2) {
      // fp64 scores of the candidates, a warp each; they replace the fp32 ones in the workspace
      auto score = [&](int i) {
        const int page = a.table[(int64_t)b * a.max_pages + i];
        double best = -INFINITY;
        if (page >= 0 && page < a.n_pages) {
          const T* bd = bounds + ((int64_t)page * a.Hkv + kvh) * 2 * D;
          for (int g = 0; g < a.G; ++g) {
            const T* qp = q + ((int64_t)b * a.H + kvh * a.G + g) * D;
            double u = 0.0;
#pragma unroll
            for (int d = lane; d < D; d += 32) {
              const float x = to_f(qp[d]);
              u = fma((double)x, (double)to_f(x > 0.f ? bd[d] : bd[D + d]), u);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
            best = u > best ? u : best;
          }
        }
        if (lane == 0) exact[i] = best;
      };
      if (tid == 0) s_n = 0;
      __syncthreads();
      if (n_cand <= 1024) {                          // a list of them, so that every warp has work
        for (int i = tid; i < np; i += kRankThreads)
          if (!forced(i) && s_key[i] <= hi_key && s_key[i] >= lo_key) s_cand[atomicAdd(&s_n, 1)] = i;
        __syncthreads();
        for (int e = warp; e < n_cand; e += kRankThreads / 32) score(s_cand[e]);
      } else {
        for (int i = warp; i < np; i += kRankThreads / 32)
          if (!forced(i) && s_key[i] <= hi_key && s_key[i] >= lo_key) score(i);
      }
      __syncthreads();
      auto is_cand = [&](int i) { return !forced(i) && s_key[i] <= hi_key && s_key[i] >= lo_key; };
      last = radix_select<uint64_t>(np, rest, s_hist, s_pick, [&](int i) { return key_of(exact[i]); }, is_cand);
      ties = s_pick[1];
    }
  }
  // columns in order: each thread a stretch of them; ties are given out in order too
  const int stretch = (np + kRankThreads - 1) / kRankThreads;
  const int i0 = min(np, tid * stretch), i1 = min(np, i0 + stretch);
  auto state = [&](int i) {                          // 1 taken, 0 not, 2 one of the ties
    if (forced(i) || s_key[i] > hi_key) return 1;
    if (take == 0 || s_key[i] < lo_key) return 0;
    if (take == 1) return 1;
    const uint64_t x = key_of(exact[i]);
    return x > last ? 1 : x == last ? 2 : 0;
  };
  int n_tie = 0, n_in = 0, total;
  for (int i = i0; i < i1; ++i) n_tie += state(i) == 2;
  int tie = block_scan(n_tie, s_warp, &total);
  const int tie0 = tie;
  for (int i = i0; i < i1; ++i) {
    const int st = state(i);
    n_in += st == 1 || (st == 2 && tie < ties);
    tie += st == 2;
  }
  int at = block_scan(n_in, s_warp, &total);
  tie = tie0;
  for (int i = i0; i < i1; ++i) {
    const int st = state(i);
    const bool in = st == 1 || (st == 2 && tie < ties);
    tie += st == 2;
    if (in && at < a.n_sel) sel[at++] = i;
  }
  // (scores that are not numbers may leave fewer)
  for (int i = total + tid; i < a.n_sel; i += kRankThreads) sel[i] = -1;
}

template <typename T, int D>
cudaError_t launch(const kvc_paged* c, const void* q, const SelArgs& a, cudaStream_t s, bool prepare) {
  if (prepare)
    return cudaFuncSetAttribute(k_paged_rank<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, KVC_PG_MAX_SCORED * 4);
  const int blocks = (a.max_pages + 8 * 4 - 1) / (8 * 4);
  const cudaError_t e = kvc_launch_pdl(k_paged_score<T, D>, dim3(blocks, a.Hkv, a.B), dim3(kScoreThreads), 0, s, (const T*)q,
                                 (const T*)c->bounds, a);
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
