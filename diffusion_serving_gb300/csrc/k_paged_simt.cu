// Attention over a paged store in fp32 FMA arithmetic, for any type and shape: the kernel of fp32
// stores, and a cross-check of the tensor-core kernels (KVC_KERNEL_SIMT).
//
// An item's up to 16 query rows (tokens x heads of one group) stream the row's slots in tiles of 64:
//   s = scale q k^T, running max m and sum l per row, O = sum 2^(s - m) v,
// K and V of a tile staged as fp32 in shared memory, 16 threads to a query row.  Work is shared out
// among the blocks by tiles (paged_internal.h), so one long row keeps every SM busy.  Bound by
// shared-memory reads: each FMA of the two products takes a quarter of a 16-byte read per operand.  On a 16-bit store,
// as a cross-check: 1.4 ms where the streaming kernel takes 0.17 (32 rows of up to 16384 slots), 28 ms where the
// tensor-core kernel takes 0.285 (chunks over 16384 slots).
#include "paged_finish.h"

namespace {

constexpr int kR = KVC_PG_SIMT_ROWS, kTS = KVC_PG_SIMT_TILE;
constexpr int kThreads = 256;
constexpr int kLanes = kThreads / kR;                  // threads per query row

template <int D>
struct SimtSmem {
  float k[kTS][D + 4];      // + 4: the 16 slots that a row's threads read at once lie on different banks
  float v[kTS][D];
  float q[kR][D];
  float p[kR][kTS];
  float o[kR][D];
  float ml[kR][2];
  long long slot[kTS];      // slot's row in the pools, -1: left out
  int pos[kTS];             // its position (INT_MAX: left out)
  int limit[kR];
  int flag;
};

__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 u = pg_ld(reinterpret_cast<const float4*>(p));
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
}
template <typename T2, typename T>
__device__ __forceinline__ void load4_16(const T* p, float* x) {
  const uint2 u = pg_ld(reinterpret_cast<const uint2*>(p));
  const T2* h = reinterpret_cast<const T2*>(&u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = (float)h[i].x;
    x[2 * i + 1] = (float)h[i].y;
  }
}
__device__ __forceinline__ void load4(const __half* p, float* x) { load4_16<__half2>(p, x); }
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) { load4_16<__nv_bfloat162>(p, x); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_paged_simt(const T* q, const T* kp, const T* vp, T* __restrict__ out,
             kvc_pg_args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem);
  kvc_pdl_wait();
  kvc_pdl_release();
  kvc_pg_sched<kR, kTS> sch;
  sch.init(a, smem + ((sizeof(SimtSmem<D>) + 15) & ~(size_t)15), 1, 1, 1, gridDim.x);
  const int tid = threadIdx.x;
  const int r = tid / kLanes, ln = tid % kLanes;
  kvc_pg_item it;
  if (!sch.first(a, blockIdx.x, it)) return;
  const int ps = 1 << a.ps_log2;
  auto bar = [] { __syncthreads(); };
  for (bool more = true; more; more = sch.next(a, it)) {
    const int tile0 = it.tile0, tile1 = it.tile1;
    const int n_tok = min(sch.T, it.r.n - it.k * sch.T);
    const int rows = n_tok * a.Gv;
    __syncthreads();
    if (tid < kR) {
      int lim = 0;
      if (tid < rows) {
        const int i = it.k * sch.T + tid / a.Gv;
        // selected pages: the whole row is visible, up to its length
        lim = a.phase == 1 ? pg_prefix_limit(a, i, it.r.len)
                           : a.sel != nullptr ? a.kv_len[it.b] : pg_limit(a, it.r, i);
      }
      sm.limit[tid] = lim;
    }
    for (int e = tid; e < kR * (D / 4); e += kThreads) {
      const int rr = e / (D / 4), d = 4 * (e % (D / 4));
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (rr < rows) {
        const int t = it.r.t0 + it.k * sch.T + rr / a.Gv;
        load4(q + ((int64_t)t * a.H + it.vh * a.Gv + rr % a.Gv) * D + d, x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.q[rr][d + i] = x[i];
    }
    float m = -INFINITY, l = 0.f;
    float o[D / kLanes];
#pragma unroll
    for (int i = 0; i < D / kLanes; ++i) o[i] = 0.f;
    for (int j = tile0; j < tile1; ++j) {
      __syncthreads();
      if (tid < kTS) {
        const int key = it.r.lo + j * kTS + tid;          // position, or place among the selected slots
        long long slot = -1;
        int pos = 0x7fffffff;
        if (key < it.r.len) {
          int col = key >> a.ps_log2;
          if (a.sel != nullptr) col = pg_ld(a.sel + ((int64_t)it.b * a.Hkv + it.vh / a.sub) * a.n_sel + col);
          if (col >= 0) {
            const int page = pg_page(a, it.b, col);
            if (page >= 0) {
              slot = (long long)page * ps + (key & (ps - 1));
              pos = (col << a.ps_log2) + (key & (ps - 1));
            }
          }
        }
        sm.slot[tid] = slot;
        sm.pos[tid] = pos;
      }
      __syncthreads();
      for (int e = tid; e < kTS * (D / 4); e += kThreads) {
        const int s = e / (D / 4), d = 4 * (e % (D / 4));
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        if (sm.slot[s] >= 0) {
          const int64_t off = (sm.slot[s] * a.Hkv + it.vh / a.sub) * D + d;
          load4(kp + off, x);
          load4(vp + off, y);
          // a slot behind the row's length may hold anything: its value must not meet a weight of 0
          const int end = a.sel != nullptr ? sm.limit[0] : it.r.len;
          if (sm.pos[s] >= end) y[0] = y[1] = y[2] = y[3] = 0.f;
        }
        *reinterpret_cast<float4*>(&sm.k[s][d]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&sm.v[s][d]) = make_float4(y[0], y[1], y[2], y[3]);
      }
      __syncthreads();
      float s[kTS / kLanes];
#pragma unroll
      for (int i = 0; i < kTS / kLanes; ++i) s[i] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 qv = *reinterpret_cast<const float4*>(&sm.q[r][d]);
#pragma unroll
        for (int i = 0; i < kTS / kLanes; ++i) {
          const float4 kv = *reinterpret_cast<const float4*>(&sm.k[ln + i * kLanes][d]);
          s[i] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[i]))));
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kTS / kLanes; ++i) {
        s[i] = sm.pos[ln + i * kLanes] < sm.limit[r] ? s[i] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[i]);
      }
#pragma unroll
      for (int w = kLanes / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float m_new = fmaxf(m, mx);
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m - base);               // 0 for the first visible tile
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kTS / kLanes; ++i) {
        const float w = exp2f(s[i] - base);
        sm.p[r][ln + i * kLanes] = w;
        sum += w;
      }
#pragma unroll
      for (int w = kLanes / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l = l * alpha + sum;
      m = m_new;
#pragma unroll
      for (int i = 0; i < D / kLanes; ++i) o[i] *= alpha;
      __syncwarp();
#pragma unroll 4
      for (int t = 0; t < kTS; ++t) {
        const float w = sm.p[r][t];
#pragma unroll
        for (int i = 0; i < D / kLanes; i += 4) {
          const float4 vv = *reinterpret_cast<const float4*>(&sm.v[t][4 * ln + i * kLanes]);
          o[i] = fmaf(w, vv.x, o[i]);
          o[i + 1] = fmaf(w, vv.y, o[i + 1]);
          o[i + 2] = fmaf(w, vv.z, o[i + 2]);
          o[i + 3] = fmaf(w, vv.w, o[i + 3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < D / kLanes; i += 4)
      *reinterpret_cast<float4*>(&sm.o[r][4 * ln + i * kLanes]) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    if (ln == 0) {
      sm.ml[r][0] = m;
      sm.ml[r][1] = l;
    }
    __syncthreads();
    pg_finish<T, D, kR>(
        a, pg_end(a, sch, it), out, &sm.flag, tid, kThreads, a.phase == 2 && sch.lo > 0,
        [&](int rr, int d, float* M, float* L) {
          *M = sm.ml[rr][0];
          *L = sm.ml[rr][1];
          return *reinterpret_cast<const float4*>(&sm.o[rr][d]);
        },
        [&](int rr, int d, float2* ml, float4* y) { pg_load_prefix<D>(a, pg_at(a, sch, it, rr), d, ml, y); },
        [&](int rr) { return pg_at(a, sch, it, rr); }, bar);
  }
}

template <typename T, int D>
cudaError_t launch(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prepare) {
  if (prepare)
    return cudaFuncSetAttribute(k_paged_simt<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(SimtSmem<D>) + 16 + pg_sched_bytes(KVC_PG_MAX_BATCH)));
  const size_t smem = ((sizeof(SimtSmem<D>) + 15) & ~(size_t)15) + pg_sched_bytes(a.phase == 1 ? 1 : a.B);
  return kvc_launch_pdl(k_paged_simt<T, D>, dim3(KVC_PG_GRID_SIMT), dim3(kThreads), smem, s, (const T*)q,
                        (const T*)c->k, (const T*)c->v, (T*)out, a);
}

cudaError_t dispatch(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prep) {
  const bool d64 = c->cfg.head_dim == 64;
  switch (c->cfg.dtype) {
    case KVC_F32: return d64 ? launch<float, 64>(c, a, q, out, s, prep) : launch<float, 128>(c, a, q, out, s, prep);
    case KVC_F16: return d64 ? launch<__half, 64>(c, a, q, out, s, prep) : launch<__half, 128>(c, a, q, out, s, prep);
    default:
      return d64 ? launch<__nv_bfloat16, 64>(c, a, q, out, s, prep) : launch<__nv_bfloat16, 128>(c, a, q, out, s, prep);
  }
}

}  // namespace

cudaError_t kvc_pg_prepare_simt(const kvc_paged* c) { return dispatch(c, kvc_pg_args{}, nullptr, nullptr, 0, true); }

cudaError_t kvc_pg_launch_simt(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  return dispatch(c, a, q, out, s, false);
}
