// Attention of few query rows per group over a paged store (16-bit): decode steps, drafted tokens,
// the selected pages of sparse attention, and what follows a shared prefix.
//
// Up to R = 8 or 16 query rows (tokens x heads of one group) share one read of their kv head's K
// and V, so the kernel is HBM-bound: 2 x 2 bytes x D per slot against 4 D R flops.  Work goes to one
// block per SM by tiles of 64 slots (paged_internal.h): a block streams one stretch of the line of
// all rows' tiles, whatever the rows' lengths, through a ring of shared-memory stages that runs on
// across the borders between rows.  A producer warp looks up the page numbers a tile ahead and
// issues one TMA box per page, half head and tensor (64 dims x page_size slots, 128-byte swizzle).
// Four consumer warps take 16 slots of each tile: S = Q K^T and O += P V as warp-level m16n8k16
// MMAs (query rows in M, slots or dims in N), online softmax per row in between; P goes from
// accumulators to operands in registers.
//
// R = 8 leaves half of M free, and P uses it: rows 8..15 carry what rounding P to 16 bits lost, so
// O is as exact as from fp32 weights at no further MMA.  R = 16 uses all of M, with P rounded once.
#include "paged_finish.h"
#include "paged_ptx.h"

namespace {

using namespace pg;

constexpr int kWarps = 4;                         // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;       // + one producer warp
constexpr int kTile = kWarps * 16;                // slots per tile
constexpr uint32_t kHalf = kTile * 128u;          // bytes of 64 dims of a tile
constexpr int kMinTiles = 4;

template <int D> constexpr int kStages = D == 128 ? 5 : 9;
template <int D> constexpr uint32_t kStageBytes = 2u * (D / 64) * kHalf;   // K and V

template <int D, int R>
struct Smem {
  uint8_t stage[kStages<D>][kStageBytes<D>];      // 1024-byte aligned
  float acc[kWarps][R][D];
  float ml[kWarps][R][2];
  float own_ml[R][2];
  float row[R][2];
  int pos[kStages<D>][kTile];                     // slot positions of a stage, INT_MAX: left out
  uint64_t full[kStages<D>], empty[kStages<D>];
  WaitCtl wc;
  int flag, abort;
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// d += A B, A 16 x 16 (rows lane / 4 in a0, a2; rows lane / 4 + 8 in a1, a3), B 16 x 8
template <typename T>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two weights as a 16-bit pair, and what the rounding left of them as another
__device__ __forceinline__ uint32_t split2(float x, float y, uint32_t* rest, const __half*) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  *rest = *reinterpret_cast<const uint32_t*>(&l);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t split2(float x, float y, uint32_t* rest, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
  *rest = *reinterpret_cast<const uint32_t*>(&l);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_decode(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const T* __restrict__ q, T* __restrict__ out, kvc_pg_args a) {
  constexpr int HB = D / 64;           // 64-dim boxes per tensor
  constexpr int NT = D / 8;            // n-tiles of 8 dims in O
  constexpr int NR = R / 8;            // query rows per lane
  constexpr int S = kStages<D>;
  extern __shared__ uint8_t raw[];
  Smem<D, R>& sm = *reinterpret_cast<Smem<D, R>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile WaitCtl* wc = &sm.wc;

  // set-up that touches no global memory runs before the wait for the previous kernel
  if (threadIdx.x < S) {
    mbar_init(&sm.full[threadIdx.x], 32);
    mbar_init(&sm.empty[threadIdx.x], kWarps);
  }
  if (threadIdx.x == 0) wait_init(&sm.wc, a.stall_ns);
  if (threadIdx.x == kWarps * 32) {
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  fence_mbar_init();
  __syncthreads();
  kvc_pdl_wait();
  kvc_pdl_release();
  kvc_pg_sched<R, kTile> sch;
  sch.init(a, reinterpret_cast<uint8_t*>(&sm) + ((sizeof(Smem<D, R>) + 15) & ~(size_t)15), kMinTiles);
  long long p = (long long)blockIdx.x * sch.per;
  const long long p_end = min(sch.total, p + sch.per);
  if (p >= p_end) return;
  kvc_pg_item it = sch.at(a, p);
  const int ps = 1 << a.ps_log2;

  if (warp == kWarps) {
    // ---------------- producer: TMA boxes of K and V into the stage ring ----------------
    const int box_log2 = min(a.ps_log2, 6);                 // slots per box
    const int per_tile = kTile >> box_log2;                 // boxes (of one half and tensor) per tile
    const uint32_t box_bytes = 128u << box_log2;
    // lane i < per_tile: the table column and page of the tile's ith box
    auto look = [&](const kvc_pg_item& w, int j, int* col, int* page) {
      *col = -1;
      *page = -1;
      const int key = w.r.lo + j * kTile + (lane << box_log2);
      if (lane < per_tile && key < w.r.len) {
        int c = key >> a.ps_log2;
        if (a.sel != nullptr) c = __ldg(a.sel + ((int64_t)w.b * a.Hkv + w.vh / a.sub) * a.n_sel + c);
        *col = c;
        if (c >= 0) *page = pg_page(a, w.b, c);
      }
    };
    int t = 0;
    bool ok = true;
    int col, page;
    look(it, (int)(p - it.start), &col, &page);
    for (; ok && p < p_end;) {
      const int tile0 = (int)(p - it.start);
      const int tile1 = (int)min((long long)it.tiles, p_end - it.start);
      const int kvh = it.vh / a.sub;
      kvc_pg_item nx = it;
      const bool more = it.start + tile1 < p_end;
      if (more) sch.next(a, nx);
      for (int j = tile0; j < tile1; ++j, ++t) {
        int ncol = -1, npage = -1;                          // the next tile's, in flight meanwhile
        if (j + 1 < tile1) look(it, j + 1, &ncol, &npage);
        else if (more) look(nx, 0, &ncol, &npage);
        const int st = t % S;
        if (t >= S) ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[st], (t / S - 1) & 1, wc));
        if (!ok) break;
        const unsigned good = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) mbar_expect_tx(&sm.full[st], __popc(good) * 2 * HB * box_bytes);
        // positions of the tile's slots
        const int first = it.r.lo + j * kTile;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int s = lane + 32 * i;
          const int c = __shfl_sync(0xffffffffu, col, s >> box_log2), g = __shfl_sync(0xffffffffu, page, s >> box_log2);
          sm.pos[st][s] = g >= 0 && first + s < it.r.len ? (c << a.ps_log2) + ((first + s) & (ps - 1)) : 0x7fffffff;
        }
        uint8_t* dst = sm.stage[st];
        const int i = lane & (per_tile - 1), w = lane / per_tile;   // box of the tile; half and tensor (at most 16 boxes)
        const int g = __shfl_sync(0xffffffffu, page, i);
        if (w < 2 * HB && g >= 0) {
          const int h = w % HB;
          tma_load_4d(w < HB ? &tm_k : &tm_v, &sm.full[st], dst + w * kHalf + i * box_bytes, 64 * h, kvh,
                      (first + (i << box_log2)) & (ps - 1), g);
        }
        __syncwarp();
        if (lane != 0) mbar_arrive(&sm.full[st]);
        col = ncol;
        page = npage;
      }
      p = it.start + tile1;
      if (ok && more) it = nx;
    }
    if (wc->abort && lane == 0) {   // let every load issued here land before the block releases its shared memory
      for (int i = max(0, t - S); i < t; ++i) mbar_wait(&sm.full[i % S], (i / S) & 1, wc, false);
    }
  } else {
    // ---------------- consumers ----------------
    const int hq = lane >> 2, quad = lane & 3;
    const int r0 = warp * 16;                               // this warp's slots of every tile
    auto bar = [] { named_bar<1>(kWarps * 32); };
    int t = 0;
    for (; p < p_end;) {
      const int tile0 = (int)(p - it.start);
      const int tile1 = (int)min((long long)it.tiles, p_end - it.start);
      const int rows = min(sch.T, it.r.n - it.k * sch.T) * a.Gv;
      uint32_t qa[D / 16][4];
      int limit[NR];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = hq + 8 * x;
        const bool real = x < NR && r < rows;
        const int i = it.k * sch.T + (real ? r / a.Gv : 0);
        const T* qp = q + ((int64_t)(it.r.t0 + i) * a.H + it.vh * a.Gv + (real ? r % a.Gv : 0)) * D + 2 * quad;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][x] = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kk)) : 0u;
          qa[kk][x + 2] = real ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kk + 8)) : 0u;
        }
        if (x < NR) limit[x] = !real ? 0 : a.sel != nullptr ? a.kv_len[it.b] : pg_limit(a, it.r, i);
      }
      // slots at or behind `end` hold nothing of the row
      const int end = a.sel != nullptr ? a.kv_len[it.b] : it.r.len;
      float o[NT][4];
      float m[NR], l[NR];
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
      }
      bool ok = true;
      for (int j = tile0; j < tile1; ++j, ++t) {
        const int st = t % S;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[st], (t / S) & 1, wc));
        if (!ok) break;
        const uint32_t kbase = smem_u32(sm.stage[st]), vbase = kbase + HB * kHalf;
        const int2 pa = *reinterpret_cast<const int2*>(&sm.pos[st][r0 + 2 * quad]);
        const int2 pb = *reinterpret_cast<const int2*>(&sm.pos[st][r0 + 8 + 2 * quad]);
        const int pos[4] = {pa.x, pa.y, pb.x, pb.y};
        const bool dead = pa.x >= end || pa.y >= end || pb.x >= end || pb.y >= end;
        const bool any_dead = __any_sync(0xffffffffu, dead);
        const bool any_live = __any_sync(0xffffffffu, pa.x < end || pa.y < end || pb.x < end || pb.y < end);
        if (any_live) {
          if (any_dead) {
            // such slots may hold anything (NaN included): their V rows become 0, so that P = 0 there adds nothing
            for (int e = lane; e < 16 * HB * 8; e += 32) {
              const int s = r0 + e / (HB * 8), h = (e / 8) % HB, c = e % 8;
              if (sm.pos[st][s] >= end)
                *reinterpret_cast<uint4*>(sm.stage[st] + (HB + h) * kHalf + s * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();                            // before TMA reuses the stage
            __syncwarp();
          }
          // S: 16 slots x 16 dims per ldmatrix (slots r0..7 | r0 + 8..15) x (dims 16 kk..+7 | +8..+15)
          float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          {
            const int jj = lane >> 3, i = lane & 7;
            const int slot = r0 + (jj >> 1) * 8 + i;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int chunk = (kk & 3) * 2 + (jj & 1);
              uint32_t bk[4];
              ldsm_x4(kbase + (kk >> 2) * kHalf + slot * 128 + ((chunk ^ (slot & 7)) << 4), bk);
              mma<T>(sc[0], qa[kk], bk[0], bk[1]);
              mma<T>(sc[1], qa[kk], bk[2], bk[3]);
            }
          }
          // online softmax of this lane's rows over the warp's 16 slots
          uint32_t pw[4];
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = pos[e] < limit[x] ? sc[e >> 1][2 * x + (e & 1)] * a.scale_log2 : -INFINITY;
            float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx > m[x]) {                                // the running max grows
              const float alpha = pg_ex2(m[x] - mx);        // 0 on the first visible tile (m = -inf)
              m[x] = mx;
              l[x] *= alpha;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                o[n][2 * x] *= alpha;
                o[n][2 * x + 1] *= alpha;
                if (NR == 1) {
                  o[n][2] *= alpha;
                  o[n][3] *= alpha;
                }
              }
            }
            const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = pg_ex2(y[e] - base);
              l[x] += y[e];
            }
            uint32_t rest0, rest1;
            pw[x] = split2(y[0], y[1], &rest0, (const T*)nullptr);       // slots 2 quad, + 1
            pw[x + 2] = split2(y[2], y[3], &rest1, (const T*)nullptr);   // slots 8 + 2 quad, + 1
            if (NR == 1) {
              pw[1] = rest0;
              pw[3] = rest1;
            }
          }
          // O += P V: (slots r0..7 | r0 + 8..15) x (dims 8 n..+7 | 8 n + 8..+15) per transposed ldmatrix
          {
            const int jj = lane >> 3, i = lane & 7;
            const int slot = r0 + (jj & 1) * 8 + i;
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
              const int chunk = (n & 7) + (jj >> 1);
              uint32_t bv[4];
              ldsm_x4_t(vbase + (n >> 3) * kHalf + slot * 128 + ((chunk ^ (slot & 7)) << 4), bv);
              mma<T>(o[n], pw, bv[0], bv[1]);
              mma<T>(o[n + 1], pw, bv[2], bv[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);          // this warp is done with the stage
      }
      // the block's state: the warps' states, merged
      bar();
      if (threadIdx.x == 0) sm.abort = wc->abort;
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = hq + 8 * x;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 y = NR == 1 ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3])
                                   : make_float2(o[n][2 * x], o[n][2 * x + 1]);
          *reinterpret_cast<float2*>(&sm.acc[warp][r][8 * n + 2 * quad]) = y;
        }
        if (quad == 0) {
          sm.ml[warp][r][0] = m[x];
          sm.ml[warp][r][1] = l[x];
        }
      }
      bar();
      if (sm.abort) break;                                  // (the same for every consumer)
      for (int v = threadIdx.x; v < rows * (D / 4); v += kWarps * 32) {
        const int r = v / (D / 4), d = 4 * (v % (D / 4));
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][r][0]);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          pg_acc4(x, pg_weight(sm.ml[w][r][0], M), *reinterpret_cast<const float4*>(&sm.acc[w][r][d]));
        *reinterpret_cast<float4*>(&sm.acc[0][r][d]) = x;
      }
      if (threadIdx.x < R) {
        const int r = threadIdx.x;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][r][0]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) L = fmaf(pg_weight(sm.ml[w][r][0], M), sm.ml[w][r][1], L);
        sm.own_ml[r][0] = M;
        sm.own_ml[r][1] = L;
      }
      bar();
      pg_finish<T, D, R, kTile>(a, sch, it, &sm.acc[0][0][0], &sm.own_ml[0][0], out, &sm.flag, &sm.row[0][0], threadIdx.x,
                                kWarps * 32, bar);
      p = it.start + tile1;
      if (p < p_end) sch.next(a, it);
    }
    if (threadIdx.x == 0 && wc->abort) atomicOr(a.err, KVC_DEV_TIMEOUT);
  }
}

template <int D, int R>
size_t smem_bytes(int rows) {
  return 1024 + ((sizeof(Smem<D, R>) + 15) & ~(size_t)15) + pg_sched_bytes(rows);
}

template <typename T, int D, int R>
cudaError_t launch(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prepare) {
  static_assert(sizeof(Smem<D, R>) + 1024 + 16 + (KVC_PG_MAX_BATCH + 1) * 8 + 16 + KVC_PG_MAX_BATCH * 16 <= 232448,
                "shared memory above the 227 KB a block may opt into");
  if (prepare)
    return cudaFuncSetAttribute(k_paged_decode<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<D, R>(KVC_PG_MAX_BATCH));
  return kvc_launch_pdl(k_paged_decode<T, D, R>, dim3(KVC_PG_GRID), dim3(kThreads), smem_bytes<D, R>(a.B), s, c->tm_k,
                        c->tm_v, (const T*)q, (T*)out, a);
}

template <typename T>
cudaError_t launch_t(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, bool wide, cudaStream_t s, bool prepare) {
  if (c->cfg.head_dim == 64)
    return wide ? launch<T, 64, 16>(c, a, q, out, s, prepare) : launch<T, 64, 8>(c, a, q, out, s, prepare);
  return wide ? launch<T, 128, 16>(c, a, q, out, s, prepare) : launch<T, 128, 8>(c, a, q, out, s, prepare);
}

}  // namespace

cudaError_t kvc_pg_prepare_decode(const kvc_paged* c) {
  const kvc_pg_args a{};
  for (int wide = 0; wide < 2; ++wide) {
    const cudaError_t e = c->cfg.dtype == KVC_F16 ? launch_t<__half>(c, a, nullptr, nullptr, wide, 0, true)
                                                  : launch_t<__nv_bfloat16>(c, a, nullptr, nullptr, wide, 0, true);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Rows of at most max_q tokens of Gv heads each: max_q * Gv <= 16.
cudaError_t kvc_pg_launch_decode(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  const bool wide = a.max_q * a.Gv > 8;
  return c->cfg.dtype == KVC_F16 ? launch_t<__half>(c, a, q, out, wide, s, false)
                                 : launch_t<__nv_bfloat16>(c, a, q, out, wide, s, false);
}
