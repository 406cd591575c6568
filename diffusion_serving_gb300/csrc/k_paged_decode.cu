// Attention of few query rows per group over a paged store (16-bit): decode steps, drafted tokens,
// the selected pages of sparse attention, and what follows a shared prefix.
//
// Up to R = 8 or 16 query rows (tokens x heads of one group) share one read of their kv head's K
// and V, so the kernel is HBM-bound: 2 x 2 bytes x D per slot against 4 D R flops.  Work goes to one
// block per SM by tiles of 64 slots (paged_internal.h): a block streams one stretch of the line of
// all rows' tiles, whatever the rows' lengths, through a ring of shared-memory stages that runs on
// across the borders between rows.  Warps:
//   0-7  consumers: a warp takes 16 slots of a tile: S = Q K^T and O += P V as warp-level m16n8k16
//        MMAs (query rows in M, slots or dims in N), online softmax per row in between, P going from
//        accumulators to operands in registers.  Tiles are 32 KB: of 64 slots of 128 dims, which two sets
//        of four warps take in turn (one set's tile takes about as long as HBM needs for one, so two keep
//        ahead of it), or of 128 slots of 64 dims, which all eight share.
//   8,10 producers of K and of V: look up page numbers a tile ahead and issue one TMA box per page:
//        [page_size slots][D / 64][64 dims], 128-byte swizzle, from a 5-d view of the pool.  (A box
//        per 64-dim half would lie free of bank conflicts, where this one's 256-byte rows meet in
//        pairs; but a copy costs the issuing warp some 80 cycles, and for pages of 16 slots even one box a
//        page and tensor from a single warp is too many: heads of 64 4.4 TB/s against 5.5 with two.)
//   9    helper: works out the next items for the consumers (their rows' places, limits, extents) and
//        brings their queries and their shared prefixes' states to shared memory, so that none of it
//        falls between two items.
// At an item's end the warps' states meet in shared memory and go straight out, or, where the item
// spans blocks, to the workspace (pg_finish).
//
// Measured: 32 rows of 234 .. 16384 slots, 8 kv heads of 128, 32 heads, bf16, pages of 16: 171 us, 6.4 TB/s, 0.94 of
// a plain copy; DRAM reads equal the algorithmic bytes, issue slots 22 % busy.  One row of 490 slots: 9.5 us, of which
// 4 go by before the first tile lands (launch, lengths, page numbers, descriptors: a chain of loads).  Heads of 64, the
// same rows: 98 us, 5.6 TB/s (from L2 8.7): a slot's 128 bytes are short pieces to DRAM.

// R = 8 leaves half of M free, and P uses it: rows 8..15 carry what rounding P to 16 bits lost, so
// O is as exact as from fp32 weights at no further MMA.  R = 16 uses all of M, with P rounded once (as much error again
// as the output's own rounding; the rest would take a second set of MMAs).
#include "paged_finish.h"
#include "paged_ptx.h"

namespace {

using namespace pg;

constexpr int kWarps = 8;                         // consumer warps
constexpr int kThreads = (kWarps + 3) * 32;       // + producer of K, helper, producer of V
template <int D> constexpr int kSets = D == 128 ? 2 : 1;                  // of consumers, which take tiles in turn
template <int D> constexpr int kTile = kWarps / kSets<D> * 16;            // slots per tile: 16 for each warp of a set
template <int D> constexpr uint32_t kHalf = kTile<D> * 128u;              // bytes of 64 dims of a tile
constexpr int kPad = 8;                           // floats: rows of the warps' states on different banks
template <int D> constexpr int kMinTiles = 512 / kTile<D>;                // fewest tiles for a block
template <int D> constexpr int kItemCost = 256 / kTile<D>;                // an item's beginning and end, in tiles

template <int D, int R> constexpr int kStages = D == 128 ? (R == 8 ? 5 : 3) : (R == 8 ? 5 : 4);
template <int D> constexpr uint32_t kStageBytes = 2u * (D / 64) * kHalf<D>;   // K and V (32 KB)

template <typename T, int D, int R>
struct Smem {
  uint8_t stage[kStages<D, R>][kStageBytes<D>];   // 1024-byte aligned
  float acc[kWarps][R][D + kPad];
  float pre_o[2][R][D];                           // an item's shared prefix
  T q[2][R][D + 8];                               // its queries (+ 8: rows on different banks)
  float2 ml[kWarps][R];
  float2 pre_ml[2][R];
  int64_t at[2][R];                               // rows of the outputs
  int limit[2][R];                                // where each query row's keys end
  kvc_pg_end end[2];
  int tiles[2];                                   // this block's tiles of the item; -1: there is none
  int keys[2];                                    // slots at or behind this hold nothing of the row
  int pos[kStages<D, R>][kTile<D>];                 // slot positions of a stage, INT_MAX: left out
  uint64_t full[kStages<D, R>], empty[kStages<D, R>];
  uint64_t q_full[2], pre_full[2], item_empty[2];
  WaitCtl wc;
  int flag;
  int fail[2];                                    // a consumer's wait gave up: before an item, within it
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
               const T* q, T* __restrict__ out, kvc_pg_args a) {
  constexpr int HB = D / 64;           // 64-dim boxes per tensor
  constexpr int NT = D / 8;            // n-tiles of 8 dims in O
  constexpr int NR = R / 8;            // query rows per lane
  constexpr int S = kStages<D, R>;
  extern __shared__ uint8_t raw[];
  using Sm = Smem<T, D, R>;
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile WaitCtl* wc = &sm.wc;

  // set-up that touches no global memory runs before the wait for the previous kernel
  if (threadIdx.x < S) {
    mbar_init(&sm.full[threadIdx.x], 64);            // both producers' lanes
    mbar_init(&sm.empty[threadIdx.x], kWarps);
  }
  if (threadIdx.x >= 32 && threadIdx.x < 34) {
    mbar_init(&sm.q_full[threadIdx.x - 32], 32);
    mbar_init(&sm.pre_full[threadIdx.x - 32], 32);
    mbar_init(&sm.item_empty[threadIdx.x - 32], kWarps);
  }
  if (threadIdx.x == 64) {
    wait_init(&sm.wc, a.stall_ns);
    sm.fail[0] = sm.fail[1] = 0;
  }
  if (threadIdx.x == kWarps * 32) {
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  fence_mbar_init();
  __syncthreads();
  kvc_pdl_wait();
  kvc_pdl_release();
  kvc_pg_sched<R, kTile<D>> sch;
  sch.init(a, reinterpret_cast<uint8_t*>(&sm) + ((sizeof(Sm) + 15) & ~(size_t)15), kMinTiles<D>, kMinTiles<D>, kItemCost<D>,
           gridDim.x);
  kvc_pg_item it;
  bool more = false;
  if (warp >= kWarps) more = sch.first(a, blockIdx.x, it);
  const int ps = 1 << a.ps_log2;
  const bool prefix = a.phase == 2 && sch.lo > 0;

  if (warp == kWarps || warp == kWarps + 2) {
    // ---------------- producers: TMA boxes of K (warp 8) and V (warp 10) into the stage ring ----------------
    const bool is_k = warp == kWarps;
    const int box_log2 = min(a.ps_log2, 6);                 // slots per box
    const int per_tile = kTile<D> >> box_log2;               // boxes (of one half and tensor) per tile
    const uint32_t box_bytes = 128u << box_log2;
    const int shared_cols = a.phase == 0 && a.prefix_len != nullptr ? *a.prefix_len >> a.ps_log2 : 0;
    // lane i < per_tile: the table column of the tile's ith box and the page number there, not looked at before it is
    // used (a tile later); column -1: no box
    auto look = [&](const kvc_pg_item& w, int j, int* col, int* page) {
      *col = -1;
      *page = 0;
      const int key = w.r.lo + j * kTile<D> + (lane << box_log2);
      if (lane < per_tile && key < w.r.len) {
        int c = key >> a.ps_log2;
        if (a.sel != nullptr) c = pg_ld(a.sel + ((int64_t)w.b * a.Hkv + w.vh / a.sub) * a.n_sel + c);
        *col = c;
        if (c >= 0) *page = pg_ld((c < shared_cols ? a.prefix_pages : a.table + (int64_t)w.b * a.max_pages) + c);
      }
    };
    int t = 0;
    bool ok = true;
    int col, page;
    if (more) look(it, it.tile0, &col, &page);
    for (; ok && more;) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      const int kvh = a.sub == 1 ? it.vh : it.vh / a.sub;
      kvc_pg_item nx = it;
      more = sch.next(a, nx);
      for (int j = tile0; j < tile1; ++j, ++t) {
        int ncol = -1, npage = 0;                           // the next tile's, in flight meanwhile
        if (j + 1 < tile1) look(it, j + 1, &ncol, &npage);
        else if (more) look(nx, 0, &ncol, &npage);
        const int st = t % S;
        if (t >= S) ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[st], (t / S - 1) & 1, wc));
        if (!ok) break;
        if (col < 0) {
          page = -1;
        } else if (page < 0 || page >= a.n_pages) {
          if (is_k) atomicOr(a.err, KVC_DEV_BAD_PAGE);
          page = -1;
        }
        const unsigned good = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) mbar_expect_tx(&sm.full[st], __popc(good) * HB * box_bytes);
        __syncwarp();
        const int first = it.r.lo + j * kTile<D>;
        if (page >= 0)                                       // (lanes of the tile's boxes alone; at most 8)
          tma_load_5d(is_k ? &tm_k : &tm_v, &sm.full[st],
                      sm.stage[st] + (is_k ? 0 : HB * kHalf<D>) + lane * HB * box_bytes, 0, 0, kvh,
                      (first + (lane << box_log2)) & (ps - 1), page);
        if (is_k) {                                          // positions of the tile's slots
#pragma unroll
          for (int x = 0; x < kTile<D> / 32; ++x) {
            const int s = lane + 32 * x;
            const int c = __shfl_sync(0xffffffffu, col, s >> box_log2), gg = __shfl_sync(0xffffffffu, page, s >> box_log2);
            sm.pos[st][s] = gg >= 0 && first + s < it.r.len ? (c << a.ps_log2) + ((first + s) & (ps - 1)) : 0x7fffffff;
          }
        }
        __syncwarp();
        if (lane != 0) mbar_arrive(&sm.full[st]);
        col = ncol;
        page = npage;
      }
      it = nx;
    }
    if (lane == 0) {   // every load issued here lands before the block releases its shared memory, consumers that gave up or not
      for (int i = max(0, t - S); i < t; ++i) mbar_wait(&sm.full[i % S], (i / S) & 1, wc, false);
    }
  } else if (warp == kWarps + 1) {
    // ---------------- helper: queries and shared prefix of the items to come ----------------
    constexpr int VQ = D / 8;                               // 16-byte vectors of a query row
    for (int n = 0;; ++n) {
      const int b = n & 1;
      if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait(&sm.item_empty[b], (n / 2 - 1) & 1, wc))) break;
      if (!more) {
        if (lane == 0) sm.tiles[b] = -1;
        __syncwarp();
        mbar_arrive(&sm.q_full[b]);
        break;
      }
      const kvc_pg_end e = pg_end(a, sch, it);
      int64_t at = 0;
      if (lane < R) {
        at = pg_at(a, sch, it, lane < e.rows ? lane : 0);
        sm.at[b][lane] = at;
        sm.limit[b][lane] = lane >= e.rows ? 0 : a.sel != nullptr ? a.kv_len[it.b]
                                                                  : pg_limit(a, it.r, it.k * sch.T + lane / a.Gv);
      }
      if (lane == 0) {
        sm.end[b] = e;
        sm.tiles[b] = it.tile1 - it.tile0;
        sm.keys[b] = a.sel != nullptr ? a.kv_len[it.b] : it.r.len;
      }
      // every load is issued before any is stored
      constexpr int NQ = R * VQ / 32, NP = R * D / 128;
      uint4 qv[NQ];
      float4 pv[NP];
      float2 pm = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const int v = lane + 32 * x, r = v / VQ, c = v % VQ;
        const int64_t row = __shfl_sync(0xffffffffu, at, r);
        qv[x] = make_uint4(0, 0, 0, 0);
        if (r < e.rows) qv[x] = pg_ld(reinterpret_cast<const uint4*>(q + row * D) + c);
      }
      if (prefix) {
        if (lane < e.rows) pm = __ldcg(a.pre_ml + at);
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          const int v = lane + 32 * x, r = v / (D / 4), d = 4 * (v % (D / 4));
          const int64_t row = __shfl_sync(0xffffffffu, at, r);
          pv[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < e.rows) pv[x] = __ldcg(reinterpret_cast<const float4*>(a.pre_o + row * D + d));
        }
      }
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const int v = lane + 32 * x;
        *reinterpret_cast<uint4*>(&sm.q[b][v / VQ][8 * (v % VQ)]) = qv[x];
      }
      mbar_arrive(&sm.q_full[b]);
      if (prefix) {
        if (lane < R) sm.pre_ml[b][lane] = pm;
#pragma unroll
        for (int x = 0; x < NP; ++x) {
          const int v = lane + 32 * x;
          *reinterpret_cast<float4*>(&sm.pre_o[b][v / (D / 4)][4 * (v % (D / 4))]) = pv[x];
        }
        mbar_arrive(&sm.pre_full[b]);
      }
      more = sch.next(a, it);
    }
  } else {
    // ---------------- consumers ----------------
    const int hq = lane >> 2, quad = lane & 3;
    const int set = kSets<D> == 1 ? 0 : warp >> 2;          // takes every other tile
    const int r0 = (kSets<D> == 1 ? warp : warp & 3) * 16;                       // this warp's slots of its tiles
    // a tile holds line HB s + h of 128 bytes for slot s and 64-dim half h; its 16-byte chunk c lies at c ^ (line & 7)
    const uint32_t row0 = r0 * HB * 128;
    auto bar = [] { named_bar<1>(kWarps * 32); };
    int t = 0;                                              // tiles of this block before the item's
    for (int n = 0;; ++n) {
      const int b = n & 1;
      bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full[b], (n / 2) & 1, wc));
      if (!ok) sm.fail[0] = 1;
      bar();                                                // (the last item's states have been read, too)
      if (sm.fail[0]) break;                                // what ends the loop is the same for every consumer
      const int tiles = sm.tiles[b];
      if (tiles < 0) break;
      uint32_t qa[D / 16][4];
      int limit[NR];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = hq + 8 * x;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][x] = x < NR ? *reinterpret_cast<const uint32_t*>(&sm.q[b][r % R][16 * kk + 2 * quad]) : 0u;
          qa[kk][x + 2] = x < NR ? *reinterpret_cast<const uint32_t*>(&sm.q[b][r % R][16 * kk + 8 + 2 * quad]) : 0u;
        }
        if (x < NR) limit[x] = sm.limit[b][r % R];
      }
      // slots at or behind `end` hold nothing of the row
      const int end = sm.keys[b];
      float o[NT][4];
      float m[NR], l[NR];
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
      }
      const int t_end = t + tiles;
      for (int u = t; ok && u < t_end; ++u) {
        const int st = u % S;
        // Every warp waits for every tile and frees every stage, the other set's too: a wait by parity has to see each
        // phase of its barrier, since two phases on it could not tell one from the other.
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[st], (u / S) & 1, wc));
        if (!ok) break;
        if (kSets<D> > 1 && (u & 1) != set) {
          if (lane == 0) mbar_arrive(&sm.empty[st]);
          continue;
        }
        const uint32_t kbase = smem_u32(sm.stage[st]) + row0, vbase = kbase + HB * kHalf<D>;
        const int2 pa = *reinterpret_cast<const int2*>(&sm.pos[st][r0 + 2 * quad]);
        const int2 pb = *reinterpret_cast<const int2*>(&sm.pos[st][r0 + 8 + 2 * quad]);
        const int pos[4] = {pa.x, pa.y, pb.x, pb.y};
        const bool any_dead = __any_sync(0xffffffffu, pa.x >= end || pa.y >= end || pb.x >= end || pb.y >= end);
        const bool any_live = !any_dead || __any_sync(0xffffffffu, pa.x < end || pa.y < end || pb.x < end || pb.y < end);
        if (any_live) {
          if (any_dead) {
            // such slots may hold anything (NaN included): their V rows become 0, so that P = 0 there adds nothing
            for (int e = lane; e < 16 * HB * 8; e += 32) {
              const int s = e / (HB * 8), h = (e / 8) % HB, c = e % 8;
              if (sm.pos[st][r0 + s] >= end)
                *reinterpret_cast<uint4*>(sm.stage[st] + HB * kHalf<D> + row0 + (HB * s + h) * 128 + c * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();                            // before TMA reuses the stage
            __syncwarp();
          }
          // S: 16 slots x 16 dims per ldmatrix (slots r0..7 | r0 + 8..15) x (dims 16 kk..+7 | +8..+15)
          float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          {
            const int jj = lane >> 3, i = lane & 7;
            const int slot = (jj >> 1) * 8 + i;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int chunk = (kk & 3) * 2 + (jj & 1);
              uint32_t bk[4];
              const int line = HB * slot + (kk >> 2);
              ldsm_x4(kbase + line * 128 + ((chunk ^ (line & 7)) << 4), bk);
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
              for (int i = 0; i < NT; ++i) {
                o[i][2 * x] *= alpha;
                o[i][2 * x + 1] *= alpha;
                if (NR == 1) {
                  o[i][2] *= alpha;
                  o[i][3] *= alpha;
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
            const int slot = (jj & 1) * 8 + i;
#pragma unroll
            for (int x = 0; x < NT; x += 2) {
              const int chunk = (x & 7) + (jj >> 1);
              uint32_t bv[4];
              const int line = HB * slot + (x >> 3);
              ldsm_x4_t(vbase + line * 128 + ((chunk ^ (line & 7)) << 4), bv);
              mma<T>(o[x], pw, bv[0], bv[1]);
              mma<T>(o[x + 1], pw, bv[2], bv[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);          // this warp is done with the stage
      }
      t = t_end;

      // ---- the item's end ----
      if (ok && prefix) ok = __all_sync(0xffffffffu, mbar_wait(&sm.pre_full[b], (n / 2) & 1, wc));
      if (!ok) sm.fail[1] = 1;
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = hq + 8 * x;
        if (r >= sm.end[b].rows) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float2 y = NR == 1 ? make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3])
                                   : make_float2(o[i][2 * x], o[i][2 * x + 1]);
          *reinterpret_cast<float2*>(&sm.acc[warp][r][8 * i + 2 * quad]) = y;
        }
        if (quad == 0) sm.ml[warp][r] = make_float2(m[x], l[x]);
      }
      bar();
      if (sm.fail[1]) break;
      const kvc_pg_end e = sm.end[b];
      pg_finish<T, D, R>(
          a, e, out, &sm.flag, threadIdx.x, kWarps * 32, prefix,
          [&](int r, int d, float* Mp, float* Lp) {
            float2 ml[kWarps];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              ml[w] = sm.ml[w][r];
              M = fmaxf(M, ml[w].x);
            }
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float wt = pg_weight(ml[w].x, M);
              L = fmaf(wt, ml[w].y, L);
              pg_acc4(x, wt, *reinterpret_cast<const float4*>(&sm.acc[w][r][d]));
            }
            *Mp = M;
            *Lp = L;
            return x;
          },
          [&](int r, int d, float2* ml, float4* y) {
            *ml = sm.pre_ml[b][r];
            *y = *reinterpret_cast<const float4*>(&sm.pre_o[b][r][d]);
          },
          [&](int r) { return sm.at[b][r]; }, bar);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[b]);
    }
    if (threadIdx.x == 0 && wc->abort) atomicOr(a.err, KVC_DEV_TIMEOUT);
  }
}

template <typename T, int D, int R>
constexpr size_t kSmemBytes = 1024 + ((sizeof(Smem<T, D, R>) + 15) & ~(size_t)15);

template <typename T, int D, int R>
cudaError_t launch(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prepare) {
  static_assert(kSmemBytes<T, D, R> + (4 * KVC_PG_MAX_BATCH + 1) * 4 + 16 <= 232448,
                "shared memory above the 227 KB a block may opt into");
  if (prepare)
    return cudaFuncSetAttribute(k_paged_decode<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(kSmemBytes<T, D, R> + pg_sched_bytes(KVC_PG_MAX_BATCH)));
  return kvc_launch_pdl(k_paged_decode<T, D, R>, dim3(KVC_PG_GRID), dim3(kThreads), kSmemBytes<T, D, R> + pg_sched_bytes(a.B), s, c->tm_dk,
                        c->tm_dv, (const T*)q, (T*)out, a);
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

// (More than 16 rows to a group make several items of up to 16, each with a pass of its own over the keys.)
cudaError_t kvc_pg_launch_decode(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  const bool wide = a.max_q * a.Gv > 8;
  return c->cfg.dtype == KVC_F16 ? launch_t<__half>(c, a, q, out, wide, s, false)
                                 : launch_t<__nv_bfloat16>(c, a, q, out, wide, s, false);
}
