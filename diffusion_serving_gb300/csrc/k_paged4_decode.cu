// Attention of few query rows per group over the 4-bit paged store: decode steps, drafted tokens (and chunks of any length,
// by items of up to 16 rows).
//
// Work goes to blocks as in the 16-bit streaming kernel (k_paged_decode.cu, paged_internal.h): a block takes one stretch
// of the line of all rows' tiles, here of 128 slots, through a ring of shared-memory stages.  A page's slots of a head are
// one record, so a tile arrives as one bulk copy per page.  Warps:
//   consumers: sets of four, 32 slots of a tile to a warp; three sets for up to 8 query rows, else two.  They take an item's tiles in
//     turn, or, where there are many items of few tiles, an item each
//   behind them three producers: page numbers and copies, a tile each in turn
//   the last: a helper, the next items' queries and extents
//
// At a quarter of the 16-bit store's bytes a slot, instructions bound this kernel as much as HBM does, so the slots stand in M
// of the m16n8k16 MMAs and the up to 8 (16: two MMAs) query rows in N: an MMA takes 16 slots x 16 dims of codes, twice what it
// would with the queries in M.  Codes become operands in registers, without a pass through shared memory:
//   S^T = K Q^T   A is K.  Any order of dims along k will do if Q has the same, so a lane's four A registers of all
//                 steps are its slot's D/4 neighbouring dims: one 16-byte load per slot, one scale.
//   O^T = V^T P^T A is V^T: pairs of neighbouring slots of one dim.  ldmatrix.trans moves 16-bit units, four codes of
//                 a slot, and leaves a lane one unit of two slots in the halves of a register, so masking the
//                 ith code of both gives such a pair; which dims share an MMA's rows does not matter.
//                 B is P^T: S^T's accumulators, packed, through movmatrix.
// Two codes become two values by a quarter of a shift, a mask-and-or and one multiply-add (paged4_internal.h), as fp16 whichever
// the 16-bit type; every other pair comes out 16 times too small, which its queries make up for, or the outputs (dims
// are rows of O^T, and a row's pairs are of one kind).  Queries are taken as fp16 too, each row times a power of 2.
// The running maximum of a query is looked for only when a weight outgrows its reference by 2^7 (one vote per tile);
// weights are taken 2^8 too large, so that fp16 holds them with full precision down to 2^-22 of the reference, and
// rounded to fp16 once for the product with V (their sum takes them unrounded).
//
// Measured: 32 rows of 234 .. 16384 slots, 8 kv heads of 128, 32 heads, bf16, pages of 16: 76 us, 3.8 TB/s of codes and scales,
// 0.56 of a plain copy (the 16-bit kernel 171 us); 2 rows of 100001 and 131072 slots, pages of 64: 61 us, 4.1 TB/s.  Bound by the
// consumers' instructions and their latency: 324 a warp for 16 slots of 128 dims, issue slots 55 to 58 % busy; of 67 us (32 rows of 8192)
// the copies by themselves take 52, the products with K and with V 18 each, waits and work split 16.  More warps of fewer registers
// (four sets: spills) took 94 us, fewer (two sets) 68; nine stages for six changed nothing.  One row of 490 slots: 8 us.
// Items of few tiles cost a block their beginnings and ends, some 3.5 us one after another; in sets of their own 128 rows of 100 slots
// take 17 us where they took 24, 512 of 300 69 for 96, 128 of 1000 45 for 51; but 128 of 2000, 16 tiles an item, 87 for 77, so it is
// done up to a mean of 8.  A long row among many short ones, whose parts in a block one set then has for itself, is faster for it too:
// one of 131072 slots with 200 of 100 take 72 us (83 shared by all consumers; 36 and 23 in calls of their own), 8 of 32768 with 512 of
// 100 147 (179), 8 of 8000 with 120 of 100 42 (47); but one of 16000 with 31 of 100 16.5 (15.6).
// Up to 16 query rows (two tiles of 8, sets of four warps at 168 registers; heads of 128 spill 176 bytes): 4 tokens of 32 heads over 8,
// heads of 128 and of 64, 1 row of 8000 slots 15 and 10 us, 8 of them 34 and 21, 32 of them 99 and 57 (one token: 10 and 9, 23 and 17,
// 63 and 43); 16 heads over 1, one token: 14 and 9, 15 and 10, 22 and 15.
#include "paged4_internal.h"
#include "paged_finish.h"
#include "paged_ptx.h"

#include <type_traits>

namespace {

using namespace pg;

constexpr int kTile = 128;                        // slots per tile: 32 for each warp of a set
template <int R> constexpr int kSets = R == 8 ? 3 : 2;                 // of four consumers, which take tiles in turn
template <int R> constexpr int kWarps = 4 * kSets<R>;                  // consumer warps
constexpr int kProducers = 3;                     // producer warps, which take tiles in turn
template <int R> constexpr int kThreads = (kWarps<R> + kProducers + 1) * 32;   // + helper
constexpr int kPad = 8;                           // floats: rows of the warps' states on different banks
constexpr int kMinTiles = 4, kItemCost = 2;       // fewest tiles for a block; an item's beginning and end, in tiles
constexpr int kItems = 6;                         // items whose queries are kept
constexpr int kBrief = 8;                         // tiles of a mean item up to which sets of consumers have items of their own
constexpr float kBias = 8.f, kTop = 15.f;         // log2 of a weight at its reference, and of the largest taken

template <int D> constexpr uint32_t kStageBytes = kTile * (D + D / 16);
template <int D, int R> constexpr int kStages = D == 128 ? 6 : 12;     // a multiple of sets and producers: a stage belongs to one of each

template <typename T, int D, int R>
struct Smem {
  uint8_t stage[kStages<D, R>][kStageBytes<D>];   // 128-byte aligned
  float acc[kWarps<R>][R][D + kPad];
  __half q[kItems][R][D + 8];                          // an item's queries (+ 8: rows on different banks)
  float q_scale[kItems][R];                            // of their scores, to log2 units
  float2 ml[kWarps<R>][R];
  int64_t at[kItems][R];                               // rows of the outputs
  int limit[kItems][R];                                // where each query row's keys end (rows that are not there: all)
  kvc_pg_end end[kItems];
  int tiles[kItems];                              // this block's tiles of the item; -1: there is none
  int first[kItems];                              // tiles of this block before them
  int key0[kItems];                                    // position of the first one's first slot
  int len[kItems], open[kItems];                            // where the row's slots end; below this every query row sees all
  uint32_t bad[kStages<D, R>];                    // records of a stage that no page stands behind
  // A stage that is full, by the set whose own item its tile is of (the first, where they share items): a set that has run ahead of
  // the others may be rounds ahead of the ring, where the parity of a barrier they shared would say nothing.
  uint64_t full[kSets<R>][kStages<D, R>], empty[kStages<D, R>];
  uint64_t q_full[kItems], item_empty[2][kItems];  // (the second: of a set's own items)
  WaitCtl wc;
  int flag[kSets<R>];                             // (a set's, or the first for all)
  int fail[kSets<R>][2];                          // a consumer's wait gave up: before an item, within it
};

__device__ __forceinline__ void bulk_load(uint64_t* bar, void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// d += A B, A 16 x 16 (rows lane / 4 in a0, a2; rows lane / 4 + 8 in a1, a3), B 16 x 8
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A query row's 8 elements, VQ lanes to a row, as pg4_query_vec has them; returns what undoes the row's factor.
template <typename T, int VQ>
__device__ __forceinline__ float as_half(uint4& v) {
  float top = pg4_query_top<T>(v, 0.f);
#pragma unroll
  for (int o = 1; o < VQ; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float undo;
  const float f = pg4_query_factor(top, &undo);
  pg4_query_vec<T>(v, f);
  return undo;
}
// (a NaN goes on)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// D / 32 words of codes at a shared address (16 or 8 bytes).
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* r) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_byte(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds_word(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads<R>, 1)
k_paged4_decode(const uint8_t* pool, const T* q, T* __restrict__ out, kvc_pg_args a, uint32_t sixty_four) {
  constexpr int kW = kWarps<R>;        // consumer warps
  constexpr int W = D / 32;            // words of a slot's codes to a lane; pieces of 32 dims
  constexpr int MT = D / 16;           // 16-dim tiles of O^T
  constexpr int NQ = R / 8;            // 8-query tiles
  constexpr int S = kStages<D, R>;
  extern __shared__ uint8_t raw[];
  using Sm = Smem<T, D, R>;
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile WaitCtl* wc = &sm.wc;

  // set-up that touches no global memory runs before the wait for the previous kernel
  if (threadIdx.x < S) {
    for (int i = 0; i < kSets<R>; ++i) mbar_init(&sm.full[i][threadIdx.x], 1);   // its producer's first lane
    mbar_init(&sm.empty[threadIdx.x], 4);             // a set's warps
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kItems) {
    mbar_init(&sm.q_full[threadIdx.x - 32], 32);
    mbar_init(&sm.item_empty[0][threadIdx.x - 32], kW);
    mbar_init(&sm.item_empty[1][threadIdx.x - 32], 4);
  }
  if (threadIdx.x == 64) {
    wait_init(&sm.wc, a.stall_ns);
    for (int i = 0; i < kSets<R>; ++i) sm.fail[i][0] = sm.fail[i][1] = 0;
  }
  fence_mbar_init();
  __syncthreads();
  kvc_pdl_wait();
  kvc_pdl_release();
  kvc_pg_sched<R, kTile> sch;
  sch.init(a, reinterpret_cast<uint8_t*>(&sm) + ((sizeof(Sm) + 15) & ~(size_t)15), kMinTiles, kMinTiles, kItemCost, gridDim.x);
  // Many items of few tiles: sets take items of their own, each every kSets-th, so that one's beginning and end pass beside another's.
  const bool own = sch.stride == 0 && sch.total - sch.n_items * sch.cost <= kBrief * sch.n_items;
  kvc_pg_item it;
  bool more = false;
  if (warp >= kW) more = sch.first(a, blockIdx.x, it);
  const int ps = 1 << a.ps_log2;
  const uint32_t record = (uint32_t)kvc_pg4_record(D, a.ps_log2);

  if (warp >= kW && warp < kW + kProducers) {
    // ---------------- producers: a tile's records, one lane each ----------------
    const int per_tile = kTile >> a.ps_log2;                // 1, 2, 4 or 8
    const int wide = 32 / per_tile;                         // tiles to a window
    // A window: the page numbers of 32 records, one to a lane, from a tile's first on; not looked at before they are used,
    // a window later (tiles are gone sooner than a load is back).  -1 behind the row's end (where -1 is found in a
    // table, it is a bad page).
    auto window = [&](const kvc_pg_item& w, int j) {
      const int key = j * kTile + (lane << a.ps_log2);
      return key < w.r.len ? pg_ld(a.table + (int64_t)w.b * a.max_pages + (key >> a.ps_log2)) : -1;
    };
    int t = 0;                                              // tiles of this block before the item's
    int u = warp - kW, st = u, round = 0;                   // this warp's next tile, its stage, rounds of the ring before it
    int owner = 0;                                          // the set whose own item this is
    uint64_t used = 0;                                      // full barriers that this warp has used an odd number of times
    bool ok = true;
    int ahead = more ? window(it, it.tile0) : -1;
    for (; ok && more;) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      const uint8_t* heads = pool + (int64_t)(a.sub == 1 ? it.vh : it.vh / a.sub) * record;
      kvc_pg_item nx = it;
      more = sch.next(a, nx);
      int pages = ahead, w0 = tile0;                        // the window at hand, and where it begins
      auto look = [&] { return w0 + wide < tile1 ? window(it, w0 + wide) : more ? window(nx, nx.tile0) : -1; };
      ahead = look();
      int j = tile0 + u - t;
      for (; j < tile1; j += kProducers, u += kProducers) {
        if (j >= w0 + wide) {                               // (a window holds a tile of each producer at least)
          w0 += wide;
          pages = ahead;
          ahead = look();
        }
        if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[st], (round - 1) & 1, wc));
        if (!ok) break;
        const int page = __shfl_sync(0xffffffffu, pages, (j - w0) * per_tile + (lane & (per_tile - 1)));
        const bool there = lane < per_tile && j * kTile + (lane << a.ps_log2) < it.r.len;
        const bool fine = there && page >= 0 && page < a.n_pages;
        const unsigned want = __ballot_sync(0xffffffffu, there), good = __ballot_sync(0xffffffffu, fine);
        if (lane == 0) {
          if (want != good) atomicOr(a.err, KVC_DEV_BAD_PAGE);
          sm.bad[st] = want ^ good;
          mbar_expect_tx(&sm.full[owner][st], __popc(good) * record);
        }
        __syncwarp();
        if (fine) bulk_load(&sm.full[owner][st], sm.stage[st] + lane * record, heads + (int64_t)page * a.Hkv * record, record);
        used ^= 1ull << (owner * S + st);
        st += kProducers;
        if (st >= S) {
          st -= S;
          ++round;
        }
      }
      if (w0 + wide < tile1 && more) ahead = window(nx, nx.tile0);   // (the last window held no tile of this warp's)
      t += tile1 - tile0;
      it = nx;
      if (own) owner = owner + 1 < kSets<R> ? owner + 1 : 0;
    }
    if (lane == 0) {   // every load issued here lands before the block releases its shared memory, consumers that gave up or not
      for (int i = 0; i < kSets<R>; ++i)
        for (int x = warp - kW; x < S; x += kProducers) mbar_wait(&sm.full[i][x], ~(uint32_t)(used >> (i * S + x)) & 1, wc, false);
    }
  } else if (warp == kW + kProducers) {
    // ---------------- helper: queries of the items to come ----------------
    constexpr int VQ = D / 8;                               // 16-byte vectors of a query row
    int first = 0, ends = own ? kSets<R> : 1;               // (each set comes to an end of its own)
    for (int n = 0;; ++n) {
      const int b = n % kItems;
      if (n >= kItems && !__all_sync(0xffffffffu, mbar_wait(&sm.item_empty[own][b], (n / kItems - 1) & 1, wc))) break;
      if (!more) {
        if (lane == 0) sm.tiles[b] = -1;
        __syncwarp();
        mbar_arrive(&sm.q_full[b]);
        if (--ends == 0) break;
        continue;
      }
      const kvc_pg_end e = pg_end(a, sch, it);
      int64_t at = 0;
      // Query rows that are not there see the row's slots: what stands behind them must not decide, by a NaN, when the warps look
      // for new references.
      int limit = it.r.len;
      if (lane < R) {
        at = pg_at(a, sch, it, lane < e.rows ? lane : 0);
        sm.at[b][lane] = at;
        if (lane < e.rows) limit = pg_limit(a, it.r, it.k * sch.T + lane / a.Gv);
        sm.limit[b][lane] = limit;
      }
      const int open = __reduce_min_sync(0xffffffffu, limit);
      if (lane == 0) {
        sm.end[b] = e;
        sm.tiles[b] = it.tile1 - it.tile0;
        sm.first[b] = first;
        sm.key0[b] = it.tile0 * kTile;
        sm.len[b] = it.r.len;
        sm.open[b] = open;
      }
      // every load is issued before any is stored
      constexpr int NL = R * VQ / 32;
      uint4 qv[NL];
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        const int v = lane + 32 * x, r = v / VQ, c = v % VQ;
        const int64_t row = __shfl_sync(0xffffffffu, at, r);
        qv[x] = make_uint4(0, 0, 0, 0);
        if (r < e.rows) qv[x] = pg_ld(reinterpret_cast<const uint4*>(q + row * D) + c);
      }
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        const int v = lane + 32 * x;
        const float f = as_half<T, VQ>(qv[x]);
        *reinterpret_cast<uint4*>(&sm.q[b][v / VQ][8 * (v % VQ)]) = qv[x];
        if (v % VQ == 0) sm.q_scale[b][v / VQ] = pg4_score_scale(f, a.scale_log2);
      }
      mbar_arrive(&sm.q_full[b]);
      first += it.tile1 - it.tile0;
      more = sch.next(a, it);
    }
  } else {
    // ---------------- consumers ----------------
    const int g = lane >> 2, quad = lane & 3;
    // Row r of S^T's first eight rows is slot 4 (r / 2) + r % 2 of the warp's sixteen, row r + 8 the slot two behind it, so that
    // a lane's four slots of P^T and V^T are neighbours (one 4-byte load of their scales).
    const int slot = 4 * (g >> 1) + (g & 1);
    const int set = warp >> 2;
    const int r0 = (warp & 3) * 32;                         // the warp's slots within a tile: two blocks of 16,
    const int rec_i = r0 >> a.ps_log2, s0 = r0 & (ps - 1);  // the first one's record, and where it begins in it;
    const bool split = ps == 16;                            // the second is the next record's, or lies behind it
    const int rec_bit[2] = {rec_i, rec_i + split};
    const uint32_t k_off = rec_i * record + (s0 + slot) * (D / 2) + quad * (D / 8);
    const uint32_t ks_off = rec_i * record + ps * D + (s0 + slot) * W + (W == 4 ? quad : quad >> 1);
    const uint32_t vs_off = rec_i * record + ps * (D + W) + s0 + 4 * quad;
    const uint32_t code_step = split ? record : 16 * (D / 2), ks_step = split ? record : 16 * W, vs_step = split ? record : 16;
    // ldmatrix: lanes 8 m .. address the rows of matrix m: slots of the first eight rows or the others, one of two pieces
    const int lr = lane & 7, l_slot = 4 * (lr >> 1) + (lr & 1) + 2 * (lane >> 3 & 1), l_piece = lane >> 4;
    const uint32_t v_off = rec_i * record + (ps + s0 + l_slot) * (D / 2);
    const int l_turn = (l_slot >> 2) & (W - 1);
    auto consume = [&](auto owned) {
    // the warps that share an item: all of the consumers, or (kOwn) a set
    constexpr bool kOwn = decltype(owned)::value;
    constexpr int kN = kOwn ? 4 : kW, kApart = kOwn ? kSets<R> : 1;
    constexpr int kStep = kOwn ? 1 : kSets<R>;              // from a tile of this warp to its next
    const int mates = kOwn ? set : 0, w0 = 4 * mates;
    auto bar = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + mates), "n"(kN * 32) : "memory"); };
    int u = set, st = set;                                  // this warp's next tile and its stage,
    uint32_t phase = 0;                                     // whose barrier's phase it is (kOwn: those of all stages, a bit each)
    for (int n = mates;; n += kApart) {
      const int b = n % kItems;
      bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full[b], (n / kItems) & 1, wc));
      if (!ok) sm.fail[mates][0] = 1;
      bar();                                                // (the last item's states have been read, too)
      if (sm.fail[mates][0]) break;                         // what ends the loop is the same for all that share an item
      const int tiles = sm.tiles[b];
      if (tiles < 0) break;
      uint32_t qb[NQ][2 * W][2];                            // B operands: query 8 x + g, this lane's dims
      float qs[NQ][2];                                      // scales of queries 8 x + 2 quad + {0, 1}
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int kk = 0; kk < 2 * W; ++kk) {
          const uint2 v = *reinterpret_cast<const uint2*>(&sm.q[b][8 * x + g][quad * (D / 4) + 4 * kk]);
          qb[x][kk][0] = v.x;
          qb[x][kk][1] = v.y;
        }
        qs[x][0] = sm.q_scale[b][8 * x + 2 * quad];
        qs[x][1] = sm.q_scale[b][8 * x + 2 * quad + 1];
      }
      const int len = sm.len[b], open = sm.open[b];
      const int t = sm.first[b], t_end = t + tiles;
      if (kOwn) {
        u = t;
        st = u % S;
      }
      int key = sm.key0[b] + r0 + (u - t) * kTile;          // position of the warp's first slot
      float o[NQ][MT][4];
      float nm[NQ][2], l[NQ][2];                            // kBias less the references, sums of this lane's slots
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
        nm[x][0] = nm[x][1] = INFINITY;
        l[x][0] = l[x][1] = 0.f;
      }
      for (; u < t_end; u += kStep, key += kStep * kTile) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[mates][st], kOwn ? phase >> st & 1 : phase, wc));
        if (!ok) break;
        const uint32_t base = smem_u32(sm.stage[st]);
        const uint32_t gone = sm.bad[st];
        if (key < len) {
          // ---- S^T ----
          float sc[2][NQ][4];
          {
            uint32_t k0[2][W], k1[2][W], b0[2], b1[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              lds_words<W>(base + k_off + s * code_step, k0[s]);
              lds_words<W>(base + k_off + 2 * (D / 2) + s * code_step, k1[s]);
              b0[s] = lds_byte(base + ks_off + s * ks_step);
              b1[s] = lds_byte(base + ks_off + 2 * W + s * ks_step);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
              for (int x = 0; x < NQ; ++x) sc[s][x][0] = sc[s][x][1] = sc[s][x][2] = sc[s][x][3] = 0.f;
            }
            kvc_pg4_fast_scale s_0[2], s_1[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              s_0[s] = pg4_fast_scale(b0[s] * 0x101u);
              s_1[s] = pg4_fast_scale(b1[s] * 0x101u);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                uint32_t x0[4], x1[4];
                pg4_fast_pairs(k0[s][w], s_0[s], sixty_four, x0);
                pg4_fast_pairs(k1[s][w], s_1[s], sixty_four, x1);
                const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                  mma(sc[s][x], a0, qb[x][2 * w][0], qb[x][2 * w][1]);
                  mma(sc[s][x], a1, qb[x][2 * w + 1][0], qb[x][2 * w + 1][1]);
                }
              }
            }
          }
          uint32_t v[2][2 * W], vs[2][W];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int x = 0; x < W; x += 2) ldsm_x4_t(base + v_off + 16 * ((x + l_piece) ^ l_turn) + s * code_step, v[s] + 2 * x);
#pragma unroll
            for (int x = 0; x < W; ++x) vs[s][x] = lds_word(base + vs_off + x * ps + s * vs_step);
          }
          // ---- weights: element e of sc is slot (e < 2 ? slot : slot + 2) of a block, query 2 quad + e % 2 ----
          if (key + 32 > open || gone) {                    // some query row does not see all of these slots
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const bool dead = gone >> rec_bit[s] & 1;
              const int first = key + 16 * s;
#pragma unroll
              for (int x = 0; x < NQ; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (dead || first + slot + (e & 2) >= sm.limit[b][8 * x + 2 * quad + (e & 1)]) sc[s][x][e] = -INFINITY;
              }
              // slots at or behind the row's end may hold anything (a scale of NaN included): their values become 0
              const int left = dead ? 0 : len - first - 4 * quad;
              const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1;
#pragma unroll
              for (int x = 0; x < W; ++x) vs[s][x] &= keep;
            }
          }
          uint32_t pb[2][NQ][2];
          float p[2][NQ][4];
          float top = -INFINITY;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
#pragma unroll
              for (int e = 0; e < 4; ++e) p[s][x][e] = fmaf(sc[s][x][e], qs[x][e & 1], nm[x][e & 1]);
              top = max3(top, p[s][x][0], p[s][x][1]);
              top = max3(top, p[s][x][2], p[s][x][3]);
            }
          }
          if (__any_sync(0xffffffffu, !(top <= kTop))) {              // a reference is too low (or not there yet, or a score is NaN)
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float mx = fmaxf(fmaxf(sc[0][x][y], sc[0][x][y + 2]), fmaxf(sc[1][x][y], sc[1][x][y + 2])) * qs[x][y];
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float nm_new = fminf(nm[x][y], kBias - mx);
                const float alpha = nm[x][y] == INFINITY ? 0.f : pg_ex2(nm_new - nm[x][y]);
                nm[x][y] = nm_new;
                l[x][y] *= alpha;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  o[x][i][y] *= alpha;
                  o[x][i][y + 2] *= alpha;
                }
                const float off = nm_new == INFINITY ? 0.f : nm_new;     // (no slot seen so far: every score is -inf)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                  p[s][x][y] = fmaf(sc[s][x][y], qs[x][y], off);
                  p[s][x][y + 2] = fmaf(sc[s][x][y + 2], qs[x][y], off);
                }
              }
            }
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
#pragma unroll
              for (int e = 0; e < 4; ++e) p[s][x][e] = pg_ex2(p[s][x][e]);
              l[x][0] += p[s][x][0] + p[s][x][2];
              l[x][1] += p[s][x][1] + p[s][x][3];
              pb[s][x][0] = transposed(pg4_pack(p[s][x][0], p[s][x][1]));
              pb[s][x][1] = transposed(pg4_pack(p[s][x][2], p[s][x][3]));
            }
          }
          // ---- O^T ----
#pragma unroll
          for (int y = 0; y < W; ++y) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              uint32_t x0[4], x1[4];
              pg4_fast_pairs(v[s][2 * y], pg4_fast_scale(vs[s][y]), sixty_four, x0);
              pg4_fast_pairs(v[s][2 * y + 1], pg4_fast_scale(vs[s][y] >> 16), sixty_four, x1);
              const uint32_t a0[4] = {x0[0], x0[1], x1[0], x1[1]}, a1[4] = {x0[2], x0[3], x1[2], x1[3]};
#pragma unroll
              for (int x = 0; x < NQ; ++x) {
                mma(o[x][2 * y], a0, pb[s][x][0], pb[s][x][1]);
                mma(o[x][2 * y + 1], a1, pb[s][x][0], pb[s][x][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);          // this warp is done with the stage
        if (kOwn) phase ^= 1u << st;
        st += kStep;
        if (st >= S) {
          st -= S;
          if (!kOwn) phase ^= 1;
        }
      }

      // ---- the item's end ----
      if (!ok) sm.fail[mates][1] = 1;
      const kvc_pg_end e = sm.end[b];
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], w);
          const int r = 8 * x + 2 * quad + y;
          if (r >= e.rows) continue;
          // unit g of a piece holds dims 8 (g / 2) + g % 2 + 2 i, its codes i = 0 .. 3
          float* dst = &sm.acc[warp][r][8 * (g >> 1) + (g & 1)];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            dst[32 * (i >> 1) + 4 * (i & 1)] = 16.f * o[x][i][y];
            dst[32 * (i >> 1) + 4 * (i & 1) + 2] = o[x][i][y + 2];
          }
          if (g == 0) sm.ml[warp][r] = make_float2(-nm[x][y], l[x][y]);
        }
      }
      bar();
      if (sm.fail[mates][1]) break;
      pg_finish<T, D, R>(
          a, e, out, &sm.flag[mates], threadIdx.x - 32 * w0, kN * 32, false,
          [&](int r, int d, float* Mp, float* Lp) {
            float2 ml[kN];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kN; ++w) {
              ml[w] = sm.ml[w0 + w][r];
              M = fmaxf(M, ml[w].x);
            }
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kN; ++w) {
              const float wt = pg_weight(ml[w].x, M);
              L = fmaf(wt, ml[w].y, L);
              pg_acc4(x, wt, *reinterpret_cast<const float4*>(&sm.acc[w0 + w][r][d]));
            }
            *Mp = M;
            *Lp = L;
            return x;
          },
          [](int, int, float2*, float4*) {}, [&](int r) { return sm.at[b][r]; }, bar);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[kOwn][b]);
    }
    };
    if (own) consume(std::true_type());
    else consume(std::false_type());
    if (threadIdx.x % 128 == 0 && wc->abort) atomicOr(a.err, KVC_DEV_TIMEOUT);
  }
}

template <typename T, int D, int R>
constexpr size_t kSmemBytes = 128 + ((sizeof(Smem<T, D, R>) + 15) & ~(size_t)15);

template <typename T, int D, int R>
cudaError_t launch(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prepare) {
  static_assert(kSmemBytes<T, D, R> + (4 * KVC_PG_MAX_BATCH + 1) * 4 + 16 <= 232448,
                "shared memory above the 227 KB a block may opt into");
  if (prepare)
    return cudaFuncSetAttribute(k_paged4_decode<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(kSmemBytes<T, D, R> + pg_sched_bytes(KVC_PG_MAX_BATCH)));
  return kvc_launch_pdl(k_paged4_decode<T, D, R>, dim3(KVC_PG_GRID), dim3(kThreads<R>), kSmemBytes<T, D, R> + pg_sched_bytes(a.B), s,
                        (const uint8_t*)c->pages, (const T*)q, (T*)out, a, 0x54005400u);
}

template <typename T>
cudaError_t launch_t(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, bool wide, cudaStream_t s, bool prepare) {
  if (c->cfg.head_dim == 64)
    return wide ? launch<T, 64, 16>(c, a, q, out, s, prepare) : launch<T, 64, 8>(c, a, q, out, s, prepare);
  return wide ? launch<T, 128, 16>(c, a, q, out, s, prepare) : launch<T, 128, 8>(c, a, q, out, s, prepare);
}

}  // namespace

cudaError_t kvc_pg4_prepare_decode(const kvc_paged4* c) {
  const kvc_pg_args a{};
  for (int wide = 0; wide < 2; ++wide) {
    const cudaError_t e = c->cfg.dtype == KVC_F16 ? launch_t<__half>(c, a, nullptr, nullptr, wide, 0, true)
                                                  : launch_t<__nv_bfloat16>(c, a, nullptr, nullptr, wide, 0, true);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// (More than 16 rows to a group make several items of up to 16, each with a pass of its own over the keys.)
cudaError_t kvc_pg4_launch_decode(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  const bool wide = (int64_t)a.max_q * a.Gv > 8;
  return c->cfg.dtype == KVC_F16 ? launch_t<__half>(c, a, q, out, wide, s, false)
                                 : launch_t<__nv_bfloat16>(c, a, q, out, wide, s, false);
}
