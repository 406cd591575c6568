// Attention of many query rows per group over a paged store (16-bit): chunks of prompts, and the
// shared prefix of a batch (sm_103a: tcgen05 + TMEM + TMA).
//
// An item is up to 128 query rows, tokens x heads of one group: the Gv heads of a group sit next to
// one another in q, so one TMA box (64 dims x Gv heads x T tokens) stacks them, and the group's K
// and V tiles are read once for all of them.  Over a shared prefix the tokens of the whole batch
// are stacked, which turns B memory-bound passes over the prefix into one product per tile.
// Items and their 128-slot tiles are shared out evenly among the blocks (paged_internal.h); an item
// that spans blocks leaves partial states.  Where items are many, few blocks share one, and the last of them joins it
// here; where they are few, an item has ten or twenty parts of 64 KB each, and k_paged_join spreads the joining over the
// GPU (the crossing lies near a third of the blocks: 152 / 3 items); a shared prefix's parts go to k_paged_join_prefix.
//
// A block is one CTA per SM (256 threads).  Warps: 0 TMA producer of Q and K, 3 of V, 1 issues
// S = Q K^T (and owns TMEM), 2 issues O += P V, 4-7 softmax, one query row per thread.  TMEM holds
// three S buffers and O (128 columns each); P overwrites S as packed 16-bit pairs and is the A
// operand of the second product.  S(j + 3) waits for PV(j) alone, so QK, softmax and PV of
// neighbouring tiles overlap; the QK issuer also waits until PV(j - 2) is being issued, which keeps
// the tensor queue alternating.  The running max is moved (and O rescaled) only when a tile's sum of
// weights shows that it grew by more than 2^8.
// P is rounded to the store's type, once, for its product (l sums it unrounded): a second product for what the rounding left
// would be half as much tensor work again in a kernel that this bounds.  It adds as much error again as rounding the output does (against
// 64 bits 0.0023 of the output in bf16 where the output's own rounding makes 0.0017, 0.00028 and 0.00021 in fp16).
// K and V arrive page by page: one box per page, 64-dim half and tensor (64 dims x min(page, 64)
// slots); boxes of a tile lie where one 128-slot box would put them (the 128-byte swizzle goes by
// the address).
//
// Bound by the tensor pipe and the softmax warps that feed it.  Chunks of 700 and 1024 tokens over 9000 and 16384 slots,
// causal, 32 heads over 8 kv heads of 128, bf16, pages of 64: 288 us, 1.26 PFLOP/s of visible pairs (0.65 of a library
// matrix product's burst, 0.74 of its sustained rate); the rest is masked halves of diagonal tiles and the last wave's cut
// items.  2 x 1024 tokens over 2 x 16384 slots, not causal: 391 us, 1.36 PFLOP/s, against 377 us of the linear store's
// kernel.  Pages of 16 make it 520 us: 16 copies a tile from one warp, some 80 cycles each, are more than a tile's products
// take.  (Lanes issue in turn; one lane issuing all takes twice that a copy.)  The causal chunks above, replayed by themselves: 268 us
// with pages of 64, 297 of 32, 362 of 16, and 362 of 128.
//
// Every mbarrier wait is bounded (0.5 s); on expiry the block records KVC_DEV_TIMEOUT, lets its TMA
// loads and MMAs land, frees TMEM and returns.
#include "paged_finish.h"
#include "paged_ptx.h"

#include <type_traits>

namespace {

using namespace pg;

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 256;
constexpr int kSBufs = 3, kKStages = 3, kVStages = 2;
constexpr uint32_t kBoxBytes = 64 * 2 * 128;             // 64 dims x 128 slots (or query rows)
constexpr float kRescaleThreshold = 8.0f;                // log2 units
constexpr float kRescaleSum = 256.0f;                    // 2^kRescaleThreshold
constexpr int kBadRing = 8;

// An item as the softmax warps see it (worked out by the PV issuer, which would otherwise idle, so that none of it
// takes registers next to a row of S).
struct Desc {
  int tiles;             // this block's; -1: no more items
  int key0;              // position of the first tile's first slot
  int len, limit0;       // where the keys end, and for the item's first token (causal)
  int i0;                // its first token within the row
  int64_t at0;           // output row of its first token and head
  kvc_pg_end end;
};

template <int D>
struct Smem {
  uint8_t q[D / 64][kBoxBytes];
  uint8_t k[kKStages][D / 64][kBoxBytes];
  uint8_t v[kVStages][D / 64][kBoxBytes];
  uint64_t q_full, q_free;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[kSBufs], p_ready[kSBufs], s_free[kSBufs];
  uint64_t o_done, o_free;
  uint64_t pv_issued[2];
  uint64_t drain[2];
  uint64_t desc_full[2];
  Desc desc[2];
  // boxes of a tile that no page stands behind: read by the softmax warps up to six tiles after the K
  // producer wrote it (QK(T) is issued once softmax(T - 3) is done, and K(T) loaded once QK(T - 3) is)
  uint32_t k_bad[kBadRing];
  uint32_t v_bad[kVStages];
  uint32_t tmem_base;
  WaitCtl wc;
};

// ---- tcgen05 ------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Instruction descriptor, kind::f16: fp32 accumulate, A and B of one 16-bit type (0 fp16, 1 bf16), A K-major, B K-major
// or MN-major, M = 128, N = n.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t fmt, uint32_t b_mn_major, uint32_t n) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (b_mn_major << 16) | ((n >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}
// Shared-memory matrix descriptor (128-byte swizzle) as two words; the K steps of a product add their offset >> 4 to the
// low one (shared addresses stay below 227 KB, so the 14-bit field never carries).
struct SDesc {
  uint32_t lo, hi;
};
__device__ __forceinline__ SDesc sdesc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return {((saddr >> 4) & 0x3FFFu) | (((lbo_bytes >> 4) & 0x3FFFu) << 16),
          ((sbo_bytes >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29)};
}
__device__ __forceinline__ void mma_ss(uint32_t d, SDesc a, SDesc b, uint32_t off, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo + (off >> 4)), "r"(a.hi), "r"(b.lo + (off >> 4)), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, SDesc b, uint32_t b_off, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

#define PG_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                 "=r"(r[i + 6]), "=r"(r[i + 7])
#define PG_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), \
                 "r"(r[i + 7])
#define PG_T8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                 "+r"(r[i + 6]), "+r"(r[i + 7])
// 32 TMEM lanes (one per thread of the warp) x 32 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : PG_R8(0), PG_R8(8), PG_R8(16), PG_R8(24)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      PG_W8(0), PG_W8(8), PG_W8(16), PG_W8(24)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      PG_W8(0), PG_W8(8)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// ties 32 loaded registers to the preceding wait
__device__ __forceinline__ void reg_fence32(uint32_t* r) {
  asm volatile("" : PG_T8(0), PG_T8(8), PG_T8(16), PG_T8(24));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 32 bytes at once (32-byte aligned): the rows that a warp's threads write lie apart, so each store fills a sector
__device__ __forceinline__ void st_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), PG_W8(0) : "memory");
}

template <bool kMask>
__device__ __forceinline__ float row_max(const uint32_t* sr, int valid) {
  float mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBN; i += 2) {
    float x0 = __uint_as_float(sr[i]), x1 = __uint_as_float(sr[i + 1]);
    if (kMask) {
      x0 = i < valid ? x0 : -INFINITY;
      x1 = i + 1 < valid ? x1 : -INFINITY;
    }
    mx[(i >> 1) & 7] = fmax3(mx[(i >> 1) & 7], x0, x1);
  }
  return fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// p = 2^(s c - m), 0 past `valid` when kMask, packed over the first 64 columns of S; returns the row's sum of p.
template <bool kBf16, bool kMask>
__device__ __forceinline__ float exp_pack_store(const uint32_t* sr, int valid, float c, float m_use, uint32_t s_addr) {
  const float2 c2 = make_float2(c, c), nm2 = make_float2(-m_use, -m_use);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c0 = q4 * 32 + 2 * i;
      const float2 t = __ffma2_rn(make_float2(__uint_as_float(sr[c0]), __uint_as_float(sr[c0 + 1])), c2, nm2);
      float x0 = pg_ex2(t.x), x1 = pg_ex2(t.y);
      if (kMask) {
        x0 = c0 < valid ? x0 : 0.f;
        x1 = c0 + 1 < valid ? x1 : 0.f;
      }
      sum[i & 1] = __fadd2_rn(sum[i & 1], make_float2(x0, x1));
      pk[i] = pack2<kBf16>(x0, x1);
    }
    tmem_st16(s_addr + q4 * 16, pk);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_paged_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, T* __restrict__ out, kvc_pg_args a) {
  constexpr bool kBf16 = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
  constexpr int HB = D / 64;
  extern __shared__ uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile WaitCtl* wc = &sm.wc;

  // set-up that touches no global memory runs before the wait for the previous kernel
  if (threadIdx.x == 0) {
    wait_init(&sm.wc, a.stall_ns);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.drain[i], 1);
      mbar_init(&sm.pv_issued[i], 1);
      mbar_init(&sm.desc_full[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&sm.s_full[i], 2);               // the MMAs' commit, and the issuer (for k_bad)
      mbar_init(&sm.p_ready[i], kBM / 32);       // one arrival per softmax warp
      mbar_init(&sm.s_free[i], 1);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, kBM / 32);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.k_full[i], 32);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.v_full[i], 32);
      mbar_init(&sm.v_empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * 3) {
    prefetch_map(&tm_q);
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  // query rows that no box writes (Gv does not divide 128)
  const int stacked = kBM / a.Gv * a.Gv;
  for (int e = stacked * HB * 8 + threadIdx.x; e < kBM * HB * 8; e += kThreads) {
    const int r = e / (HB * 8), h = (e / 8) % HB, c = e % 8;
    *reinterpret_cast<uint4*>(sm.q[h] + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  kvc_pdl_wait();
  kvc_pdl_release();
  kvc_pg_sched<kBM, kBN, true> sch;
  sch.init(a, reinterpret_cast<uint8_t*>(&sm) + ((sizeof(Smem<D>) + 15) & ~(size_t)15), a.phase == 1 ? 1 : KVC_PG_TC_MIN,
           a.phase == 1 ? 1 : KVC_PG_TC_WHOLE, KVC_PG_TC_COST, gridDim.x);
  const int ps = 1 << a.ps_log2;
  kvc_pg_item it;
  bool more = sch.first(a, blockIdx.x, it);

  if (warp == 0 || warp == 3) {
    // ---------------- TMA producers: warp 0 Q and K, warp 3 V ----------------
    const bool kq = warp == 0;
    const int stages = kq ? kKStages : kVStages;
    const CUtensorMap* tm = kq ? &tm_k : &tm_v;
    const int box_log2 = min(a.ps_log2, 6);
    const int per_tile = kBN >> box_log2;               // boxes of one half: 2, 4 or 8
    const uint32_t box_bytes = 128u << box_log2;
    // lane i < per_tile: the page number of the tile's ith box, not looked at before it is used (a tile later); -1 behind
    // the row's end (where -1 is found in a table, it is a bad page: the box lies before the end)
    auto look = [&](const kvc_pg_item& w, int j) {
      const int key = w.r.lo + j * kBN + (lane << box_log2);
      if (lane >= per_tile || key >= w.r.len) return -1;
      const int col = key >> a.ps_log2;
      return a.phase == 1 ? pg_ld(a.prefix_pages + col) : pg_ld(a.table + (int64_t)w.b * a.max_pages + col);
    };
    int t = 0, n = 0, q_issued = 0;
    bool ok = true;
    int page = more ? look(it, it.tile0) : -1;
    for (; ok && more;) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      const int kvh = it.vh / a.sub;
      kvc_pg_item nx = it;
      more = sch.next(a, nx);
      if (kq) {
        if (n >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_free, (n - 1) & 1, wc));   // the last item's last QK
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(&sm.q_full, HB * stacked * 128);
          for (int h = 0; h < HB; ++h)
            tma_load_4d(&tm_q, &sm.q_full, sm.q[h], 64 * h, it.vh * a.Gv, it.r.t0 + it.k * sch.T, 0);
        }
        q_issued = n + 1;
      }
      for (int j = tile0; j < tile1; ++j, ++t) {
        int npage = -1;
        if (j + 1 < tile1) npage = look(it, j + 1);
        else if (more) npage = look(nx, nx.tile0);
        const int st = t % stages;
        uint64_t* full = kq ? &sm.k_full[st] : &sm.v_full[st];
        if (t >= stages)
          ok = __all_sync(0xffffffffu, mbar_wait(kq ? &sm.k_empty[st] : &sm.v_empty[st], (t / stages - 1) & 1, wc));
        if (!ok) break;
        const bool there = lane < per_tile && it.r.lo + j * kBN + (lane << box_log2) < it.r.len;
        const bool fine = there && page >= 0 && page < a.n_pages;
        if (there && !fine) atomicOr(a.err, KVC_DEV_BAD_PAGE);
        if (!fine) page = -1;
        const unsigned good = __ballot_sync(0xffffffffu, fine), bad = __ballot_sync(0xffffffffu, there && !fine);
        if (lane == 0) {
          if (kq) sm.k_bad[t % kBadRing] = bad;
          else sm.v_bad[st] = bad;
          mbar_expect_tx(full, __popc(good) * HB * box_bytes);
        }
        __syncwarp();
        uint8_t* dst = kq ? sm.k[st][0] : sm.v[st][0];
        const int i = lane & (per_tile - 1), h = lane / per_tile;   // box of the tile, half
        const int g = __shfl_sync(0xffffffffu, page, i);
        if (h < HB && g >= 0)
          tma_load_4d(tm, full, dst + h * kBoxBytes + i * box_bytes, 64 * h, kvh,
                      (it.r.lo + j * kBN + (i << box_log2)) & (ps - 1), g);
        __syncwarp();
        if (lane != 0) mbar_arrive(full);
        page = npage;
      }
      ++n;
      it = nx;
    }
    if (lane == 0) {
      // every load this warp issued lands before the CTA's shared memory is released, whether or not a warp gave up (one
      // may yet do so after this warp is through)
      if (q_issued > 0) mbar_wait(&sm.q_full, (q_issued - 1) & 1, wc, false);
      for (int i = max(0, t - stages); i < t; ++i)
        mbar_wait(kq ? &sm.k_full[i % stages] : &sm.v_full[i % stages], (i / stages) & 1, wc, false);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- QK issuer: S(t) = Q K(t)^T into S buffer t % 3 ----------------
    constexpr uint32_t kIdQK = idesc_f16(kBf16 ? 1u : 0u, 0, kBN);
    int t = 0, n = 0;
    bool ok = true;
    for (; ok && more; more = sch.next(a, it)) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full, n & 1, wc));
      for (int j = tile0; ok && j < tile1; ++j, ++t) {
        const int st = t % kKStages, sb = t % kSBufs;
        // K(t) landed, PV(t - 3) has read its P from this buffer, and PV(t - 2) is being issued (two barriers in
        // turn, since a parity could not tell t - 2 from t)
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.k_full[st], (t / kKStages) & 1, wc) &&
                                         (t < kSBufs || mbar_wait(&sm.s_free[sb], (t / kSBufs - 1) & 1, wc)) &&
                                         (t < 2 || mbar_wait(&sm.pv_issued[t & 1], ((t - 2) >> 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const SDesc qd = sdesc(smem_u32(sm.q[0]), 16, 1024), kd = sdesc(smem_u32(sm.k[st][0]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + sb * 128u, qd, kd, (kk >> 2) * kBoxBytes + (kk & 3) * 32, kIdQK, kk > 0);
          mma_commit(&sm.s_full[sb]);
          mma_commit(&sm.k_empty[st]);
          if (j + 1 == tile1) mma_commit(&sm.q_free);
          mbar_arrive(&sm.s_full[sb]);              // (hands k_bad on)
        }
        __syncwarp();
      }
      ++n;
    }
    if (lane == 0) {                                     // (lands before TMEM is freed, whichever warp gave up)
      mma_commit(&sm.drain[0]);
      mbar_wait(&sm.drain[0], 0, wc, false);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- PV issuer: O += P(t) V(t) ----------------
    constexpr uint32_t kIdPV = idesc_f16(kBf16 ? 1u : 0u, 1, D);
    const int box_log2 = min(a.ps_log2, 6);
    int t = 0, n = 0;
    bool ok = true;
    for (;; more = sch.next(a, it)) {
      // (the softmax warps are done with item n - 2's descriptor: o_free of that item has been waited for)
      if (lane == 0) {
        Desc& d = sm.desc[n & 1];
        d.tiles = more ? it.tile1 - it.tile0 : -1;
        if (more) {
          d.key0 = it.r.lo + it.tile0 * kBN;
          d.len = it.r.len;
          d.i0 = it.k * sch.T;
          d.limit0 = pg_limit(a, it.r, d.i0);
          d.at0 = (int64_t)(it.r.t0 + d.i0) * a.H + it.vh * a.Gv;
          d.end = pg_end(a, sch, it);
        }
        mbar_arrive(&sm.desc_full[n & 1]);
      }
      __syncwarp();
      if (!more) break;
      const int tile0 = it.tile0, tile1 = it.tile1;
      if (n >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_free, (n - 1) & 1, wc));   // the epilogue has read O
      for (int j = tile0; ok && j < tile1; ++j, ++t) {
        const int st = t % kVStages, sb = t % kSBufs;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.v_full[st], (t / kVStages) & 1, wc));
        if (!ok) break;
        const int rem = it.r.len - (it.r.lo + j * kBN);
        const uint32_t bad = sm.v_bad[st];
        if (rem < kBN || bad) {
          // slots that hold nothing of the row may hold anything (NaN included): their V rows become 0, so that P = 0
          // there adds exactly nothing
          for (int e = lane; e < kBN * HB * 8; e += 32) {
            const int r = e / (HB * 8), h = (e / 8) % HB, c = e % 8;
            if (r >= rem || ((bad >> (r >> box_log2)) & 1))
              *reinterpret_cast<uint4*>(sm.v[st][h] + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_ready[sb], (t / kSBufs) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const SDesc vd = sdesc(smem_u32(sm.v[st][0]), kBoxBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            mma_ts(tmem + 384u, tmem + sb * 128u + kk * 8, vd, kk * 16 * 128, kIdPV, (j > tile0 || kk > 0) ? 1u : 0u);
            if (kk == 3) mbar_arrive(&sm.pv_issued[t & 1]);
          }
          mma_commit(&sm.s_free[sb]);
          mma_commit(&sm.v_empty[st]);
          if (j + 1 == tile1) mma_commit(&sm.o_done);
        }
        __syncwarp();
      }
      ++n;
      if (!ok) break;
    }
    if (lane == 0) {                                     // (lands before TMEM is freed, whichever warp gave up)
      mma_commit(&sm.drain[1]);
      mbar_wait(&sm.drain[1], 0, wc, false);
    }
    __syncwarp();
  } else {
    // ---------------- softmax and epilogue (one query row per thread) ----------------
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t o_addr = lane_addr + 384u;
    const float c = a.scale_log2;
    const int box_log2 = min(a.ps_log2, 6);
    const bool prefix = a.phase == 2 && sch.lo > 0;
    const int i_tok = r / a.Gv, g = r - i_tok * a.Gv;        // this row's token and head within an item
    int t = 0;
    bool ok = true;
    for (int n = 0;; ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.desc_full[n & 1], (n >> 1) & 1, wc));
      if (!ok) break;
      const volatile Desc& it = sm.desc[n & 1];
      const int tiles = it.tiles;
      if (tiles < 0) break;
      // where this row's keys end; rows that are not there see everything (no mask on their account)
      int limit = 0x3fffffff;
      if (r < it.end.rows)
        limit = a.phase == 1 ? pg_prefix_limit(a, it.i0 + i_tok, it.len) : a.causal ? it.limit0 + i_tok : it.len;
      limit -= it.key0;                                      // (as of the first tile)
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j, ++t) {
        const int sb = t % kSBufs;
        const uint32_t s_addr = lane_addr + sb * 128u;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[sb], (t / kSBufs) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        const int valid = limit - j * kBN;
        const uint32_t bad = sm.k_bad[t % kBadRing];
        auto tile = [&](auto mask) {
          constexpr bool kM = decltype(mask)::value;
          uint32_t sr[128];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) tmem_ld32(s_addr + q4 * 32, sr + q4 * 32);
          tmem_ld_wait();
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) reg_fence32(sr + q4 * 32);
          // After the first tile P is taken against the running reference at once: every p is at most the row's
          // sum, so a sum of at most 2^threshold shows that the maximum did not grow by more, and P stands.
          if (j > 0) {
            const float lsum = exp_pack_store<kBf16, kM>(sr, valid, c, m_ref, s_addr);
            if (!__any_sync(0xffffffffu, !(lsum <= kRescaleSum))) {   // (a NaN sum takes the slow path)
              l += lsum;
              return true;
            }
          }
          const float m_tile = row_max<kM>(sr, valid) * c;
          const bool rescale = m_tile > m_ref + kRescaleThreshold || m_ref == -INFINITY;
          const float m_new = rescale ? m_tile : m_ref;
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          if (j > 0) {
            tmem_st_wait();                             // the optimistic P is overwritten below
            // O may be rescaled only once PV(t - 1) has finished accumulating into it
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_free[(t - 1) % kSBufs], ((t - 1) / kSBufs) & 1, wc)))
              return false;
            tc_fence_after();
            const float alpha = rescale ? pg_ex2(m_ref - m_use) : 1.f;
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t orow[32];
              tmem_ld32(o_addr + q4 * 32, orow);
              tmem_ld_wait();
              reg_fence32(orow);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 y = __fmul2_rn(make_float2(__uint_as_float(orow[i]), __uint_as_float(orow[i + 1])),
                                            make_float2(alpha, alpha));
                orow[i] = __float_as_uint(y.x);
                orow[i + 1] = __float_as_uint(y.y);
              }
              tmem_st32(o_addr + q4 * 32, orow);
            }
            tmem_st_wait();
            l *= alpha;
          }
          m_ref = m_new;
          l += exp_pack_store<kBf16, kM>(sr, valid, c, m_use, s_addr);
          return true;
        };
        if (bad) {                                      // slots without a page: their scores become -inf where they are
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t x[32];
            tmem_ld32(s_addr + q4 * 32, x);
            tmem_ld_wait();
            reg_fence32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bad >> ((q4 * 32 + i) >> box_log2)) & 1) x[i] = 0xff800000u;
            tmem_st32(s_addr + q4 * 32, x);
          }
          tmem_st_wait();
        }
        ok = __all_sync(0xffffffffu, valid >= kBN) ? tile(std::false_type{}) : tile(std::true_type{});
        if (!ok) break;                                 // (the same for the whole warp)
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[sb]);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.o_done, n & 1, wc));
      if (!ok) break;
      tc_fence_after();
      // ---- the item's (or this part's) state: straight out, or left as a partial ----
      const bool real = r < it.end.rows;
      const int64_t at = it.at0 + (int64_t)i_tok * a.H + g;
      bool last = !it.end.left;                          // this block writes the item's output
      if (it.end.left) {
        float* dst = (a.phase == 1 ? a.pre : a.part) + (int64_t)it.end.slot * (kBM * (D + 2));
        float* mine = dst + r * (a.phase == 1 ? D : 8);
        const int step = a.phase == 1 ? 8 : kBM * 8;         // between the row's vectors of 8 dims
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t orow[32];
          __syncwarp();
          tmem_ld32(o_addr + q4 * 32, orow);
          tmem_ld_wait();
          reg_fence32(orow);
          if (real) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_v8(mine + (q4 * 4 + i) * step, orow + 8 * i);
          }
        }
        if (real) *reinterpret_cast<float2*>(dst + kBM * D + 2 * r) = make_float2(m_ref, l);
        if (a.join_here) {
          // Each warp has a ticket of its own for its 32 rows: its stores precede its release, and the last block's
          // loads follow the acquire.
          __syncwarp();
          int* ticket = a.warp_tickets + 4 * it.end.c0 + quad;
          int prev = 0;
          if (lane == 0)
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(prev) : "l"(ticket) : "memory");
          prev = __shfl_sync(0xffffffffu, prev, 0);
          __syncwarp();                                  // (orders lane 0's acquire before the other lanes' loads)
          last = prev == it.end.c1 - it.end.c0;
          if (last && lane == 0) *ticket = 0;            // every block of the item is past it
        }
      }
      if (last) {
        // The prefix's state, then the parts in their order on the line (this block's from TMEM), whichever block is last.
        const int c0 = it.end.left ? it.end.c0 : (int)blockIdx.x, c1 = it.end.left ? it.end.c1 : (int)blockIdx.x;
        auto part = [&](int cc) { return a.part + (int64_t)(2 * cc + (cc == c0 ? 1 : 0)) * (kBM * (D + 2)); };
        auto ml_of = [&](int cc) {
          if (cc == (int)blockIdx.x) return make_float2(m_ref, l);
          return __ldcg(reinterpret_cast<const float2*>(part(cc) + kBM * D + 2 * r));
        };
        float2 pm = make_float2(-INFINITY, 0.f);
        float M = -INFINITY, L = 0.f;
        if (real) {
          if (prefix) pm = __ldcg(a.pre_ml + at);
          M = pm.x;
          for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, ml_of(cc).x);
          L = pg_weight(pm.x, M) * pm.y;
          for (int cc = c0; cc <= c1; ++cc) {
            const float2 ml = ml_of(cc);
            L = fmaf(pg_weight(ml.x, M), ml.y, L);
          }
        }
        const float inv = L != 0.f ? 1.f / L : 0.f;
        const float pw = pm.y != 0.f ? pg_weight(pm.x, M) * inv : 0.f;
        if (a.lse != nullptr && real)
          a.lse[at] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        T* dst = out + at * D;
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t orow[32];
          __syncwarp();
          tmem_ld32(o_addr + q4 * 32, orow);
          tmem_ld_wait();
          reg_fence32(orow);
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
          auto add = [&](float w, const float* src, int step) {    // step: between a row's vectors of 8 dims
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 y = __ldcg(reinterpret_cast<const float4*>(src + (q4 * 4 + (i >> 3)) * step + (i & 7)));
              x[i] = fmaf(w, y.x, x[i]);
              x[i + 1] = fmaf(w, y.y, x[i + 1]);
              x[i + 2] = fmaf(w, y.z, x[i + 2]);
              x[i + 3] = fmaf(w, y.w, x[i + 3]);
            }
          };
          if (pw != 0.f) add(pw, a.pre_o + at * D, 8);
          for (int cc = c0; cc <= c1; ++cc) {
            const float2 ml = real ? ml_of(cc) : make_float2(0.f, 0.f);
            const float w = ml.y != 0.f ? pg_weight(ml.x, M) * inv : 0.f;
            if (cc == (int)blockIdx.x) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = fmaf(w, __uint_as_float(orow[i]), x[i]);
            } else if (w != 0.f) {
              add(w, part(cc) + r * 8, kBM * 8);
            }
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack2<kBf16>(x[2 * i], x[2 * i + 1]);
          if (real) {                                    // (out is 16-byte aligned, no more)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + q4 * 32 + 8 * i) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
      }
      // every TMEM read of O is complete (the next item's first PV may overwrite it), and the descriptor read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sm.wc.abort) atomicOr(a.err, KVC_DEV_TIMEOUT);
}

// More than half of an SM's shared memory even where D = 64 needs less: one block per SM, since each takes all of TMEM.
template <int D>
size_t smem_bytes(int rows) {
  const size_t n = 1024 + ((sizeof(Smem<D>) + 15) & ~(size_t)15) + pg_sched_bytes(rows, true);
  return n < 120 * 1024 ? 120 * 1024 : n;
}

template <typename T, int D>
cudaError_t launch(const kvc_paged* c, kvc_pg_args a, const void* q, void* out, cudaStream_t s, bool prepare) {
  static_assert(sizeof(Smem<D>) + 1024 + 16 + (5 * KVC_PG_MAX_BATCH + KVC_PG_GRID + 3) * 4 + 16 <= 232448,
                "shared memory above the 227 KB a block may opt into");
  if (prepare)
    return cudaFuncSetAttribute(k_paged_tc<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<D>(KVC_PG_MAX_BATCH));
  CUtensorMap tm_q;
  const uint32_t box[4] = {64, (uint32_t)a.Gv, (uint32_t)(kBM / a.Gv), 1};
  if (!kvc_make_box_map(&tm_q, c->cfg.dtype, q, D, a.H, a.n_tokens, 1, box)) return cudaErrorInvalidValue;
  const int rows = a.phase == 1 ? 1 : a.B;
  const int T_tok = kBM / a.Gv;
  a.join_here = a.phase != 1 && 3 * (int64_t)a.Hv * ((a.n_tokens + T_tok - 1) / T_tok) >= KVC_PG_GRID;
  const cudaError_t e = kvc_launch_pdl(k_paged_tc<T, D>, dim3(KVC_PG_GRID), dim3(kThreads), smem_bytes<D>(rows), s, tm_q,
                                 c->tm_k, c->tm_v, (T*)out, a);
  if (e != cudaSuccess || a.phase == 1 || a.join_here) return e;
  // rows that hold no more than an uncut item's slots, and at most an item a block: nothing to join (the launch would take 5 us)
  const int64_t items = (int64_t)a.Hv * ((a.n_tokens + T_tok - 1) / T_tok + a.B);
  if (((int64_t)a.max_pages << a.ps_log2) <= KVC_PG_TC_WHOLE * kBN && items <= KVC_PG_GRID) return e;
  return kvc_pg_launch_join(c, a, out, s);
}

cudaError_t dispatch(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prep) {
  const bool d64 = c->cfg.head_dim == 64;
  if (c->cfg.dtype == KVC_F16) return d64 ? launch<__half, 64>(c, a, q, out, s, prep) : launch<__half, 128>(c, a, q, out, s, prep);
  return d64 ? launch<__nv_bfloat16, 64>(c, a, q, out, s, prep) : launch<__nv_bfloat16, 128>(c, a, q, out, s, prep);
}

}  // namespace

cudaError_t kvc_pg_prepare_tc(const kvc_paged* c) { return dispatch(c, kvc_pg_args{}, nullptr, nullptr, 0, true); }

cudaError_t kvc_pg_launch_tc(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  return dispatch(c, a, q, out, s, false);
}
