// Attention of many query rows per group over the 4-bit paged store: chunks of prompts (sm_103a: tcgen05 + TMEM + TMA).
//
// Items, tiles, their division among blocks and the join of split items are the 16-bit kernel's (k_paged_tc.cu): an item is up to
// 128 query rows, tokens x heads of one group, over tiles of 128 slots.  Records arrive packed, one bulk copy per page; eight
// warps expand them into the swizzled operand tiles that the MMAs read, once per tile for all 128 rows, while the tensor cores and
// the softmax are at the tiles before.  Both are expanded to fp16, whichever the 16-bit type, by one piece of code: exact but for a
// factor of 16 on half of the dims, which K's queries make up for (taken to fp16 too, paged4_internal.h) and O when it leaves
// TMEM.  P is fp16, rounded once.
//
// A block is one CTA per SM (512 threads).  Warps: 0 producer of Q (TMA) and of records, 1 issues S = Q K^T (and owns TMEM),
// 2 issues O += P V, 4-7 softmax, one query row per thread, 8-11 expand K, 12-15 V (and turn an
// item's queries to fp16).  TMEM: two S buffers (128 columns), two P (64),
// O (128).  P has columns of its own, so S(t + 2) waits for the softmax of t alone, not for its product with V, and the softmax,
// which finds S where it was if its weights turn out too large, takes a row by pieces of 32 columns (the 128 registers that
// 512 threads leave it would not hold it whole).
// The running max is moved (and O rescaled) only when a tile's sum of weights shows that it grew by more than 2^8; weights are
// taken 2^6 too large, so that fp16 holds them with full precision down to 2^-20 of the reference.
//
// Measured: chunks of 700 and 1024 tokens over 9000 and 16384 slots, causal, 32 heads over 8 kv heads of 128, bf16: 356 us, 1.03
// PFLOP/s of visible pairs, 352 replayed (the 16-bit kernel 286 to 292, 266 replayed); 1560 tokens over 32760 slots, 12 heads: 340 us, 330
// replayed (the 16-bit kernel 390).  Bound by what a tile of some 2000 cycles
// (the products' own 1024) asks of each scheduler's four warps: 1390 instructions, and of shared memory, 73 % busy: the MMAs' 96 KB,
// 64 KB of expanded operands, 35 KB of records.  1024 tokens over 16384 slots take 262 us; without the expansion 207, without the
// weights 211, without the products 243.  With four expanding warps 277, with sixteen (24 warps) 285, with two softmax warps to 32 rows
// and four expanding 299.  Loops are kept short because the roles share an instruction cache: expanding unrolled 214 us where
// this took 172, weights by 64 columns 175 where by 32 they took 148.
//
// Every mbarrier wait is bounded (0.5 s); on expiry the block records KVC_DEV_TIMEOUT, lets its copies and MMAs land, frees
// TMEM and returns.
#include "paged4_internal.h"
#include "paged_finish.h"
#include "paged_tcgen05.h"

#include <type_traits>

namespace {

using namespace pg;

constexpr int kBN = 128;
constexpr int kThreads = 512;
constexpr int kRaw = 2;                                  // stages of records, of K tiles, of V tiles, S and P buffers
constexpr uint32_t kBoxBytes = 64 * 2 * 128;             // 64 dims x 128 slots (or query rows)
constexpr uint32_t kTmS = 0, kTmP = 256, kTmO = 384;     // TMEM columns
constexpr float kBias = 6.0f;                            // log2 of a weight at its reference
constexpr float kRescaleThreshold = 8.0f;                // log2 units
constexpr float kRescaleSum = 16384.0f;                  // 2^(kBias + kRescaleThreshold)
constexpr int kBadRing = 8;
// Items left over from whole waves are cut among all blocks.  Where that makes more than so many parts each, of rows as long
// as so many tiles a block, a launch of its own (some 10 us) joins them, spread over the GPU, instead of the block that is last:
// 1560 tokens over 32768 slots, 12 heads (156 items, four of them in 38 parts each): 328 us, and 418 joined by the last block;
// 1024 tokens over 8192 slots, 32 heads over 8 (256 items, parts of 1.5 blocks): 159 and 148.
constexpr int kManyParts = 6, kLong = 48;

// An item as the softmax warps see it (worked out by the PV issuer, which would otherwise idle).
struct Desc {
  int tiles;             // this block's; -1: no more items
  int key0;              // position of the first tile's first slot
  int len, limit0;       // where the keys end, and for the item's first token (causal)
  int64_t at0;           // output row of its first token and head
  kvc_pg_end end;
};

template <int D>
struct Smem {
  uint8_t q[D / 64][kBoxBytes];
  uint8_t k[2][D / 64][kBoxBytes];
  uint8_t v[2][D / 64][kBoxBytes];
  uint8_t raw[kRaw][kBN * (D + D / 16)];
  uint64_t q_full, q_ready, q_free;
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_ready[2], pv_done[2];
  uint64_t o_done, o_free;
  uint64_t drain[2];
  uint64_t desc_full[2];
  Desc desc[2];
  // of an item's scores, to log2 units.  Four: item n's are written once the products of item n - 1 with K are done, and then
  // the softmax, two tiles behind them at most, may be about to read item n - 2's (items of a tile each).
  float q_scale[4][kBM];
  // records of a tile that no page stands behind: the producer is at most four tiles ahead of the softmax (two of records,
  // two of K tiles)
  uint32_t bad[kBadRing];
  uint32_t tmem_base;
  WaitCtl wc;
};

// mbar_wait with its polling out of line, so that the roles' loops stay small.
__device__ __noinline__ bool poll(uint64_t* bar, uint32_t parity, volatile WaitCtl* wc, bool honour_abort) {
  return mbar_wait(bar, parity, wc, honour_abort);
}
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, volatile WaitCtl* wc, bool honour_abort = true) {
  return mbar_test_wait(bar, parity) || poll(bar, parity, wc, honour_abort);
}
__device__ __forceinline__ void bulk_load(uint64_t* bar, void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// One warp's 32 slots of a tile: records to rows of operand tiles (64 dims each, 128-byte swizzle).  A lane takes 32 dims of a slot
// at a time; which ones eight neighbouring lanes have is such that neither their loads nor their stores of 16 bytes meet in a bank.
template <int D>
struct Expand {
  static constexpr int W = D / 32;                 // pieces of a slot
  static constexpr int RN = W / 2;                 // rounds of 32 / W slots in a half, 16 slots
  uint32_t code[RN], scale;                        // where a round's codes and its scale stand among a tile's records,
  uint32_t code_step, scale_step;                  // and how much further they do in the second half
  int slot0;                                       // the first slot,
  uint32_t row;                                    // whose row it is in the operand tile, and the pieces' turn in it
  int turn, piece;
  uint32_t scale_round;                            // a scale's way to the next round's

  __device__ __forceinline__ void init(int warp, int lane, int ps_log2, bool is_v) {
    const int ps = 1 << ps_log2;
    const uint32_t record = (uint32_t)kvc_pg4_record(D, ps_log2);
    // Eight neighbouring lanes: two pieces of four slots, or (D = 128) pieces 0 and 1 of two slots and 2 and 3 of the next two.
    piece = W == 4 ? lane >> 1 & 3 : lane & 1;
    slot0 = 32 * warp + (W == 4 ? (lane & 1) | ((lane >> 1 ^ lane >> 2) & 2) | (lane >> 2 & 4) : lane >> 1);
    turn = slot0 & 7;
    row = (piece >> 1) * kBoxBytes + slot0 * 128;
    const int rec = slot0 >> ps_log2, s0 = slot0 & (ps - 1);
#pragma unroll
    for (int n = 0; n < RN; ++n) {
      const int s = s0 + 8 * n;
      code[n] = rec * record + (is_v ? ps + s : s) * (D / 2) + 16 * (is_v ? piece ^ ((s >> 2) & (W - 1)) : piece);
    }
    scale = rec * record + ps * D + (is_v ? ps * W + piece * ps + s0 : s0 * W + piece);
    scale_round = is_v ? 8 : 8 * W;
    code_step = ps == 16 ? record : 16 * (D / 2);
    scale_step = ps == 16 ? record : 2 * scale_round;
  }
  // dead: some slots hold nothing of the row (those from `rem` on, or of a record in `bad`).  They may hold anything, NaN
  // included: they become 0, so that P = 0 adds nothing (a key's score is masked, whatever it is).
  __device__ __forceinline__ void run(uint32_t raw, uint32_t dst, bool dead, int rem, uint32_t bad, int ps_log2, uint32_t base) const {
    uint32_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = dst + row + 16 * (((piece & 1) * 4 + i) ^ turn);
    // (rolled up: three roles' loops share a scheduler's instruction cache)
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t w[RN][4], sb[RN];
#pragma unroll
      for (int n = 0; n < RN; ++n) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[n][0]), "=r"(w[n][1]), "=r"(w[n][2]), "=r"(w[n][3])
                     : "r"(raw + code[n] + h * code_step));
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb[n]) : "r"(raw + scale + h * scale_step + n * scale_round));
      }
      if (dead) {
#pragma unroll
        for (int n = 0; n < RN; ++n) {
          const int slot = slot0 + 16 * h + 8 * n;
          if (slot >= rem || (bad >> (slot >> ps_log2) & 1)) sb[n] = 0;
        }
      }
#pragma unroll
      for (int n = 0; n < RN; ++n) {
        const uint32_t two = sb[n] * 0x101u;
        const kvc_pg4_fast_scale sc = pg4_fast_scale(two);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[4];
          pg4_fast_pairs(w[n][i], sc, base, x);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at[i] + n * (8 * 128)), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                       "r"(x[3])
                       : "memory");
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] += 16 * 128;
    }
  }
};

// p = 2^(s c + off), 0 past `valid` when kMask, of the row's 128 scores at s_addr, packed to p_addr; returns the row's sum of p.
template <bool kMask>
__device__ __forceinline__ float exp_row(uint32_t s_addr, uint32_t p_addr, int valid, float c, float off) {
  const float2 c2 = make_float2(c, c), o2 = make_float2(off, off);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  // (rolled up, without a load ahead: the roles' loops share an instruction cache, and 64 columns a turn take 175 us where these
  // take 148: 1024 tokens over 8192 slots, 32 heads)
#pragma unroll 1
  for (int q4 = 0; q4 < 4; ++q4) {
    uint32_t x[32];
    tmem_ld32(s_addr + q4 * 32, x);
    tmem_ld_wait();
    reg_fence32(x);
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c0 = q4 * 32 + 2 * i;
      const float2 t = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, o2);
      float x0 = pg_ex2(t.x), x1 = pg_ex2(t.y);
      if (kMask) {
        x0 = c0 < valid ? x0 : 0.f;
        x1 = c0 + 1 < valid ? x1 : 0.f;
      }
      sum[i & 1] = __fadd2_rn(sum[i & 1], make_float2(x0, x1));
      pk[i] = pack2<false>(x0, x1);
    }
    tmem_st16(p_addr + q4 * 16, pk);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}
__device__ __forceinline__ float row_max(uint32_t s_addr, int valid) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int q4 = 0; q4 < 4; ++q4) {
    uint32_t x[32];
    tmem_ld32(s_addr + q4 * 32, x);
    tmem_ld_wait();
    reg_fence32(x);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
      x0 = q4 * 32 + i < valid ? x0 : -INFINITY;
      x1 = q4 * 32 + i + 1 < valid ? x1 : -INFINITY;
      mx = fmax3(mx, x0, x1);
    }
  }
  return mx;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_paged4_tc(const __grid_constant__ CUtensorMap tm_q, const uint8_t* pool, T* __restrict__ out, kvc_pg_args a, uint32_t base) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int HB = D / 64;
  extern __shared__ uint8_t raw_smem[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile WaitCtl* wc = &sm.wc;

  // set-up that touches no global memory runs before the wait for the previous kernel
  if (threadIdx.x == 0) {
    wait_init(&sm.wc, a.stall_ns);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_ready, 4);
    mbar_init(&sm.q_free, 1);
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 8);                    // the expanding warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.drain[i], 1);
      mbar_init(&sm.desc_full[i], 1);
      mbar_init(&sm.k_full[i], 4);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 2);                       // the MMAs' commit, and the issuer (for `bad`)
      mbar_init(&sm.p_ready[i], kBM / 32);               // one arrival per softmax warp
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, kBM / 32);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * 3) prefetch_map(&tm_q);
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
  sch.init(a, reinterpret_cast<uint8_t*>(&sm) + ((sizeof(Smem<D>) + 15) & ~(size_t)15), KVC_PG_TC_MIN, KVC_PG_TC_WHOLE, KVC_PG_TC_COST,
           gridDim.x);
  kvc_pg_item it;
  bool more = sch.first(a, blockIdx.x, it);

  if (warp == 0) {
    // ---------------- producer: Q, and a tile's records, one lane each ----------------
    const int per_tile = kBN >> a.ps_log2;                  // 1, 2, 4 or 8
    const uint32_t record = (uint32_t)kvc_pg4_record(D, a.ps_log2);
    // A window: the page numbers of 32 records, one to a lane, from a tile's first on; not looked at before they are used, a
    // window later (a load takes as long as a tile).  -1 behind the row's end (where -1 is found in a table, it is a bad page).
    const int wide = 32 / per_tile;                         // tiles to a window
    auto window = [&](const kvc_pg_item& w, int j) {
      const int key = j * kBN + (lane << a.ps_log2);
      return key < w.r.len ? pg_ld(a.table + (int64_t)w.b * a.max_pages + (key >> a.ps_log2)) : -1;
    };
    int t = 0, n = 0, q_issued = 0;
    bool ok = true;
    int ahead = more ? window(it, it.tile0) : -1;
    for (; ok && more;) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      const uint8_t* heads = pool + (int64_t)(it.vh / a.sub) * record;
      kvc_pg_item nx = it;
      more = sch.next(a, nx);
      if (n >= 1) ok = __all_sync(0xffffffffu, await(&sm.q_free, (n - 1) & 1, wc));   // the last item's last QK
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(&sm.q_full, HB * stacked * 128);
        for (int h = 0; h < HB; ++h)
          tma_load_4d(&tm_q, &sm.q_full, sm.q[h], 64 * h, it.vh * a.Gv, it.r.t0 + it.k * sch.T, 0);
      }
      q_issued = n + 1;
      int pages = -1, at = wide;                            // this window, and the next tile's place in it
      for (int j = tile0; j < tile1; ++j, ++t, ++at) {
        if (at == wide) {
          at = 0;
          pages = ahead;
          if (j + wide < tile1) ahead = window(it, j + wide);
          else if (more) ahead = window(nx, nx.tile0);
        }
        const int st = t % kRaw;
        if (t >= kRaw) ok = __all_sync(0xffffffffu, await(&sm.raw_empty[st], (t / kRaw - 1) & 1, wc));
        if (!ok) break;
        const int page = __shfl_sync(0xffffffffu, pages, at * per_tile + (lane & (per_tile - 1)));
        const bool there = lane < per_tile && j * kBN + (lane << a.ps_log2) < it.r.len;
        const bool fine = there && page >= 0 && page < a.n_pages;
        const unsigned want = __ballot_sync(0xffffffffu, there), good = __ballot_sync(0xffffffffu, fine);
        if (lane == 0) {
          if (want != good) atomicOr(a.err, KVC_DEV_BAD_PAGE);
          sm.bad[t % kBadRing] = want ^ good;
          mbar_expect_tx(&sm.raw_full[st], __popc(good) * record);
        }
        __syncwarp();
        if (fine) bulk_load(&sm.raw_full[st], sm.raw[st] + lane * record, heads + (int64_t)page * a.Hkv * record, record);
        __syncwarp();
      }
      ++n;
      it = nx;
    }
    if (lane == 0) {
      // every load this warp issued lands before the CTA's shared memory is released, whether or not a warp gave up
      if (q_issued > 0) await(&sm.q_full, (q_issued - 1) & 1, wc, false);
      for (int i = max(0, t - kRaw); i < t; ++i) await(&sm.raw_full[i % kRaw], (i / kRaw) & 1, wc, false);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- QK issuer: S(t) = Q K(t)^T ----------------
    constexpr uint32_t kIdQK = idesc_f16(0u, 0, kBN);
    int t = 0, n = 0;
    bool ok = true;
    for (; ok && more; more = sch.next(a, it)) {
      const int tile0 = it.tile0, tile1 = it.tile1;
      ok = __all_sync(0xffffffffu, await(&sm.q_ready, n & 1, wc));
      for (int j = tile0; ok && j < tile1; ++j, ++t) {
        const int sb = t & 1;
        // K(t) is expanded, and the softmax of t - 2 has read this buffer
        ok = __all_sync(0xffffffffu, await(&sm.k_full[sb], (t >> 1) & 1, wc) &&
                                         (t < 2 || await(&sm.p_ready[sb], ((t >> 1) - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const SDesc qd = sdesc(smem_u32(sm.q[0]), 16, 1024), kd = sdesc(smem_u32(sm.k[sb][0]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + kTmS + sb * 128u, qd, kd, (kk >> 2) * kBoxBytes + (kk & 3) * 32, kIdQK, kk > 0);
          mma_commit(&sm.s_full[sb]);
          mma_commit(&sm.k_empty[sb]);
          if (j + 1 == tile1) mma_commit(&sm.q_free);
          mbar_arrive(&sm.s_full[sb]);              // (hands `bad` on)
        }
        __syncwarp();
      }
      ++n;
    }
    if (lane == 0) {                                     // (lands before TMEM is freed, whichever warp gave up)
      mma_commit(&sm.drain[0]);
      await(&sm.drain[0], 0, wc, false);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- PV issuer: O += P(t) V(t) ----------------
    constexpr uint32_t kIdPV = idesc_f16(0u, 1, D);
    int t = 0, n = 0;
    bool ok = true;
    for (;; more = sch.next(a, it)) {
      // (the softmax warps are done with item n - 2's descriptor: o_free of that item has been waited for)
      if (lane == 0) {
        Desc& d = sm.desc[n & 1];
        d.tiles = more ? it.tile1 - it.tile0 : -1;
        if (more) {
          d.key0 = it.tile0 * kBN;
          d.len = it.r.len;
          d.limit0 = pg_limit(a, it.r, it.k * sch.T);
          d.at0 = (int64_t)(it.r.t0 + it.k * sch.T) * a.H + it.vh * a.Gv;
          d.end = pg_end(a, sch, it);
        }
        mbar_arrive(&sm.desc_full[n & 1]);
      }
      __syncwarp();
      if (!more) break;
      const int tile0 = it.tile0, tile1 = it.tile1;
      if (n >= 1) ok = __all_sync(0xffffffffu, await(&sm.o_free, (n - 1) & 1, wc));   // the epilogue has read O
      for (int j = tile0; ok && j < tile1; ++j, ++t) {
        const int sb = t & 1;
        ok = __all_sync(0xffffffffu, await(&sm.v_full[sb], (t >> 1) & 1, wc) && await(&sm.p_ready[sb], (t >> 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const SDesc vd = sdesc(smem_u32(sm.v[sb][0]), kBoxBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts(tmem + kTmO, tmem + kTmP + sb * 64u + kk * 8, vd, kk * 16 * 128, kIdPV, (j > tile0 || kk > 0) ? 1u : 0u);
          mma_commit(&sm.pv_done[sb]);
          mma_commit(&sm.v_empty[sb]);
          if (j + 1 == tile1) mma_commit(&sm.o_done);
        }
        __syncwarp();
      }
      ++n;
      if (!ok) break;
    }
    if (lane == 0) {                                     // (lands before TMEM is freed, whichever warp gave up)
      mma_commit(&sm.drain[1]);
      await(&sm.drain[1], 0, wc, false);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---------------- expanding warps: records to operand tiles ----------------
    const bool is_v = warp >= 12;
    Expand<D> e;
    e.init(warp & 3, lane, a.ps_log2, is_v);
    uint64_t *full = is_v ? sm.v_full : sm.k_full, *empty = is_v ? sm.v_empty : sm.k_empty;
    const uint32_t tiles = smem_u32(is_v ? sm.v[0][0] : sm.k[0][0]);
    int t = 0, n = 0;
    bool ok = true;
    for (; ok && more; more = sch.next(a, it), ++n) {
      if (is_v) {
        // ---- the item's queries to fp16, where they are: a row to a lane ----
        ok = __all_sync(0xffffffffu, await(&sm.q_full, n & 1, wc));
        if (!ok) break;
        const int r = (warp - 12) * 32 + lane;
        float top = 0.f, undo;
#pragma unroll 1
        for (int h = 0; h < HB; ++h) {
#pragma unroll
          for (int c = 0; c < 8; ++c) top = pg4_query_top<T>(*reinterpret_cast<const uint4*>(sm.q[h] + r * 128 + 16 * (c ^ (r & 7))), top);
        }
        const float f = pg4_query_factor(top, &undo);
        sm.q_scale[n & 3][r] = pg4_score_scale(undo, a.scale_log2);
#pragma unroll 1
        for (int h = 0; h < HB; ++h) {
#pragma unroll 4
          for (int c = 0; c < 8; ++c) {
            uint4* p = reinterpret_cast<uint4*>(sm.q[h] + r * 128 + 16 * (c ^ (r & 7)));
            uint4 v = *p;
            pg4_query_vec<T>(v, f);
            *p = v;
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready);
      }
      for (int j = it.tile0; j < it.tile1; ++j, ++t) {
        const int st = t % kRaw, buf = t & 1;
        ok = __all_sync(0xffffffffu, await(&sm.raw_full[st], (t / kRaw) & 1, wc) &&
                                         (t < 2 || await(&empty[buf], ((t >> 1) - 1) & 1, wc)));
        if (!ok) break;
        const int rem = it.r.len - j * kBN;
        const uint32_t bad = sm.bad[t % kBadRing];
        e.run(smem_u32(sm.raw[st]), tiles + buf * HB * kBoxBytes, rem < kBN || bad, rem, bad, a.ps_log2, base);
        fence_proxy_async();                             // (before the MMAs read the tile, and a copy overwrites the records)
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[buf]);
          mbar_arrive(&sm.raw_empty[st]);
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- softmax and epilogue (one query row per thread) ----------------
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t o_addr = lane_addr + kTmO;
    const int i_tok = r / a.Gv, g = r - i_tok * a.Gv;        // this row's token and head within an item
    int t = 0;
    bool ok = true;
    for (int n = 0;; ++n) {
      ok = __all_sync(0xffffffffu, await(&sm.desc_full[n & 1], (n >> 1) & 1, wc));
      if (!ok) break;
      const volatile Desc& it = sm.desc[n & 1];
      const int tiles = it.tiles;
      if (tiles < 0) break;
      // where this row's keys end; rows that are not there see everything (no mask on their account)
      int limit = 0x3fffffff;
      if (r < it.end.rows) limit = a.causal ? it.limit0 + i_tok : it.len;
      limit -= it.key0;                                      // (as of the first tile)
      float m_ref = -INFINITY, l = 0.f, c = 0.f;
      for (int j = 0; j < tiles; ++j, ++t) {
        const int sb = t & 1;
        const uint32_t s_addr = lane_addr + kTmS + sb * 128u, p_addr = lane_addr + kTmP + sb * 64u;
        // S(t) is there, and PV(t - 2) has read this buffer's P
        ok = __all_sync(0xffffffffu, await(&sm.s_full[sb], (t >> 1) & 1, wc) &&
                                         (t < 2 || await(&sm.pv_done[sb], ((t >> 1) - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (j == 0) c = sm.q_scale[n & 3][r];
        const int valid = limit - j * kBN;
        const uint32_t bad = sm.bad[t % kBadRing];
        if (bad) {                                      // slots without a page: their scores become -inf where they are
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t x[32];
            tmem_ld32(s_addr + q4 * 32, x);
            tmem_ld_wait();
            reg_fence32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bad >> ((q4 * 32 + i) >> a.ps_log2)) & 1) x[i] = 0xff800000u;
            tmem_st32(s_addr + q4 * 32, x);
          }
          tmem_st_wait();
        }
        // After the first tile P is taken against the running reference at once: every p is at most the row's
        // sum, so a sum of at most 2^threshold shows that the maximum did not grow by more, and P stands.
        bool stands = false;
        if (j > 0) {
          const float lsum = __all_sync(0xffffffffu, valid >= kBN) ? exp_row<false>(s_addr, p_addr, valid, c, kBias - m_ref)
                                                                   : exp_row<true>(s_addr, p_addr, valid, c, kBias - m_ref);
          stands = !__any_sync(0xffffffffu, !(lsum <= kRescaleSum));      // (not with a NaN sum)
          if (stands) l += lsum;
        }
        if (!stands) {
          const float m_tile = row_max(s_addr, valid) * c;
          const bool rescale = m_tile > m_ref + kRescaleThreshold || m_ref == -INFINITY;
          const float m_new = rescale ? m_tile : m_ref;
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          if (j > 0) {
            tmem_st_wait();                             // the optimistic P is overwritten below
            // O may be rescaled only once PV(t - 1) has finished accumulating into it
            ok = __all_sync(0xffffffffu, await(&sm.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, wc));
            if (!ok) break;
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
          l += exp_row<true>(s_addr, p_addr, valid, c, kBias - m_use);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[sb]);
      }
      ok = ok && __all_sync(0xffffffffu, await(&sm.o_done, n & 1, wc));
      if (!ok) break;
      tc_fence_after();
      // ---- the item's (or this part's) state: straight out, or left as a partial ----
      const float m_out = m_ref - kBias;                 // (the weights are 2^kBias too large)
      // dims whose codes were expanded 16 times too small: 8 w + {0, 1, 4, 5}
      auto fetch = [&](int q4, float* x) {
        uint32_t orow[32];
        __syncwarp();
        tmem_ld32(o_addr + q4 * 32, orow);
        tmem_ld_wait();
        reg_fence32(orow);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(orow[i]) * (i & 2 ? 1.f : 16.f);
      };
      const bool real = r < it.end.rows;
      const int64_t at = it.at0 + (int64_t)i_tok * a.H + g;
      bool last = !it.end.left;                          // this block writes the item's output
      if (it.end.left) {
        float* dst = a.part + (int64_t)it.end.slot * (kBM * (D + 2));
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          float x[32];
          fetch(q4, x);
          if (real) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_v8(dst + r * 8 + (q4 * 4 + i) * (kBM * 8), reinterpret_cast<const uint32_t*>(x) + 8 * i);
          }
        }
        if (real) *reinterpret_cast<float2*>(dst + kBM * D + 2 * r) = make_float2(m_out, l);
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
        // The parts in their order on the line (this block's from TMEM), whichever block is last.
        const int c0 = it.end.left ? it.end.c0 : (int)blockIdx.x, c1 = it.end.left ? it.end.c1 : (int)blockIdx.x;
        auto part = [&](int cc) { return a.part + (int64_t)(2 * cc + (cc == c0 ? 1 : 0)) * (kBM * (D + 2)); };
        auto ml_of = [&](int cc) {
          if (cc == (int)blockIdx.x) return make_float2(m_out, l);
          return __ldcg(reinterpret_cast<const float2*>(part(cc) + kBM * D + 2 * r));
        };
        float M = -INFINITY, L = 0.f;
        if (real) {
          for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, ml_of(cc).x);
          for (int cc = c0; cc <= c1; ++cc) {
            const float2 ml = ml_of(cc);
            L = fmaf(pg_weight(ml.x, M), ml.y, L);
          }
        }
        const float inv = L != 0.f ? 1.f / L : 0.f;
        if (a.lse != nullptr && real)
          a.lse[at] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        T* dst = out + at * D;
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          float mine[32], x[32];
          fetch(q4, mine);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
          for (int cc = c0; cc <= c1; ++cc) {
            const float2 ml = real ? ml_of(cc) : make_float2(0.f, 0.f);
            const float w = ml.y != 0.f ? pg_weight(ml.x, M) * inv : 0.f;
            if (cc == (int)blockIdx.x) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = fmaf(w, mine[i], x[i]);
            } else if (w != 0.f) {
              const float* src = part(cc) + r * 8;
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(src + (q4 * 4 + (i >> 3)) * (kBM * 8) + (i & 7)));
                x[i] = fmaf(w, y.x, x[i]);
                x[i + 1] = fmaf(w, y.y, x[i + 1]);
                x[i + 2] = fmaf(w, y.z, x[i + 2]);
                x[i + 3] = fmaf(w, y.w, x[i + 3]);
              }
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
cudaError_t launch(const kvc_paged4* c, kvc_pg_args a, const void* q, void* out, cudaStream_t s, bool prepare) {
  static_assert(sizeof(Smem<D>) + 1024 + 16 + (5 * KVC_PG_MAX_BATCH + KVC_PG_GRID + 3) * 4 + 16 <= 232448,
                "shared memory above the 227 KB a block may opt into");
  if (prepare)
    return cudaFuncSetAttribute(k_paged4_tc<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<D>(KVC_PG_MAX_BATCH));
  CUtensorMap tm_q;
  const int T_tok = kBM / a.Gv;
  const uint32_t box[4] = {64, (uint32_t)a.Gv, (uint32_t)T_tok, 1};
  if (!kvc_make_box_map(&tm_q, c->cfg.dtype, q, D, a.H, a.n_tokens, 1, box)) return cudaErrorInvalidValue;
  const int64_t items = (int64_t)a.Hv * ((a.n_tokens + T_tok - 1) / T_tok);            // as one row's
  const int64_t tiles = ((int64_t)a.max_pages << a.ps_log2) / kBN + 1;                 // of one, at most
  const int64_t left = items % KVC_PG_GRID;
  a.waves = 3 * items >= KVC_PG_GRID;
  a.idle = KVC_PG_TC_JOIN;
  a.join_here = a.waves && !(left > 0 && left * kManyParts < KVC_PG_GRID && items * tiles >= (int64_t)KVC_PG_GRID * kLong);
  const cudaError_t e = kvc_launch_pdl(k_paged4_tc<T, D>, dim3(KVC_PG_GRID), dim3(kThreads), smem_bytes<D>(a.B), s, tm_q,
                                       (const uint8_t*)c->pages, (T*)out, a, kvc_pg4_type<__half>::kBase);
  if (e != cudaSuccess || a.join_here) return e;
  // rows that hold no more than an uncut item's slots, and at most an item a block: nothing to join
  if (((int64_t)a.max_pages << a.ps_log2) <= KVC_PG_TC_WHOLE * kBN && items + (int64_t)a.Hv * a.B <= KVC_PG_GRID) return e;
  return kvc_pg_launch_join(c->cfg, a, out, s);
}

cudaError_t dispatch(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s, bool prep) {
  const bool d64 = c->cfg.head_dim == 64;
  if (c->cfg.dtype == KVC_F16) return d64 ? launch<__half, 64>(c, a, q, out, s, prep) : launch<__half, 128>(c, a, q, out, s, prep);
  return d64 ? launch<__nv_bfloat16, 64>(c, a, q, out, s, prep) : launch<__nv_bfloat16, 128>(c, a, q, out, s, prep);
}

}  // namespace

cudaError_t kvc_pg4_prepare_tc(const kvc_paged4* c) { return dispatch(c, kvc_pg_args{}, nullptr, nullptr, 0, true); }

cudaError_t kvc_pg4_launch_tc(const kvc_paged4* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s) {
  return dispatch(c, a, q, out, s, false);
}
