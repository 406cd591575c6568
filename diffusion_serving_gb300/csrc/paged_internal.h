// Internal declarations of the paged cache: the handle, the rows of a call as the kernels
// see them, and how the attention kernels share work among blocks.
#pragma once

#include "../../include/kvc_paged.h"
#include "../../include/kvc_rope_axes.h"
#include "kvc_internal.h"

// Blocks of the attention kernels' grids (one per SM of a 152-SM GB300; two for the FMA
// kernel).  Constants, so that workspace sizes do not depend on the device queried; no
// block waits for another, so a device with fewer SMs runs them in turn.
#define KVC_PG_GRID 152
#define KVC_PG_GRID_SIMT 304
#define KVC_PG_MAX_BATCH 1024
#define KVC_PG_MAX_SCORED 32768   // pages per row that kvc_paged_attend_sparse can rank

struct kvc_paged {
  kvc_paged_config cfg;
  int ps_log2;
  int sub;              // a kv head's group is taken as `sub` groups of Gv <= 16 heads
  int Gv, Hv;           // heads per (virtual) group, groups: Gv * Hv = H, Hv = Hkv * sub
  float scale;
  void* k;
  void* v;
  void* bounds;
  const int32_t* table;
  const int32_t* kv_len;
  uint8_t* ws;
  int device;
  uint64_t debug_stall_ns;
  // pages of a 16-bit store: boxes of 64 dims x min(page_size, 64) slots of one head, for the tensor-core kernel;
  // boxes of [min(page_size, 64) slots][D / 64][64 dims], for the streaming kernel
  CUtensorMap tm_k, tm_v, tm_dk, tm_dv;
};

// Workspace, in bytes from its start.
struct kvc_pg_layout {
  size_t tickets;       // int32 per block: blocks that have left their part of a split item
  size_t warp_tickets;  // the same per softmax warp of the tensor-core kernel
  size_t score_max;     // fp32 per (row, kv head): bound of a score's terms
  size_t zeroed;        // end of what has to start at zero (and is left at zero)
  size_t parts;         // split partials
  size_t prefix;        // partials of a shared prefix
  size_t pre_o, pre_ml; // what they join to: fp32 [max_tokens * H][D], and (max, sum)
  size_t scores;        // 8 bytes [batch, Hkv, max_pages]: fp32 scores, or the border's in fp64
  size_t total;
};
kvc_pg_layout kvc_pg_workspace(const kvc_paged_config& cfg);

// What a launch is told.  `phase`: 0 attends a row's slots (with prefix_len, the first of them in the shared list's
// pages: the streaming kernel alone); 1 the shared prefix (one row of all tokens, partials only); 2 the slots behind the
// prefix, joined with phase 1's partials.
struct kvc_pg_args {
  int B, H, Hkv, Hv, Gv, sub;
  int ps_log2, n_pages, max_pages;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  int n_tokens, max_q;
  int even;                   // tokens per row where cu is null
  int causal, phase;
  float scale_log2;
  float* lse;
  int32_t* err;
  const int32_t* prefix_pages;
  const int32_t* prefix_len;
  int prefix_cap;             // pages of the shared list
  const int32_t* sel;         // [B, Hkv, n_sel] table columns to attend, ascending, -1 behind the last
  int n_sel;
  float* part;                // [2 * grid][R][D + 2]: O (unnormalised), then (max, sum) per row
  int* tickets;
  int* warp_tickets;          // the tensor-core kernels', 4 per block, where they join split items themselves (join_here)
  int join_here;
  int waves;                  // many items: whole ones in waves, where that pays
  int idle;                   // the idle tiles per block that taking every item whole may leave before some are cut
  float* pre;                 // phase 1's partials [items + blocks][R][D + 2]
  float* pre_o;               // joined: [n_tokens * H][D], unnormalised
  float2* pre_ml;             // (max, sum)
  uint64_t stall_ns;
};

kvc_pg_args kvc_pg_base_args(const kvc_paged* c);

// ---- the host's part that paged stores of 16, 32 and 4 bits share ----
// Checks return KVC_OK, or what the call returns.
int kvc_pg_check_config(const kvc_paged_config* g);
int kvc_pg_check_rows(const kvc_paged_config& g, int32_t n_tokens, const int32_t* d_cu);
int kvc_pg_sub_groups(int G);     // a group of G query heads is taken as so many groups of at most 16
bool kvc_pg_on_device(int device);
// Reports and clears the error word at `word`; after KVC_DEV_TIMEOUT the `counters` bytes from there on.
int kvc_pg_get_error(int32_t* word, size_t counters, cudaStream_t s, int32_t* bits);
// Arguments of an append.
int kvc_pg_check_append(const kvc_paged_config& g, const void* k, const void* v, int64_t kv_stride, const void* q,
                        int64_t q_stride, const void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope,
                        int32_t rope_positions, uint32_t flags);
int kvc_pg_check_axes(const kvc_paged_config& g, const float* d_rope, const kvc_rope_axes* axes, const int32_t* d_positions);

// ---- launchers ----------------------------------------------------------------------
cudaError_t kvc_pg_launch_append(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                                 int64_t q_stride, void* q_out, int n_tokens, const int32_t* cu, const float* rope,
                                 int rope_positions, const kvc_rope_axes* axes, const int32_t* positions, bool half,
                                 cudaStream_t s);
cudaError_t kvc_pg_launch_simt(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s);
cudaError_t kvc_pg_launch_select(kvc_paged* c, const void* q, int n_sel, int first, int recent, int32_t* sel,
                                 cudaStream_t s);
cudaError_t kvc_pg_launch_decode(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s);
cudaError_t kvc_pg_launch_tc(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, cudaStream_t s);
// Phase 1's partials joined to one state per token and head; `simt`: phase 1 ran in the FMA kernel.
cudaError_t kvc_pg_launch_join_prefix(const kvc_paged* c, const kvc_pg_args& a, bool simt, cudaStream_t s);
// Split items of the tensor-core kernel.
cudaError_t kvc_pg_launch_join(const kvc_paged_config& g, const kvc_pg_args& a, void* out, cudaStream_t s);
// Shared-memory opt-ins of the kernels a handle may launch, once per handle.
cudaError_t kvc_pg_prepare_simt(const kvc_paged* c);
cudaError_t kvc_pg_prepare_select(const kvc_paged* c);
cudaError_t kvc_pg_prepare_decode(const kvc_paged* c);
cudaError_t kvc_pg_prepare_tc(const kvc_paged* c);
// query rows per item and slots per tile of the tensor-core kernel
#define KVC_PG_TC_ROWS 128
#define KVC_PG_TC_TILE 128
// fewest tiles for a block (a shared prefix is always cut evenly), what an item's beginning and end cost, in tiles, and
// the items that are not worth cutting: joining takes longer than eight tiles (434 tokens over 600 slots, 32 heads:
// 15.7 us whole, 33.8 cut by two tiles; 40 over 2000 slots, sixteen tiles: 19 cut, 22 to 24 in two halves or whole)
#define KVC_PG_TC_MIN 2
#define KVC_PG_TC_COST 3
#define KVC_PG_TC_WHOLE 8
// the idle tiles per block that taking every item whole may leave before some are cut and joined instead (3 x 434 tokens
// over 600 slots, 336 items of up to five tiles: 50 us cut, 35 whole; over 2000 slots 78 and 58)
#define KVC_PG_TC_JOIN 24
// partial rows per item and slots per tile of the FMA kernel
#define KVC_PG_SIMT_ROWS 16
#define KVC_PG_SIMT_TILE 64

#ifdef __CUDACC__
// Loads of what the kernel before may have written: plain ones, not the read-only path of __ldg (or of const __restrict__
// pointers), which is defined for data that nobody writes while the kernel lives; a programmatic dependent lives while its
// predecessor still writes.  Volatile, so that they stay behind kvc_pdl_wait().
__device__ __forceinline__ int32_t pg_ld(const int32_t* p) {
  int32_t x;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 pg_ld(const uint2* p) {
  uint2 x;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint4 pg_ld(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ float4 pg_ld(const float4* p) {
  float4 x;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
  return x;
}

// ---- rows of a call -------------------------------------------------------------------
// Row b: tokens [t0, t0 + n) of the call, keys at positions [lo, len) (`len` counts virtual slots
// of the selected pages when pages are selected).  n = 0 for a row that is skipped.
struct kvc_pg_row {
  int t0, n, len, lo;
};

// What the device arrays say of row b, loaded together (each load waits for none of the others).
struct kvc_pg_raw {
  int lo, hi, len, prefix;
};
__device__ __forceinline__ kvc_pg_raw pg_load(const kvc_pg_args& a, int b) {
  kvc_pg_raw x;
  x.lo = a.cu == nullptr ? b * a.even : a.cu[b];
  x.hi = a.cu == nullptr ? x.lo + a.even : a.cu[b + 1];
  x.len = a.kv_len[b];
  x.prefix = a.prefix_len != nullptr ? *a.prefix_len : 0;
  return x;
}
// The checks, each with its error bit.
__device__ __forceinline__ bool pg_tokens_ok(const kvc_pg_args& a, const kvc_pg_raw& x) {
  const bool ok = x.lo >= 0 && x.hi >= x.lo && x.hi <= a.n_tokens && x.hi - x.lo <= a.max_q;
  if (!ok) atomicOr(a.err, KVC_DEV_BAD_CUSEQ);
  return ok;
}
__device__ __forceinline__ bool pg_len_ok(const kvc_pg_args& a, int len) {
  const bool ok = len >= 0 && len <= (a.max_pages << a.ps_log2);
  if (!ok) atomicOr(a.err, KVC_DEV_BAD_KVLEN);
  return ok;
}
__device__ __forceinline__ bool pg_prefix_ok(const kvc_pg_args& a, int p) {
  const bool ok = p >= 0 && (p & ((1 << a.ps_log2) - 1)) == 0 && (p >> a.ps_log2) <= a.prefix_cap;
  if (!ok) atomicOr(a.err, KVC_DEV_BAD_KVLEN);
  return ok;
}

__device__ __forceinline__ kvc_pg_row pg_row(const kvc_pg_args& a, int b) {
  const kvc_pg_row none{0, 0, 0, 0};
  if (a.phase == 1) {
    const int p = *a.prefix_len;
    return pg_prefix_ok(a, p) && p > 0 ? kvc_pg_row{0, a.n_tokens, p, 0} : none;
  }
  const kvc_pg_raw x = pg_load(a, b);
  const bool tok = pg_tokens_ok(a, x), len = pg_len_ok(a, x.len);
  if (!tok || !len || (a.prefix_len != nullptr && !pg_prefix_ok(a, x.prefix))) return none;
  kvc_pg_row r{x.lo, x.hi - x.lo, x.len, a.phase == 2 ? min(x.prefix, x.len) : 0};
  if (a.sel != nullptr) r.len = min((x.len + (1 << a.ps_log2) - 1) >> a.ps_log2, a.n_sel) << a.ps_log2;
  return r;
}

// Position behind the last one that token i of row b sees (plain rows; not phase 1).
__device__ __forceinline__ int pg_limit(const kvc_pg_args& a, const kvc_pg_row& r, int i) {
  return a.causal ? r.len - r.n + i + 1 : r.len;
}

// The row that token t of the call belongs to, or -1: binary search in cu, which need not be in
// order for it to end.
__device__ __forceinline__ int pg_row_of(const kvc_pg_args& a, int t) {
  if (a.cu == nullptr) return t / a.even;
  int lo = 0, hi = a.B;   // the last b with cu[b] <= t
#pragma unroll 1
  for (int step = 0; step < 11 && hi - lo > 1; ++step) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return t >= a.cu[lo] && t < a.cu[lo + 1] ? lo : -1;
}

// Phase 1: how far into the prefix token t of the call sees (0 for a token of no valid row).
__device__ __forceinline__ int pg_prefix_limit(const kvc_pg_args& a, int t, int prefix) {
  const int b = pg_row_of(a, t);
  if (b < 0) return 0;
  const kvc_pg_raw x = pg_load(a, b);
  if (!pg_tokens_ok(a, x) || !pg_len_ok(a, x.len)) return 0;
  return max(0, min(prefix, a.causal ? x.len - (x.hi - x.lo) + (t - x.lo) + 1 : x.len));
}

// ---- work ------------------------------------------------------------------------------
// An item is the R query rows (T = R / Gv tokens x Gv heads) of one (row, group) and token tile;
// it takes tiles of TS slots, at least one (an item without keys still writes its output).
// All items stand in one line, rows outermost, then groups, then token tiles, each as `cost` empty
// places (what beginning and ending an item costs, in tiles) and then its tiles; block c takes the
// stretch [c * per, (c + 1) * per) of that line, so every block has the same to do whatever the rows'
// lengths, and an item that spans several blocks is joined from their partials.  Rows' totals are
// summed up in shared memory by every block.
//
// Where there are no more items than blocks, and they are alike or short, each item gets a whole
// number of blocks instead: it is padded to `stride` places, a multiple of `per` (no empty ones), so
// that no block works on two and no item is cut without need (at most `whole` tiles: not at all).
//
// Where there are many more items than blocks (kWaves, the tensor-core kernel), stretches would spread
// the blocks over all rows and groups at once, whose K and V together may not fit in L2; then block c
// first takes the whole items c, c + grid, ... of as many waves as surely end before the mean
// load (blocks that run together are on neighbouring items and share their K and V), and the rest of
// the line is cut into stretches that bring every block to that load; where all of them taken whole
// leave less idle than cutting costs, nothing is cut.
__host__ __device__ inline void pg_even(int tiles, int items, int grid, int min_tiles, int whole, int* per, int* stride) {
  *per = *stride = whole;
  if (tiles <= whole) return;
  const int chunks = grid / items;
  const int even = (tiles + chunks - 1) / chunks;
  *per = even > min_tiles ? even : min_tiles;
  *stride = (tiles + *per - 1) / *per * *per;
}

// Whether `items` items of `tiles` tiles in all, the longest of `most`, are padded: no more than blocks, short or alike, and
// the padded line within 32 bits (places, with room for the blocks' rounding).
#define KVC_PG_LINE (0x7fffffffll - 65536)
__host__ __device__ inline bool pg_padded(int most, long long items, long long tiles, int grid, int min_tiles, int whole, int* per,
                                          int* stride) {
  if (items <= 0 || items > grid) return false;
  if (most > (whole > 2 * min_tiles ? whole : 2 * min_tiles) && most * items * 4 > 5 * tiles) return false;
  pg_even(most, (int)items, grid, min_tiles, whole, per, stride);
  return items * *stride <= KVC_PG_LINE;
}

// Tiles of token tile k of a row: the keys that its last token sees, causal, or all.
__device__ __forceinline__ int pg_item_tiles(const kvc_pg_row& r, int k, int T, int TS, bool causal) {
  const int end = causal ? min(r.len, r.len - r.n + min((k + 1) * T, r.n)) : r.len;
  const int keys = end - r.lo;
  return keys > TS ? (keys + TS - 1) / TS : 1;
}

struct kvc_pg_item {
  int b, vh, k;          // row, group, token tile
  int tiles, start;      // its tiles, the first one's place on the line
  int tile0, tile1;      // those of this block
  bool whole;            // taken whole, in a wave
  kvc_pg_row r;
};

// Shared memory of the sums: rows + 1 first places, then each row's (t0, n, len); with waves, rows + 1 first items and
// the blocks' borders behind.
__host__ __device__ inline size_t pg_sched_bytes(int B, bool waves = false) {
  return ((size_t)(4 * B + 1 + (waves ? B + 1 + KVC_PG_GRID + 1 : 0)) * 4 + 15) & ~(size_t)15;
}

template <int R, int TS, bool kWaves = false>
struct kvc_pg_sched {
  int* base;             // [rows + 1] first place of each row
  int* rows;             // [rows][3]
  int n_rows, T, lo;     // lo: where the rows' own keys begin (behind a shared prefix, or 0)
  bool causal;
  int n_items;
  int total, per, stride, cost;   // stride: places between items' beginnings where they are padded, else 0
  int end;               // of this block's stretch
  int waves, wave, from; // waves of whole items (0: none), the one at hand, where the stretches begin on the line
  int* ibase;            // [rows + 1] first item of each row
  int* cut;              // [KVC_PG_GRID + 1] the stretches' borders, as of `from`

  __device__ __forceinline__ kvc_pg_row row(int b) const {
    return kvc_pg_row{rows[3 * b], rows[3 * b + 1], rows[3 * b + 2], min(lo, rows[3 * b + 2])};
  }
  __device__ __forceinline__ int token_tiles(int n) const { return n <= T ? n > 0 : (n + T - 1) / T; }

  // Every thread of the block calls it (it holds barriers).  A line too long for 32 bits is refused
  // with KVC_DEV_OVERFLOW (nothing is attended).
  __device__ __forceinline__ void init(const kvc_pg_args& a, void* smem, int min_tiles, int whole, int item_cost, int grid) {
    n_rows = a.phase == 1 ? 1 : a.B;
    T = a.Gv == 1 ? R : R / a.Gv;
    causal = a.causal && a.phase != 1 && a.sel == nullptr;
    base = reinterpret_cast<int*>(smem);
    rows = base + n_rows + 1;
    lo = a.phase == 2 ? max(0, *a.prefix_len) : 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // base[b + 1]: the row's tiles over its token tiles, per group; -1: more than 32 bits hold
    auto capped = [&](long long x) { return x <= 0x7fffffffll ? (int)x : -1; };
    for (int b = threadIdx.x; b < n_rows; b += blockDim.x) {
      const kvc_pg_row r = pg_row(a, b);
      rows[3 * b] = r.t0;
      rows[3 * b + 1] = r.n;
      rows[3 * b + 2] = r.len;
      const int m = token_tiles(r.n);
      if (!causal || m <= 1) base[b + 1] = m == 0 ? 0 : capped((long long)m * pg_item_tiles(r, 0, T, TS, causal));
    }
    __syncthreads();
    if (causal) {
      for (int b = warp; b < n_rows; b += blockDim.x >> 5) {
        const kvc_pg_row r = row(b);
        const int m = token_tiles(r.n);
        if (m <= 1) continue;
        long long x = 0;
        for (int k = lane; k < m; k += 32) x += pg_item_tiles(r, k, T, TS, true);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) base[b + 1] = capped(x);
      }
      __syncthreads();
    }
    // every warp works out the same sums (no warp has to hand them on)
    long long tiles = 0, items = 0;
    int most = 0;
    bool over = false;
    for (int b = lane; b < n_rows; b += 32) {
      const int x = base[b + 1];
      over = over || x < 0;
      const kvc_pg_row r = row(b);
      const int m = token_tiles(r.n);
      tiles += x;
      items += m;
      if (m > 0) most = max(most, pg_item_tiles(r, m - 1, T, TS, causal));
    }
    if (n_rows > 1) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        items += __shfl_xor_sync(0xffffffffu, items, o);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
    } else {
      tiles = __shfl_sync(0xffffffffu, tiles, 0);
      items = __shfl_sync(0xffffffffu, items, 0);
      most = __shfl_sync(0xffffffffu, most, 0);
    }
    tiles *= a.Hv;
    items *= a.Hv;
    over = __any_sync(0xffffffffu, over) || tiles + items * item_cost > KVC_PG_LINE;
    cost = item_cost;
    n_items = (int)items;
    waves = 0;
    if (over) {
      if (threadIdx.x == 0) atomicOr(a.err, KVC_DEV_OVERFLOW);
      total = 0;
      per = 1;
      stride = 0;
      return;
    }
    if (pg_padded(most, items, tiles, grid, min_tiles, whole, &per, &stride)) {
      cost = 0;
      total = (int)items * stride;
    } else {
      stride = 0;
      total = (int)(tiles + items * cost);
      per = max(min_tiles, (total + grid - 1) / grid);
      if (kWaves && a.waves) {
        const long long rounds = (items + grid - 1) / grid;
        waves = rounds * (most + cost) <= total / grid + a.idle ? (int)rounds : (total / grid) / (most + cost);
      }
    }
    __syncthreads();                       // (every warp has read the rows' own tiles)
    if (kWaves && waves > 0 && warp == 1) {
      ibase = rows + 3 * n_rows;
      int carry = 0;
      for (int b0 = 0; b0 < n_rows; b0 += 32) {
        const int b = b0 + lane;
        int x = b < n_rows ? a.Hv * token_tiles(rows[3 * b + 1]) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (b < n_rows) ibase[b + 1] = carry + x;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) ibase[0] = 0;
    }
    if (warp == 0) {
      int carry = 0;
      for (int b0 = 0; b0 < n_rows; b0 += 32) {
        const int b = b0 + lane;
        int x = 0;
        if (b < n_rows) {
          const int m = token_tiles(rows[3 * b + 1]);
          x = a.Hv * (stride ? m * stride : base[b + 1] + m * cost);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (b < n_rows) base[b + 1] = carry + x;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) base[0] = 0;
    }
    __syncthreads();
    if (kWaves && waves > 0) {
      ibase = rows + 3 * n_rows;
      cut = ibase + n_rows + 1;
      // what each block's whole items leave of the mean load (a place more, so that it is never nothing)
      const int mean = total / grid + 2;
      const bool all = (long long)waves * grid >= items;         // nothing is left to cut
      for (int c = threadIdx.x; c < grid; c += blockDim.x) {
        int load = all ? mean : 0;
        if (!all)
          for (int w = 0; w < waves; ++w) load += item(a, c + w * grid).tiles + cost;
        cut[c + 1] = mean - load;
      }
      from = all ? total : item(a, waves * grid, true).start - cost;
      __syncthreads();
      if (warp == 0) {
        long long carry = 0;
        for (int c0 = 0; c0 < grid; c0 += 32) {
          const int c = c0 + lane;
          long long x = c < grid ? cut[c + 1] : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          if (c < grid) cut[c + 1] = (int)min((long long)(total - from), carry + x);
          carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) cut[0] = 0;
      }
      __syncthreads();
    }
  }

  // Item i of the line, whole; with tiles = 0 where there are not so many.  Its start is left out unless asked for (token
  // tiles before it are added up one by one where they differ).
  __device__ __forceinline__ kvc_pg_item item(const kvc_pg_args& a, int i, bool with_start = false) const {
    kvc_pg_item it;
    it.tiles = 0;
    if (i >= ibase[n_rows]) return it;
    int b = 0, hi = n_rows;
#pragma unroll 1
    for (int step = 0; step < 11 && hi - b > 1; ++step) {
      const int mid = (b + hi) >> 1;
      if (ibase[mid] <= i) b = mid;
      else hi = mid;
    }
    it.b = b;
    it.r = row(b);
    const int m = token_tiles(it.r.n);
    i -= ibase[b];
    it.vh = i / m;
    it.k = i - it.vh * m;
    it.tiles = pg_item_tiles(it.r, it.k, T, TS, causal);
    it.start = 0;
    if (with_start) {
      it.start = base[b] + it.vh * ((base[b + 1] - base[b]) / a.Hv) + cost;
      if (!causal) it.start += it.k * (it.tiles + cost);
      else
        for (int k = 0; k < it.k; ++k) it.start += pg_item_tiles(it.r, k, T, TS, true) + cost;
    }
    it.tile0 = 0;
    it.tile1 = it.tiles;
    it.whole = true;
    return it;
  }

  // The blocks that an item spans.
  __device__ __forceinline__ void span(const kvc_pg_item& it, int* c0, int* c1) const {
    if (kWaves && it.whole) {
      *c0 = *c1 = blockIdx.x;
      return;
    }
    if (!kWaves || waves == 0) {
      *c0 = it.start / per;
      *c1 = (it.start + it.tiles - 1) / per;
      return;
    }
    auto block_of = [&](int p) {           // the last c with cut[c] <= p (a block without a stretch holds no place)
      int c = 0, hi = KVC_PG_GRID;
#pragma unroll 1
      for (int step = 0; step < 9 && hi - c > 1; ++step) {
        const int mid = (c + hi) >> 1;
        if (cut[mid] <= p) c = mid;
        else hi = mid;
      }
      return c;
    };
    *c0 = block_of(it.start - from);
    *c1 = block_of(it.start + it.tiles - 1 - from);
  }

  // The item that holds place p of the line (p < total); a whole warp calls it.
  __device__ __forceinline__ kvc_pg_item at(const kvc_pg_args& a, int p) const {
    kvc_pg_item it;
    it.whole = false;
    int b = 0, hi = n_rows;
#pragma unroll 1
    for (int step = 0; step < 11 && hi - b > 1; ++step) {
      const int mid = (b + hi) >> 1;
      if (base[mid] <= p) b = mid;
      else hi = mid;
    }
    it.b = b;
    it.r = row(b);
    const int m = token_tiles(it.r.n);
    const int group = stride ? m * stride : (base[b + 1] - base[b]) / a.Hv;
    p -= base[b];
    it.vh = p / group;
    it.start = base[b] + it.vh * group;
    p -= it.vh * group;
    if (stride || !causal || m == 1) {
      const int step = stride ? stride : pg_item_tiles(it.r, 0, T, TS, causal) + cost;
      it.k = m == 1 ? 0 : p / step;
      it.start += it.k * step + cost;
      it.tiles = pg_item_tiles(it.r, it.k, T, TS, causal);
      return it;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;                        // places of the token tiles up to k0
    it.k = 0;
    it.tiles = 1;
    for (int k0 = 0; k0 < m; k0 += 32) {
      const int mine = k0 + lane < m ? pg_item_tiles(it.r, k0 + lane, T, TS, true) : 0;
      int x = mine > 0 ? mine + cost : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, k0 + lane < m && before + x > p);
      if (behind) {
        const int l = __ffs(behind) - 1;
        it.k = k0 + l;
        it.tiles = __shfl_sync(0xffffffffu, mine, l);
        it.start += before + __shfl_sync(0xffffffffu, x, l) - it.tiles;
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    return it;
  }

  // Block c's first item; false if it has none.  A whole warp calls it.
  __device__ __forceinline__ bool first(const kvc_pg_args& a, int c, kvc_pg_item& it) {
    if (kWaves && waves > 0) {
      wave = 0;
      it = item(a, c);
      return it.tiles > 0;
    }
    if ((long long)c * per >= total) return false;
    const int p = c * per;
    return stretch(a, p, total - p > per ? p + per : total, it);
  }
  __device__ __forceinline__ bool stretch(const kvc_pg_args& a, int p, int end_, kvc_pg_item& it) {
    end = end_;
    it = at(a, p);
    it.tile0 = max(0, p - it.start);
    it.tile1 = min(it.tiles, end - it.start);
    return it.tile1 > it.tile0;            // (not if the stretch ends before the item's tiles begin)
  }

  // The block's next item; false if there is none.  A whole warp calls it.
  __device__ __forceinline__ bool next(const kvc_pg_args& a, kvc_pg_item& it) {
    if (kWaves && waves > 0 && wave < waves) {
      if (++wave < waves) {
        it = item(a, blockIdx.x + wave * gridDim.x);
        return it.tiles > 0;
      }
      const int p = from + cut[blockIdx.x], e = from + cut[blockIdx.x + 1];
      return p < e && stretch(a, p, e, it);
    }
    if (stride || it.start + it.tiles + cost >= end) return false;
    it.start += it.tiles + cost;
    if ((it.k + 1) * T < it.r.n) {
      ++it.k;
    } else {
      it.k = 0;
      if (++it.vh == a.Hv) {
        it.vh = 0;
        ++it.b;
        for (; it.b + 1 < n_rows && base[it.b + 1] == it.start - cost; ++it.b) {
        }
        it.r = row(it.b);
      }
    }
    it.tiles = pg_item_tiles(it.r, it.k, T, TS, causal);
    it.tile0 = 0;
    it.tile1 = min(it.tiles, end - it.start);
    return true;
  }
};

// Page number of table column `col` of row b (phase 1: of the shared list), or -1 with the error bit.
__device__ __forceinline__ int pg_page(const kvc_pg_args& a, int b, int col) {
  const int p = a.phase == 1 ? pg_ld(a.prefix_pages + col) : pg_ld(a.table + (int64_t)b * a.max_pages + col);
  if (p < 0 || p >= a.n_pages) {
    atomicOr(a.err, KVC_DEV_BAD_PAGE);
    return -1;
  }
  return p;
}
#endif  // __CUDACC__
