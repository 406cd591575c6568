// C-ABI entry points of the paged cache (declared and documented in include/kvc_paged.h):
// host-side validation, handle state and kernel selection.  Every call only enqueues work on
// the caller's stream; nothing here allocates device memory.
#include <math.h>

#include <new>

#include "paged_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
int launched(cudaError_t e) { return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int check_cfg(const kvc_paged_config* g) {
  if (g == nullptr) return KVC_ERR_ARG;
  if (g->batch < 1 || g->heads < 1 || g->kv_heads < 1 || g->heads % g->kv_heads) return KVC_ERR_ARG;
  if (g->dtype < KVC_F32 || g->dtype > KVC_BF16) return KVC_ERR_ARG;
  if (g->n_pages < 1 || g->max_pages < 1 || g->max_tokens < 1) return KVC_ERR_ARG;
  if (!(g->softmax_scale >= 0.f) || isinf(g->softmax_scale)) return KVC_ERR_ARG;
  if (g->head_dim != 64 && g->head_dim != 128) return KVC_ERR_UNSUPPORTED;
  if (g->page_size != 16 && g->page_size != 32 && g->page_size != 64 && g->page_size != 128) return KVC_ERR_UNSUPPORTED;
  if (g->batch > KVC_PG_MAX_BATCH || g->heads > 4096) return KVC_ERR_UNSUPPORTED;
  if ((int64_t)g->max_pages * g->page_size > (1 << 30)) return KVC_ERR_ARG;
  return KVC_OK;
}

// A group of G query heads is taken as `sub` groups of at most 16.
int sub_groups(int G) {
  for (int sub = 1; sub < G; ++sub)
    if (G % sub == 0 && G / sub <= 16) return sub;
  return G;
}

// The handle's device has to be the current one: its streams and buffers belong to it.
bool on_device(const kvc_paged* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

int check_rows(const kvc_paged* c, int32_t n_tokens, const int32_t* d_cu) {
  if (n_tokens < 1 || !aligned(d_cu, 4)) return KVC_ERR_ARG;
  if (d_cu == nullptr && n_tokens % c->cfg.batch) return KVC_ERR_ARG;
  return KVC_OK;
}

int check_attend(const kvc_paged* c, const void* q, const void* out, const float* lse, int32_t n_tokens,
                 const int32_t* d_cu, int32_t max_q, uint32_t flags) {
  if (c == nullptr || !q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return KVC_ERR_ARG;
  if (flags & ~(uint32_t)(KVC_CAUSAL | KVC_KERNEL_SIMT)) return KVC_ERR_ARG;
  if (d_cu != nullptr && max_q < 1) return KVC_ERR_ARG;
  const int rc = check_rows(c, n_tokens, d_cu);
  if (rc != KVC_OK) return rc;
  return on_device(c) ? KVC_OK : KVC_ERR_ARG;
}

// Kernel by type and shape: fp32 stores (and KVC_KERNEL_SIMT) run the FMA kernel; 16-bit ones with few
// query rows per group the streaming kernel, with more (and for a shared prefix, where the batch's rows
// are stacked) the tensor-core kernel.  "Few" is 16 rows, one pass over a row's keys, or 32, two passes,
// where all rows' and groups' slots (behind the prefix) are at most 128 K: 20 rows a group, 8 groups of 128 dims, take
// 18.5 us in two passes and 23.1 in the tensor-core kernel for a batch of 1 over 8000 slots, 25.6 and 27.6 for 8 over 2000,
// 26.4 and 34.1 for 32 over 300; but 85 and 64 for 8 over 8000, 96 and 67 for 32 over 2000.  Lengths are on the device, so the slots
// are those that the table has columns for: with one sized for far longer rows these batches take the second figure of each pair.
bool simt_only(const kvc_paged* c, uint32_t flags) { return c->cfg.dtype == KVC_F32 || (flags & KVC_KERNEL_SIMT); }

bool few_rows(const kvc_pg_args& a, int64_t slots) {
  return (int64_t)a.max_q * a.Gv <= (a.B * a.Hv * slots <= 128 * 1024 ? 32 : 16);
}

cudaError_t run_attend(const kvc_paged* c, const kvc_pg_args& a, const void* q, void* out, uint32_t flags, cudaStream_t s) {
  if (simt_only(c, flags)) return kvc_pg_launch_simt(c, a, q, out, s);
  const int64_t slots = (int64_t)(a.max_pages - (a.phase == 2 ? a.prefix_cap : 0)) << a.ps_log2;
  if (a.phase != 1 && few_rows(a, slots)) return kvc_pg_launch_decode(c, a, q, out, s);
  return kvc_pg_launch_tc(c, a, q, out, s);
}

// A shared prefix of few rows is cheaper read once per row, from L2, in the streaming kernel alone (it takes the page
// numbers below the prefix's end from the shared list) than once for all in three launches.  What counts is the bytes
// that all rows' passes over it read: at 34 MB (8 rows, 1024 slots, 8 heads of 128) 12.6 us against 22.2, at 67 MB 17.1
// against 24.0, at 134 MB 26.1 against 25.3 (pages of 64: 23.0 against 25.5; heads of 64: 26.2 against 25.1), at 268 MB
// 43 and 26.  (The prefix counts with the length of its list, not the length on the device: 1024 slots in a list of 8192, 21.3 us.)
bool one_pass(const kvc_pg_args& a, int head_dim) {
  const int T = 16 / a.Gv;                             // tokens to an item
  const int64_t passes = (int64_t)a.B * a.Hv * ((a.max_q + T - 1) / T);
  return passes * ((int64_t)a.prefix_cap << a.ps_log2) * head_dim * 4 <= (int64_t)96 << 20;
}

kvc_pg_args attend_args(const kvc_paged* c, float* lse, int32_t n_tokens, const int32_t* d_cu, int32_t max_q,
                        uint32_t flags) {
  kvc_pg_args a = kvc_pg_base_args(c);
  a.lse = lse;
  a.n_tokens = n_tokens;
  a.cu = d_cu;
  a.even = n_tokens / c->cfg.batch;
  a.max_q = d_cu != nullptr ? max_q : n_tokens / c->cfg.batch;
  a.causal = (flags & KVC_CAUSAL) != 0;
  return a;
}

}  // namespace

kvc_pg_layout kvc_pg_workspace(const kvc_paged_config& g) {
  kvc_pg_layout w{};
  const size_t D2 = (size_t)g.head_dim + 2;
  const int sub = sub_groups(g.heads / g.kv_heads);
  const size_t Gv = (size_t)g.heads / g.kv_heads / sub, Hv = (size_t)g.kv_heads * sub;
  w.tickets = 256;
  w.warp_tickets = w.tickets + 4 * (size_t)KVC_PG_GRID_SIMT;
  w.score_max = w.warp_tickets + 4 * 4 * (size_t)KVC_PG_GRID;
  w.zeroed = up256(w.score_max + 4 * (size_t)g.batch * g.kv_heads);
  w.parts = w.zeroed;
  // two partials a block; a shared prefix's are at most its items and blocks together
  auto parts = [&](size_t grid, size_t R) { return 2 * grid * R * D2 * 4; };
  auto prefix = [&](size_t grid, size_t R) {
    const size_t T = R / Gv;
    return (Hv * (((size_t)g.max_tokens + T - 1) / T) + grid) * R * D2 * 4;
  };
  const bool tc = g.dtype != KVC_F32;
  const size_t p0 = parts(KVC_PG_GRID_SIMT, KVC_PG_SIMT_ROWS), p1 = tc ? parts(KVC_PG_GRID, KVC_PG_TC_ROWS) : 0;
  const size_t x0 = prefix(KVC_PG_GRID_SIMT, KVC_PG_SIMT_ROWS), x1 = tc ? prefix(KVC_PG_GRID, KVC_PG_TC_ROWS) : 0;
  w.prefix = w.parts + up256(p0 > p1 ? p0 : p1);
  w.pre_o = w.prefix + up256(x0 > x1 ? x0 : x1);
  const size_t rows = (size_t)g.max_tokens * g.heads;
  w.pre_ml = w.pre_o + up256(rows * g.head_dim * 4);
  w.scores = w.pre_ml + up256(rows * 8);
  const size_t scored = g.max_pages <= KVC_PG_MAX_SCORED ? (size_t)g.batch * g.kv_heads * g.max_pages * 8 : 0;
  w.total = up256(w.scores + scored);
  return w;
}

kvc_pg_args kvc_pg_base_args(const kvc_paged* c) {
  const kvc_paged_config& g = c->cfg;
  const kvc_pg_layout w = kvc_pg_workspace(g);
  kvc_pg_args a{};
  a.B = g.batch;
  a.H = g.heads;
  a.Hkv = g.kv_heads;
  a.Hv = c->Hv;
  a.Gv = c->Gv;
  a.sub = c->sub;
  a.ps_log2 = c->ps_log2;
  a.n_pages = g.n_pages;
  a.max_pages = g.max_pages;
  a.table = c->table;
  a.kv_len = c->kv_len;
  a.scale_log2 = c->scale * 1.4426950408889634f;
  a.err = reinterpret_cast<int32_t*>(c->ws);
  a.tickets = reinterpret_cast<int*>(c->ws + w.tickets);
  a.warp_tickets = reinterpret_cast<int*>(c->ws + w.warp_tickets);
  a.part = reinterpret_cast<float*>(c->ws + w.parts);
  a.pre = reinterpret_cast<float*>(c->ws + w.prefix);
  a.pre_o = reinterpret_cast<float*>(c->ws + w.pre_o);
  a.pre_ml = reinterpret_cast<float2*>(c->ws + w.pre_ml);
  a.stall_ns = c->debug_stall_ns;
  return a;
}

extern "C" {

size_t kvc_paged_workspace_bytes(const kvc_paged_config* cfg) {
  return check_cfg(cfg) == KVC_OK ? kvc_pg_workspace(*cfg).total : 0;
}

int kvc_paged_create(const kvc_paged_config* cfg, void* k_pages, void* v_pages, void* bounds, const int32_t* d_table,
                     const int32_t* d_kv_len, void* workspace, void* stream, kvc_paged** out) {
  if (out == nullptr) return KVC_ERR_ARG;
  *out = nullptr;
  const int rc = check_cfg(cfg);
  if (rc != KVC_OK) return rc;
  if (!k_pages || !v_pages || !d_table || !d_kv_len || !workspace) return KVC_ERR_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(bounds, 16) || !aligned(workspace, 256)) return KVC_ERR_ARG;
  if (!aligned(d_table, 4) || !aligned(d_kv_len, 4)) return KVC_ERR_ARG;
  kvc_paged* c = new (std::nothrow) kvc_paged();
  if (c == nullptr) return KVC_ERR_ARG;
  c->cfg = *cfg;
  c->ps_log2 = cfg->page_size == 16 ? 4 : cfg->page_size == 32 ? 5 : cfg->page_size == 64 ? 6 : 7;
  const int G = cfg->heads / cfg->kv_heads;
  c->sub = sub_groups(G);
  c->Gv = G / c->sub;
  c->Hv = cfg->kv_heads * c->sub;
  c->scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / sqrtf((float)cfg->head_dim);
  c->k = k_pages;
  c->v = v_pages;
  c->bounds = bounds;
  c->table = d_table;
  c->kv_len = d_kv_len;
  c->ws = reinterpret_cast<uint8_t*>(workspace);
  c->debug_stall_ns = 0;
  bool ok = cudaGetDevice(&c->device) == cudaSuccess;
  if (ok && cfg->dtype != KVC_F32) {
    const uint32_t rows = cfg->page_size < 64 ? cfg->page_size : 64;
    ok = kvc_make_tile_map(&c->tm_k, cfg->dtype, k_pages, cfg->head_dim, cfg->kv_heads, cfg->page_size, cfg->n_pages, rows) &&
         kvc_make_tile_map(&c->tm_v, cfg->dtype, v_pages, cfg->head_dim, cfg->kv_heads, cfg->page_size, cfg->n_pages, rows) &&
         kvc_make_page_map(&c->tm_dk, cfg->dtype, k_pages, cfg->head_dim, cfg->kv_heads, cfg->page_size, cfg->n_pages, rows) &&
         kvc_make_page_map(&c->tm_dv, cfg->dtype, v_pages, cfg->head_dim, cfg->kv_heads, cfg->page_size, cfg->n_pages, rows);
  }
  ok = ok && kvc_pg_prepare_simt(c) == cudaSuccess && (bounds == nullptr || kvc_pg_prepare_select(c) == cudaSuccess) &&
       (cfg->dtype == KVC_F32 ||
        (kvc_pg_prepare_decode(c) == cudaSuccess && kvc_pg_prepare_tc(c) == cudaSuccess));
  ok = ok && cudaMemsetAsync(workspace, 0, kvc_pg_workspace(*cfg).zeroed, as_stream(stream)) == cudaSuccess;
  if (!ok) {
    delete c;
    return KVC_ERR_CUDA;
  }
  *out = c;
  return KVC_OK;
}

int kvc_paged_append(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q, int64_t q_stride,
                     void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope, int32_t rope_positions,
                     uint32_t flags, void* stream) {
  if (c == nullptr || !k || !v || !aligned(k, 16) || !aligned(v, 16)) return KVC_ERR_ARG;
  if (flags & ~(uint32_t)KVC_ROPE_HALF) return KVC_ERR_ARG;
  const int rc = check_rows(c, n_tokens, d_cu);
  if (rc != KVC_OK) return rc;
  const kvc_paged_config& g = c->cfg;
  const int64_t vec = g.dtype == KVC_F32 ? 4 : 8;      // elements of 16 bytes
  const int64_t kv_row = (int64_t)g.kv_heads * g.head_dim, q_row = (int64_t)g.heads * g.head_dim;
  if (kv_stride < kv_row || kv_stride % vec) return KVC_ERR_ARG;
  if (d_rope != nullptr && (!aligned(d_rope, 16) || rope_positions < 1)) return KVC_ERR_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return KVC_ERR_ARG;
  if (q != nullptr) {
    if (d_rope == nullptr || !aligned(q, 16) || !aligned(q_out, 16) || q_stride < q_row || q_stride % vec) return KVC_ERR_ARG;
    if (q == q_out && q_stride != q_row) return KVC_ERR_ARG;
  }
  if (!on_device(c)) return KVC_ERR_ARG;
  return launched(kvc_pg_launch_append(c, k, v, kv_stride, q, q_stride, q_out, n_tokens, d_cu, d_rope, rope_positions,
                                       (flags & KVC_ROPE_HALF) != 0, as_stream(stream)));
}

int kvc_paged_attend(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_tokens, const int32_t* d_cu,
                     int32_t max_q, uint32_t flags, void* stream) {
  const int rc = check_attend(c, q, out, d_lse, n_tokens, d_cu, max_q, flags);
  if (rc != KVC_OK) return rc;
  const kvc_pg_args a = attend_args(c, d_lse, n_tokens, d_cu, max_q, flags);
  return launched(run_attend(c, a, q, out, flags, as_stream(stream)));
}

int kvc_paged_attend_shared(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_tokens,
                            const int32_t* d_cu, int32_t max_q, const int32_t* d_prefix_pages, int32_t prefix_pages,
                            const int32_t* d_prefix_len, uint32_t flags, void* stream) {
  const int rc = check_attend(c, q, out, d_lse, n_tokens, d_cu, max_q, flags);
  if (rc != KVC_OK) return rc;
  if (!d_prefix_pages || !d_prefix_len || !aligned(d_prefix_pages, 4) || !aligned(d_prefix_len, 4)) return KVC_ERR_ARG;
  if (prefix_pages < 1 || prefix_pages > c->cfg.max_pages) return KVC_ERR_ARG;
  if (n_tokens > c->cfg.max_tokens) return KVC_ERR_RANGE;
  // the prefix's tiles, over all items, are counted in 32 bits
  const int64_t items = (int64_t)c->Hv * (n_tokens / (KVC_PG_SIMT_ROWS / c->Gv) + 1);
  if (items * ((int64_t)prefix_pages * c->cfg.page_size / KVC_PG_SIMT_TILE + 1 + KVC_PG_TC_COST) > INT32_MAX - 65536) return KVC_ERR_RANGE;
  kvc_pg_args a = attend_args(c, d_lse, n_tokens, d_cu, max_q, flags);
  a.prefix_pages = d_prefix_pages;
  a.prefix_cap = prefix_pages;
  a.prefix_len = d_prefix_len;
  cudaStream_t s = as_stream(stream);
  if (!simt_only(c, flags) && few_rows(a, (int64_t)a.max_pages << a.ps_log2) && one_pass(a, c->cfg.head_dim))
    return launched(kvc_pg_launch_decode(c, a, q, out, s));
  a.phase = 1;
  cudaError_t e = run_attend(c, a, q, out, flags, s);
  if (e == cudaSuccess)
    e = kvc_pg_launch_join_prefix(c, a, simt_only(c, flags), s);
  if (e != cudaSuccess) return KVC_ERR_CUDA;
  a.phase = 2;
  return launched(run_attend(c, a, q, out, flags, s));
}

int kvc_paged_attend_sparse(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_select, int32_t first,
                            int32_t recent, int32_t* d_selected, uint32_t flags, void* stream) {
  if (c == nullptr) return KVC_ERR_ARG;
  const int rc = check_attend(c, q, out, d_lse, c->cfg.batch, nullptr, 1, flags);
  if (rc != KVC_OK) return rc;
  if (flags & KVC_CAUSAL) return KVC_ERR_ARG;
  if (d_selected == nullptr || !aligned(d_selected, 4) || n_select < 1 || first < 0 || recent < 0 ||
      (int64_t)first + recent > n_select)
    return KVC_ERR_ARG;
  if (c->bounds == nullptr) return KVC_ERR_UNSUPPORTED;
  if (c->cfg.max_pages > KVC_PG_MAX_SCORED) return KVC_ERR_RANGE;
  cudaStream_t s = as_stream(stream);
  const cudaError_t e = kvc_pg_launch_select(c, q, n_select, first, recent, d_selected, s);
  if (e != cudaSuccess) return KVC_ERR_CUDA;
  kvc_pg_args a = attend_args(c, d_lse, c->cfg.batch, nullptr, 1, flags);
  a.sel = d_selected;
  a.n_sel = n_select;
  return launched(run_attend(c, a, q, out, flags, s));
}

int kvc_paged_get_error(kvc_paged* c, void* stream, int32_t* bits) {
  if (c == nullptr || !on_device(c)) return KVC_ERR_ARG;
  cudaStream_t s = as_stream(stream);
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, c->ws, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return KVC_ERR_CUDA;
  if (bits != nullptr) *bits = word;
  if (word == 0) return KVC_OK;
  // a kernel that gave up may have left counters off zero
  const size_t n = (word & KVC_DEV_TIMEOUT) ? kvc_pg_workspace(c->cfg).zeroed : sizeof(int32_t);
  if (cudaMemsetAsync(c->ws, 0, n, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess) return KVC_ERR_CUDA;
  return KVC_ERR_DEVICE;
}

int kvc_paged_debug_stall_waits(kvc_paged* c, uint64_t ns) {
  if (c == nullptr) return KVC_ERR_ARG;
  c->debug_stall_ns = ns;
  return KVC_OK;
}

int kvc_paged_destroy(kvc_paged* c) {
  delete c;
  return KVC_OK;
}

}  // extern "C"
