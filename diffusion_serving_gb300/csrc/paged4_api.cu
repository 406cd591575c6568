// C-ABI entry points of the 4-bit paged store (declared and documented in include/kvc_paged4.h): host-side validation,
// handle state and kernel selection.  Every call only enqueues work on the caller's stream; nothing here allocates device
// memory.
#include <math.h>

#include <new>

#include "paged4_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
int launched(cudaError_t e) { return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
int log2_of(int n) { return n == 16 ? 4 : n == 32 ? 5 : n == 64 ? 6 : 7; }

int check_config(const kvc_paged_config* g) {
  const int rc = kvc_pg_check_config(g);
  return rc != KVC_OK ? rc : g->dtype == KVC_F32 ? KVC_ERR_UNSUPPORTED : KVC_OK;
}

kvc_pg4_layout workspace_of(const kvc_paged_config& g) {
  kvc_pg4_layout w{};
  w.tickets = 256;
  w.warp_tickets = w.tickets + 4 * (size_t)KVC_PG_GRID;
  w.zeroed = up256(w.warp_tickets + 4 * 4 * (size_t)KVC_PG_GRID);
  w.parts = w.zeroed;
  // two partials a block
  w.total = up256(w.parts + 2 * (size_t)KVC_PG_GRID * KVC_PG_TC_ROWS * (g.head_dim + 2) * 4);
  return w;
}

// Up to 16 query rows per group are one pass of the streaming kernel over a row's keys.  More make several passes there, which
// still beat the tensor-core kernel where they are few and short in all (four, 128 or 512 items of a head's rows, and 768 K or 4 M slots over
// them, for heads of 128 or 64).  32 heads over 8, streaming and tensor-core kernel: 32 rows a group, heads of 128: 18 and 24 us
// for a batch of 1 over 8000 slots, 21 and 29 for 8 over 2000, but 38 and 27 for 32 over 600, 183 and 165 for 32 over 8000; heads of
// 64: 32 and 50 for 8 over 8000, 102 and 141 for 32 over 8000; 64 rows: 12 and 22 for 1 over 8000 of 64 dims, 25 and 16 for 8 over 600 of
// 128.  Lengths are on the device: the slots are those that the table has columns for, so with a table far wider than its rows several
// passes are not taken (16 rows of 900 .. 9000 slots, 1 to 5 tokens, 40 heads over 8 of 64: 33 us, and 54 under a table of 131072 slots).
bool few_rows(const kvc_pg_args& a, int head_dim) {
  const int T = 16 / a.Gv;                             // tokens to an item
  const int64_t passes = ((int64_t)a.max_q + T - 1) / T, items = a.B * (int64_t)a.Hv * passes;
  if (passes == 1) return true;
  const bool d64 = head_dim == 64;
  return passes <= 4 && items <= (d64 ? 512 : 128) && items * ((int64_t)a.max_pages << a.ps_log2) <= (d64 ? 4 << 20 : 768 << 10);
}

}  // namespace

extern "C" {

size_t kvc_paged4_page_bytes(const kvc_paged_config* cfg) {
  return check_config(cfg) == KVC_OK ? (size_t)cfg->kv_heads * kvc_pg4_record(cfg->head_dim, log2_of(cfg->page_size)) : 0;
}

size_t kvc_paged4_workspace_bytes(const kvc_paged_config* cfg) {
  return check_config(cfg) == KVC_OK ? workspace_of(*cfg).total : 0;
}

int kvc_paged4_create(const kvc_paged_config* cfg, void* pages, const int32_t* d_table, const int32_t* d_kv_len,
                      void* workspace, void* stream, kvc_paged4** out) {
  if (out == nullptr) return KVC_ERR_ARG;
  *out = nullptr;
  const int rc = check_config(cfg);
  if (rc != KVC_OK) return rc;
  if (!pages || !d_table || !d_kv_len || !workspace) return KVC_ERR_ARG;
  if (!aligned(pages, 16) || !aligned(workspace, 256) || !aligned(d_table, 4) || !aligned(d_kv_len, 4)) return KVC_ERR_ARG;
  kvc_paged4* c = new (std::nothrow) kvc_paged4();
  if (c == nullptr) return KVC_ERR_ARG;
  c->cfg = *cfg;
  c->ps_log2 = log2_of(cfg->page_size);
  const int G = cfg->heads / cfg->kv_heads;
  c->sub = kvc_pg_sub_groups(G);
  c->Gv = G / c->sub;
  c->Hv = cfg->kv_heads * c->sub;
  c->scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / sqrtf((float)cfg->head_dim);
  c->pages = reinterpret_cast<uint8_t*>(pages);
  c->table = d_table;
  c->kv_len = d_kv_len;
  c->ws = reinterpret_cast<uint8_t*>(workspace);
  c->debug_stall_ns = 0;
  if (cudaGetDevice(&c->device) != cudaSuccess || kvc_pg4_prepare_decode(c) != cudaSuccess || kvc_pg4_prepare_tc(c) != cudaSuccess ||
      cudaMemsetAsync(workspace, 0, workspace_of(*cfg).zeroed, as_stream(stream)) != cudaSuccess) {
    delete c;
    return KVC_ERR_CUDA;
  }
  *out = c;
  return KVC_OK;
}

int kvc_paged4_append(kvc_paged4* c, const void* k, const void* v, int64_t kv_stride, const void* q, int64_t q_stride,
                      void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope, int32_t rope_positions,
                      const kvc_rope_axes* axes, const int32_t* d_positions, uint32_t flags, void* stream) {
  if (c == nullptr) return KVC_ERR_ARG;
  int rc = kvc_pg_check_append(c->cfg, k, v, kv_stride, q, q_stride, q_out, n_tokens, d_cu, d_rope, rope_positions, flags);
  if (rc == KVC_OK && (axes != nullptr || d_positions != nullptr)) rc = kvc_pg_check_axes(c->cfg, d_rope, axes, d_positions);
  if (rc != KVC_OK) return rc;
  if (!kvc_pg_on_device(c->device)) return KVC_ERR_ARG;
  return launched(kvc_pg4_launch_append(c, k, v, kv_stride, q, q_stride, q_out, n_tokens, d_cu, d_rope, rope_positions, axes,
                                        d_positions, (flags & KVC_ROPE_HALF) != 0, as_stream(stream)));
}

int kvc_paged4_read(kvc_paged4* c, void* k_out, void* v_out, int32_t n_tokens, const int32_t* d_cu, void* stream) {
  if (c == nullptr || (!k_out && !v_out) || !aligned(k_out, 16) || !aligned(v_out, 16)) return KVC_ERR_ARG;
  const int rc = kvc_pg_check_rows(c->cfg, n_tokens, d_cu);
  if (rc != KVC_OK) return rc;
  if (!kvc_pg_on_device(c->device)) return KVC_ERR_ARG;
  return launched(kvc_pg4_launch_read(c, k_out, v_out, n_tokens, d_cu, as_stream(stream)));
}

int kvc_paged4_attend(kvc_paged4* c, const void* q, void* out, float* d_lse, int32_t n_tokens, const int32_t* d_cu,
                      int32_t max_q, uint32_t flags, void* stream) {
  if (c == nullptr || !q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(d_lse, 4)) return KVC_ERR_ARG;
  if (flags & ~(uint32_t)KVC_CAUSAL) return KVC_ERR_ARG;
  if (d_cu != nullptr && max_q < 1) return KVC_ERR_ARG;
  const int rc = kvc_pg_check_rows(c->cfg, n_tokens, d_cu);
  if (rc != KVC_OK) return rc;
  if (!kvc_pg_on_device(c->device)) return KVC_ERR_ARG;
  const kvc_paged_config& g = c->cfg;
  const kvc_pg4_layout w = workspace_of(g);
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
  a.stall_ns = c->debug_stall_ns;
  a.lse = d_lse;
  a.n_tokens = n_tokens;
  a.cu = d_cu;
  a.even = n_tokens / g.batch;
  a.max_q = d_cu != nullptr ? max_q : n_tokens / g.batch;
  a.causal = (flags & KVC_CAUSAL) != 0;
  const cudaStream_t s = as_stream(stream);
  return launched(few_rows(a, g.head_dim) ? kvc_pg4_launch_decode(c, a, q, out, s) : kvc_pg4_launch_tc(c, a, q, out, s));
}

int kvc_paged4_get_error(kvc_paged4* c, void* stream, int32_t* bits) {
  if (c == nullptr || !kvc_pg_on_device(c->device)) return KVC_ERR_ARG;
  return kvc_pg_get_error(reinterpret_cast<int32_t*>(c->ws), workspace_of(c->cfg).zeroed, as_stream(stream), bits);
}

int kvc_paged4_debug_stall_waits(kvc_paged4* c, uint64_t ns) {
  if (c == nullptr) return KVC_ERR_ARG;
  c->debug_stall_ns = ns;
  return KVC_OK;
}

int kvc_paged4_destroy(kvc_paged4* c) {
  delete c;
  return KVC_OK;
}

}  // extern "C"
