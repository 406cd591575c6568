// Joins the partial states that attention blocks left in the workspace, spread over the whole GPU: a
// tensor-core item's partial is 64 KB (128 rows x 128 dims), so one block that joined an item's ten or
// twenty would take longer than the attention itself.
//
// Both kernels take a warp per query row, four dims a lane, eight partials in flight.  They are
// launched as programmatic dependents of the attention kernel and work out their share (lengths,
// items) while it still runs: it has begun, so whatever precedes it is done.  Bound by L2 reads of
// the partials: 5 us for 8 heads' prefix state of 64 rows (19 partials each), most of it the launch and one round of loads.
#include "paged_finish.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRowBlocks = 8;             // blocks per split item

// Block (c, y) joins rows y * 8 + warp, ... of the item that begins in k_paged_tc's block c and goes on behind it, if
// there is one.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
k_paged_join(T* __restrict__ out, kvc_pg_args a) {
  constexpr int R = KVC_PG_TC_ROWS;
  extern __shared__ __align__(16) uint8_t smem[];
  kvc_pg_sched<R, KVC_PG_TC_TILE> sch;
  sch.init(a, smem, KVC_PG_TC_MIN, KVC_PG_TC_WHOLE, KVC_PG_TC_COST, KVC_PG_GRID);
  // the item at the end of the block's stretch
  const long long end = (long long)(blockIdx.x + 1) * sch.per;
  const bool any = end < sch.total;
  kvc_pg_item it;
  int c0 = 0, c1 = 0;
  if (any) {
    it = sch.at(a, (int)end - 1);
    sch.span(it, &c0, &c1);
  }
  kvc_pdl_wait();
  kvc_pdl_release();
  if (!any || c0 != (int)blockIdx.x || c1 == c0) return;
  const bool prefix = a.phase == 2 && sch.lo > 0;
  const int rows = min(sch.T, it.r.n - it.k * sch.T) * a.Gv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = 4 * (lane % (D / 4));
  for (int r = blockIdx.y * kWarps + warp; r < rows; r += gridDim.y * kWarps) {
    const int64_t at = pg_at(a, sch, it, r);
    float M = -INFINITY, L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (prefix) {
      float2 ml;
      float4 y;
      pg_load_prefix<D>(a, at, d, &ml, &y);
      pg_join1(M, L, x, ml, y);
    }
    pg_join(c1 - c0 + 1, M, L, x,
            [&](int i, float2* ml, float4* y) { pg_load_part<R, D, true>(a.part, 2 * (c0 + i) + (i == 0 ? 1 : 0), r, d, ml, y); });
    if (lane < D / 4) pg_emit<T, D>(a, out, at, d, M, L, x);
  }
}

// Phase 1's items all have the same tiles, so which blocks held an item, and in which slots (item + block) they left
// it, follows from the prefix length.
template <int D, int R>
__global__ void __launch_bounds__(kThreads)
k_paged_join_prefix(int TS, int cost, int grid, kvc_pg_args a) {
  const int T = R / a.Gv, m = (a.n_tokens + T - 1) / T, items = m * a.Hv;
  const int prefix = *a.prefix_len;
  const int tiles = prefix > TS ? (prefix + TS - 1) / TS : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = 4 * (lane % (D / 4));
  const int r = blockIdx.y * kWarps + warp;
  kvc_pdl_wait();
  kvc_pdl_release();
  if (prefix <= 0 || !pg_prefix_ok(a, prefix) || r >= T * a.Gv) return;
  // (as kvc_pg_sched has it)
  int per, stride = tiles + cost, lead = cost;
  if (items <= grid) {
    pg_even(tiles, items, grid, 1, 1, &per, &stride);
    lead = 0;
  } else {
    per = (items * stride + grid - 1) / grid;
  }
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int vh = item / m, t = (item % m) * T + r / a.Gv;
    if (t >= a.n_tokens) continue;
    const int c0 = (item * stride + lead) / per, c1 = (item * stride + lead + tiles - 1) / per;
    float M = -INFINITY, L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    pg_join(c1 - c0 + 1, M, L, x,
            [&](int i, float2* ml, float4* y) { pg_load_part<R, D>(a.pre, item + c0 + i, r, d, ml, y); });
    const int64_t at = (int64_t)t * a.H + vh * a.Gv + r % a.Gv;
    if (lane < D / 4) *reinterpret_cast<float4*>(a.pre_o + at * D + d) = x;
    if (lane == 0) a.pre_ml[at] = make_float2(M, L);
  }
}

template <int D>
cudaError_t launch_prefix(const kvc_pg_args& a, int R, int TS, int cost, int grid, cudaStream_t s) {
  const int T = R / a.Gv;
  const int64_t items = (int64_t)a.Hv * ((a.n_tokens + T - 1) / T);
  const unsigned gx = (unsigned)(items < 4 * KVC_PG_GRID ? items : 4 * KVC_PG_GRID);
  if (R == KVC_PG_TC_ROWS)
    return kvc_launch_pdl(k_paged_join_prefix<D, KVC_PG_TC_ROWS>, dim3(gx, R / kWarps), dim3(kThreads), 0, s, TS, cost,
                          grid, a);
  return kvc_launch_pdl(k_paged_join_prefix<D, KVC_PG_SIMT_ROWS>, dim3(gx, R / kWarps), dim3(kThreads), 0, s, TS, cost,
                          grid, a);
}

template <typename T, int D>
cudaError_t launch(const kvc_pg_args& a, void* out, cudaStream_t s) {
  return kvc_launch_pdl(k_paged_join<T, D>, dim3(KVC_PG_GRID, kRowBlocks), dim3(kThreads), pg_sched_bytes(a.B), s,
                        (T*)out, a);
}

}  // namespace

cudaError_t kvc_pg_launch_join_prefix(const kvc_paged* c, const kvc_pg_args& a, bool simt, cudaStream_t s) {
  const int R = simt ? KVC_PG_SIMT_ROWS : KVC_PG_TC_ROWS, TS = simt ? KVC_PG_SIMT_TILE : KVC_PG_TC_TILE;
  const int cost = simt ? 1 : KVC_PG_TC_COST, grid = simt ? KVC_PG_GRID_SIMT : KVC_PG_GRID;
  return c->cfg.head_dim == 64 ? launch_prefix<64>(a, R, TS, cost, grid, s) : launch_prefix<128>(a, R, TS, cost, grid, s);
}

cudaError_t kvc_pg_launch_join(const kvc_paged* c, const kvc_pg_args& a, void* out, cudaStream_t s) {
  const bool d64 = c->cfg.head_dim == 64;
  if (c->cfg.dtype == KVC_F16) return d64 ? launch<__half, 64>(a, out, s) : launch<__half, 128>(a, out, s);
  return d64 ? launch<__nv_bfloat16, 64>(a, out, s) : launch<__nv_bfloat16, 128>(a, out, s);
}
