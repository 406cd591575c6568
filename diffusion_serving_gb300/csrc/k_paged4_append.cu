// Append to, and read from, the 4-bit paged store.
//
// Append: the runs, lanes and loads of the 16-bit append (k_paged_append.cu).  A lane has two vectors of 8 dims, D/2
// apart in one head, so four neighbouring lanes hold two groups of 32 dims that share a scale: two shuffles
// find a group's largest magnitude, and each lane's 8 codes make one 32-bit word.  The quotient x / s decides the code, and
// ties are common (both have few bits): x (1 / s), with 1 / s off by an ulp, is off by 2^-20, which a fused sum with 96 rounds off again (to
// 2^-17: x / s is a tie, or 2^-13 away from one), and the sum of that with 1.5 2^23 goes to the whole number, ties to even.
// 8 prompts of 512 .. 1560 tokens, 32 heads over 8 of 128, queries turned beside them: 38.4 us, 4.7 TB/s; issue slots are 66 % busy with the
// rotation and the codes, and the rest is loads waited for by the 27 warps that an SM holds at 64 registers (28 to 60 bytes spilled).  (With a branch per component of a rotated pair, not per pair, 54 us; with a longer test of a pair, codes by
// correctly rounded quotients and no prefetch 47; with a division per scale and magnitudes one by one 40.)  A step of 32 rows: 3.1
// us replayed.
//
// Read: a lane takes a word of 8 dims of the key and of the value, 4 + 1 bytes in and 16 bytes out each, of four tokens at a
// time.  8288 tokens: 7.5 us, 5.7 TB/s (one token at a time 10.5; 9360 tokens of 12 heads of 64, pages of 32: 7.4 for 6.9); a step's
// 32: 2.2 us replayed.
#include "paged4_internal.h"
#include "paged_append.h"

namespace {

// Code words of a lane's 8 dims x and of its 8 dims y, and their groups' scales, among four lanes.
struct Held {
  uint32_t w0, w1;
  uint32_t s0, s1;        // e4m3 bits
};
// Of pairs; a NaN goes on.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, const __half*) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, const __nv_bfloat16*) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <typename T>
__device__ __forceinline__ uint32_t top2(const uint4& v) {
  const T* t = nullptr;
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return max2(max2(v.x & kAbs, v.y & kAbs, t), max2(v.z & kAbs, v.w & kAbs, t), t);
}
// e4m3 of top / 7, to nearest even, 448 at most (a NaN stays one).  Ties are common (top = 7 m with five bits in m), so the quotient
// has to be the rounded exact one: q0 = x y with y = 1/7 rounded, its residual x - 7 q0, exact in a fused multiply-add, and q0 plus the
// residual times y (Markstein's correction: P. W. Markstein, Computation of elementary functions on the IBM RISC System/6000 processor,
// IBM J. Res. Dev. 34, 1990).  A test goes through every magnitude of both 16-bit types.
__device__ __forceinline__ uint32_t scale_bits(float top) {
  float x;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(top), "f"(4096.f));
  constexpr float kInv = 1.f / 7.f;
  const float q0 = x * kInv, q = __fmaf_rn(__fmaf_rn(-7.f, q0, x), kInv, q0);
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(q));
  return b & 0xFFu;
}
template <typename T>
__device__ __forceinline__ uint32_t code_word(const Vec<T>& x, uint32_t bits, float top) {
  const uint32_t h = pg4_e4m3x2(bits, (const __half*)nullptr);
  const float s = __half2float(*reinterpret_cast<const __half*>(&h));
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.f) inv = 0.f;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f(x.e[i]);
  if (!(top < 7.5f * s)) {                         // (the scale is at its end, or has few bits: else nothing rounds past 7)
    const float most = 7.f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -most), most);
  }
  // 1.5 2^23 + 8 + q: the low bits are the code; what is above them is taken off all eight at once
  uint32_t w = 0, magic = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 4 * (i >> 1) + 16 * (i & 1);
    const float q = __fadd_rn(__fmaf_rn(v[i], inv, 96.f), 12582920.f - 96.f);
    w += __float_as_uint(q) << at;
    magic += 0x4B400000u << at;
  }
  return w - magic;
}
template <typename T>
__device__ __forceinline__ Held hold(const Vec<T>& x, const Vec<T>& y) {
  const T* t = nullptr;
  const uint32_t mx = top2<T>(x.u), my = top2<T>(y.u);
  uint32_t m = max2(__byte_perm(mx, my, 0x5410), __byte_perm(mx, my, 0x7632), t);      // (x's, y's)
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o), t);
  const float2 top = pg4_floats(m, t);
  Held r;
  r.s0 = scale_bits(top.x);
  r.s1 = scale_bits(top.y);
  r.w0 = code_word(x, r.s0, top.x);
  r.w1 = code_word(y, r.s1, top.y);
  return r;
}

template <typename T, int D, int kAxes>
__global__ void __launch_bounds__(kThreads, 4)
k_paged4_append(const T* k, const T* v, const T* q, uint8_t* __restrict__ pool, T* q_out, ArgsOf<T, kAxes> a) {
  constexpr int VL = 8;
  constexpr int PH = D / 2 / VL;          // vector pairs of a head
  constexpr int NX = D / 32;              // groups of a head
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = 1 << a.ps_log2;
  int b, j;
  if (!find_run(a, b, j)) return;
  const Row r = row_of(a, b);
  if (!r.ok || r.n == 0) return;
  const int p0 = r.len - r.n;                       // position of the row's first new token
  const int column = (p0 >> a.ps_log2) + j;
  const int lo = max(p0, column << a.ps_log2), hi = min(r.len, (column + 1) << a.ps_log2);
  if (lo >= hi) return;
  const int end = !kAxes && a.rope != nullptr ? min(hi, a.rope_positions) : hi;
  if (end < hi && threadIdx.x == 0) atomicOr(a.err, KVC_DEV_BAD_POS);
  const int gw = a.groups_y;
  const int group = (int)blockIdx.y * gw + warp % gw;
  const int stride = kWarps / gw;
  if (group >= a.kv_groups) {
    append_queries<T, D, kAxes>(a, r, q, q_out, group - a.kv_groups, lo + warp / gw, end, stride, p0);
    return;
  }
  const int page = a.table[(int64_t)b * a.max_pages + column];
  if (page < 0 || page >= a.n_pages) {              // (the same for the whole block)
    if (lane == 0) atomicOr(a.err, KVC_DEV_BAD_PAGE);
    return;
  }
  const int col = group * 32 + lane;
  const bool have = col < a.kv_cols;
  const int head = have ? col / PH : 0, c = col % PH;     // (lanes past the last head take part in the shuffles)
  const int64_t src0 = (int64_t)head * D + c * VL;
  uint8_t* rec = pool + ((int64_t)page * a.Hkv + head) * kvc_pg4_record(D, a.ps_log2);
  uint32_t axes = 0;
  if constexpr (kAxes != kSlots) axes = lane_axes<T, D>(a, c, a.half);
  Places places;
  for (int p = lo + warp / gw; p < end; p += stride) {
    Vec<T> x, y, vx, vy;
    Turn<T> cs;
    const int64_t off = (int64_t)(r.t0 + p - p0) * a.kv_stride + src0;
    x.u = pg_ld(reinterpret_cast<const uint4*>(k + off));
    y.u = pg_ld(reinterpret_cast<const uint4*>(k + off + D / 2));
    if (p + stride < end) {
      const int64_t next = off + stride * a.kv_stride;
      ahead(k + next);
      ahead(k + next + D / 2);
      ahead(v + next);
      ahead(v + next + D / 2);
    }
    if constexpr (kAxes != kSlots) {
      if (!places.next(a, r.t0 + p - p0, stride, r.t0 + end - p0)) continue;               // (the same for the whole warp)
      load_turn_axes<T, D, kAxes>(cs, a.rope, places, axes, c, a.half);
    } else if (a.rope != nullptr) {
      load_turn<T, D>(cs, a.rope + (int64_t)p * (D / 2), c, a.half);
    }
    vx.u = pg_ld(reinterpret_cast<const uint4*>(v + off));
    vy.u = pg_ld(reinterpret_cast<const uint4*>(v + off + D / 2));
    if (kAxes || a.rope != nullptr) turn<T>(x, y, cs, a.half);
    const Held hk = hold(x, y), hv = hold(vx, vy);
    if (!have) continue;
    const int s = p & (ps - 1);
    const int g0 = c >> 2, g1 = NX / 2 + (c >> 2);        // groups (and 16-byte pieces) of the two words
    const int turn4 = (s >> 2) & (NX - 1);
    uint8_t* kc = rec + s * (D / 2);
    uint8_t* vc = kc + (ps * (D / 2));
    *reinterpret_cast<uint32_t*>(kc + 4 * c) = hk.w0;
    *reinterpret_cast<uint32_t*>(kc + D / 4 + 4 * c) = hk.w1;
    *reinterpret_cast<uint32_t*>(vc + 16 * (g0 ^ turn4) + 4 * (c & 3)) = hv.w0;
    *reinterpret_cast<uint32_t*>(vc + 16 * (g1 ^ turn4) + 4 * (c & 3)) = hv.w1;
    if ((c & 3) == 0) {
      uint8_t* ks = rec + ps * D + s * NX;
      uint8_t* vs = rec + ps * D + ps * NX + s;
      ks[g0] = (uint8_t)hk.s0;
      ks[g1] = (uint8_t)hk.s1;
      vs[g0 * ps] = (uint8_t)hv.s0;
      vs[g1 * ps] = (uint8_t)hv.s1;
    }
  }
}

// Eight held values.
template <typename T>
__device__ __forceinline__ uint4 unheld(uint32_t word, uint32_t bits) {
  constexpr uint32_t base = kvc_pg4_type<T>::kBase;
  const kvc_pg4_scale sc = pg4_scale<T>(pg4_e4m3x2(bits | bits << 8, (const T*)nullptr));
  return make_uint4(pg4_pair<T, 0>(word, sc, base), pg4_pair<T, 1>(word, sc, base), pg4_pair<T, 2>(word, sc, base), pg4_pair<T, 3>(word, sc, base));
}
__device__ __forceinline__ uint32_t ld_byte(const uint8_t* p) {
  uint32_t x;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4)
k_paged4_read(const uint8_t* pool, T* __restrict__ k_out, T* __restrict__ v_out, AppendArgs a) {
  constexpr int W = D / 8, NX = D / 32;
  kvc_pdl_wait();
  kvc_pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ps = 1 << a.ps_log2;
  int b, j;
  if (!find_run(a, b, j)) return;
  const Row r = row_of(a, b);
  if (!r.ok || r.n == 0) return;
  const int p0 = r.len - r.n;
  const int column = (p0 >> a.ps_log2) + j;
  const int lo = max(p0, column << a.ps_log2), hi = min(r.len, (column + 1) << a.ps_log2);
  if (lo >= hi) return;
  const int page = pg_ld(a.table + (int64_t)b * a.max_pages + column);
  if (page < 0 || page >= a.n_pages) {
    if (threadIdx.x == 0) atomicOr(a.err, KVC_DEV_BAD_PAGE);
    return;
  }
  const int gw = a.groups_y;
  const int col = ((int)blockIdx.y * gw + warp % gw) * 32 + lane;
  if (col >= a.kv_cols) return;
  const int head = col / W, w = col % W;
  const uint8_t* rec = pool + ((int64_t)page * a.Hkv + head) * kvc_pg4_record(D, a.ps_log2);
  const int stride = kWarps / gw;
  constexpr int U = 4;                    // tokens whose loads are in flight together
  for (int p = lo + warp / gw; p < hi; p += U * stride) {
    uint32_t kw[U], vw[U], ks[U], vs[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (p + i * stride >= hi) break;
      const int s = (p + i * stride) & (ps - 1);
      const int piece = (w >> 2) ^ ((s >> 2) & (NX - 1));
      kw[i] = (uint32_t)pg_ld(reinterpret_cast<const int32_t*>(rec + s * (D / 2) + 4 * w));
      vw[i] = (uint32_t)pg_ld(reinterpret_cast<const int32_t*>(rec + (ps + s) * (D / 2) + 16 * piece + 4 * (w & 3)));
      ks[i] = ld_byte(rec + ps * D + s * NX + (w >> 2));
      vs[i] = ld_byte(rec + ps * D + ps * NX + (w >> 2) * ps + s);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (p + i * stride >= hi) break;
      const int64_t dst = ((int64_t)(r.t0 + p + i * stride - p0) * a.Hkv + head) * D + 8 * w;
      if (k_out != nullptr) *reinterpret_cast<uint4*>(k_out + dst) = unheld<T>(kw[i], ks[i]);
      if (v_out != nullptr) *reinterpret_cast<uint4*>(v_out + dst) = unheld<T>(vw[i], vs[i]);
    }
  }
}

AxesArgs base_args(const kvc_paged4* c, int n_tokens, const int32_t* cu) {
  const kvc_paged_config& g = c->cfg;
  AxesArgs a{};
  a.table = c->table;
  a.kv_len = c->kv_len;
  a.cu = cu;
  a.err = reinterpret_cast<int32_t*>(c->ws);
  a.B = g.batch;
  a.n_tokens = n_tokens;
  a.ps_log2 = c->ps_log2;
  a.n_pages = g.n_pages;
  a.max_pages = g.max_pages;
  a.H = g.heads;
  a.Hkv = g.kv_heads;
  return a;
}

template <typename T, int D>
cudaError_t launch(kvc_paged4* c, const void* k, const void* v, const void* q, void* q_out, AxesArgs a, cudaStream_t s) {
  a.kv_cols = a.Hkv * (D / 16);
  a.q_cols = q != nullptr ? a.H * (D / 16) : 0;
  a.kv_groups = (a.kv_cols + 31) / 32;
  const dim3 grid = run_grid(a, a.kv_groups + (a.q_cols + 31) / 32);
  auto go = [&](auto kernel) {
    return kvc_launch_pdl(kernel, grid, dim3(kThreads), 0, s, (const T*)k, (const T*)v, (const T*)q, c->pages, (T*)q_out, a);
  };
  switch (axes_kind(a, D, 8)) {
    case kSlots: return go(k_paged4_append<T, D, kSlots>);
    case kFlat: return go(k_paged4_append<T, D, kFlat>);
    default: return go(k_paged4_append<T, D, kAny>);
  }
}
template <typename T, int D>
cudaError_t launch_read(kvc_paged4* c, void* k_out, void* v_out, AppendArgs a, cudaStream_t s) {
  a.kv_cols = a.Hkv * (D / 8);
  const dim3 grid = run_grid(a, (a.kv_cols + 31) / 32);
  return kvc_launch_pdl(k_paged4_read<T, D>, grid, dim3(kThreads), 0, s, (const uint8_t*)c->pages, (T*)k_out, (T*)v_out, a);
}

}  // namespace

cudaError_t kvc_pg4_launch_append(kvc_paged4* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                                  int64_t q_stride, void* q_out, int n_tokens, const int32_t* cu, const float* rope,
                                  int rope_positions, const kvc_rope_axes* axes, const int32_t* positions, bool half,
                                  cudaStream_t s) {
  AxesArgs a = base_args(c, n_tokens, cu);
  a.rope = reinterpret_cast<const float2*>(rope);
  a.rope_positions = rope_positions;
  a.kv_stride = kv_stride;
  a.q_stride = q_stride;
  a.half = half;
  if (axes != nullptr) set_axes(a, *axes, positions, c->cfg.head_dim);
  const bool d64 = c->cfg.head_dim == 64;
  if (c->cfg.dtype == KVC_F16) return d64 ? launch<__half, 64>(c, k, v, q, q_out, a, s) : launch<__half, 128>(c, k, v, q, q_out, a, s);
  return d64 ? launch<__nv_bfloat16, 64>(c, k, v, q, q_out, a, s) : launch<__nv_bfloat16, 128>(c, k, v, q, q_out, a, s);
}

cudaError_t kvc_pg4_launch_read(kvc_paged4* c, void* k_out, void* v_out, int n_tokens, const int32_t* cu, cudaStream_t s) {
  const AppendArgs a = base_args(c, n_tokens, cu);
  const bool d64 = c->cfg.head_dim == 64;
  if (c->cfg.dtype == KVC_F16) return d64 ? launch_read<__half, 64>(c, k_out, v_out, a, s) : launch_read<__half, 128>(c, k_out, v_out, a, s);
  return d64 ? launch_read<__nv_bfloat16, 64>(c, k_out, v_out, a, s) : launch_read<__nv_bfloat16, 128>(c, k_out, v_out, a, s);
}
