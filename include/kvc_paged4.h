/*
 * kvc_paged4.h — a paged K/V cache held in 4 bits, and the attention that reads it, on one NVIDIA GB300 (sm_103a).
 * C ABI of libkvc.so, beside kvc_paged.h, whose conventions hold here: pages, table, lengths, rows of a call, order of calls,
 * device errors.  Queries, keys, values and outputs are 16-bit (kvc_paged_config.dtype KVC_F16 or KVC_BF16); a slot takes
 * head_dim + head_dim / 16 bytes per kv head instead of 4 head_dim.
 *
 * What is held.  Of a token's key and value, each head's dims are taken in groups of 32 neighbours x (a key's after its
 * rotation and rounding to the 16-bit type):
 *   scale s = max |x| / 7, rounded to e4m3 (to nearest, ties to even; 448 at most),
 *   code  c = 8 + x / s, rounded to a whole number (ties to even) and limited to 1 .. 15; 8 where s is 0.
 * The slot then holds (c - 8) s, which both 16-bit types represent exactly.  Values of up to 3136 are held within s / 2 or
 * 7 * 2^-10 of themselves, whichever is more (groups of magnitudes up to that as zeros), larger ones, infinity too, as 3136.
 * So values should not be small: N(0, 1) keys and values, scaled down by 20 or less, are held within 10 % (rms), by 100 within 12 %,
 * by 500 not at all.
 * A group with a NaN is held as NaN throughout.
 *
 * Store.  One pool [n_pages][Hkv] of records of page_size * (D + D / 16) bytes, each:
 *   K codes  [page_size][D / 2]    dims 8 w .. 8 w + 7 are the little-endian 32-bit word w: dim 8 w + 2 i stands in
 *                                  bits 4 i .. 4 i + 3, dim 8 w + 2 i + 1 in bits 16 + 4 i .. 19 + 4 i
 *   V codes  [page_size][D / 2]    the same, but slot p's 16-byte piece x stands at piece x ^ ((p / 4) % (D / 32))
 *   K scales [page_size][D / 32]   e4m3
 *   V scales [D / 32][page_size]   e4m3
 * A record may be copied as it is (a page of another pool, host memory).
 */
#ifndef KVC_PAGED4_H_
#define KVC_PAGED4_H_

#include "kvc_rope_axes.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvc_paged4 kvc_paged4;

/* Bytes of the pool per page (all kv heads), and of the workspace (error word, split partials, counters); 0 for a config
 * that kvc_paged4_create would refuse. */
size_t kvc_paged4_page_bytes(const kvc_paged_config* cfg);
size_t kvc_paged4_workspace_bytes(const kvc_paged_config* cfg);

/* Create a handle, as kvc_paged_create.
 *  pages: n_pages * kvc_paged4_page_bytes(cfg) bytes, 16-byte aligned.
 *  cfg->max_tokens is not looked at beyond being 1 at least.
 *  Errors: KVC_ERR_ARG, KVC_ERR_UNSUPPORTED (dtype KVC_F32 too), KVC_ERR_CUDA. */
int kvc_paged4_create(const kvc_paged_config* cfg, void* pages, const int32_t* d_table, const int32_t* d_kv_len,
                      void* workspace, void* stream, kvc_paged4** out);

/* Append new tokens, as kvc_paged_append (axes NULL, d_positions NULL: positions are slots) or kvc_paged_append_axes: keys
 * are turned and rounded to the 16-bit type, then keys and values are held in 4 bits as above.  Nothing but the slots of
 * the new tokens is written.  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged4_append(kvc_paged4* c, const void* k, const void* v, int64_t kv_stride, const void* q, int64_t q_stride,
                      void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope, int32_t rope_positions,
                      const kvc_rope_axes* axes, const int32_t* d_positions, uint32_t flags, void* stream);

/* What the store holds of each row's last n_b slots, kv_len_b - n_b .. kv_len_b - 1 (with n_b = kv_len_b, of all of them).
 *  k_out, v_out: [n_tokens, Hkv, D] dense, 16-byte aligned, apart from one another; either may be NULL.
 *  Device errors, each leaving what it concerns unwritten: KVC_DEV_BAD_CUSEQ, KVC_DEV_BAD_KVLEN, KVC_DEV_BAD_PAGE, as
 *  kvc_paged_append has them.  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged4_read(kvc_paged4* c, void* k_out, void* v_out, int32_t n_tokens, const int32_t* d_cu, void* stream);

/* out = softmax(scale q k^T) v of every token over the values held of its row's slots [0, kv_len), as kvc_paged_attend
 * (with whose results over the same values it agrees but for rounding; flags: KVC_CAUSAL alone).  Slots behind a row's length
 * may hold any bits.  Weights are rounded to fp16 before their product with the values, whichever the 16-bit type.
 *  max_q, the batch and the columns of the table choose the kernel (lengths are on the device), and with it the last bits: more than
 *  16 query rows a group (tokens x heads / kv_heads) take the streaming kernel, in up to four passes, only where few items and the
 *  table's slots over them make that faster; a table sized for far longer rows sends drafted tokens to the chunks' kernel.
 *  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged4_attend(kvc_paged4* c, const void* q, void* out, float* d_lse, int32_t n_tokens, const int32_t* d_cu,
                      int32_t max_q, uint32_t flags, void* stream);

/* As kvc_paged_get_error, kvc_paged_debug_stall_waits, kvc_paged_destroy. */
int kvc_paged4_get_error(kvc_paged4* c, void* stream, int32_t* bits);
int kvc_paged4_debug_stall_waits(kvc_paged4* c, uint64_t ns);
int kvc_paged4_destroy(kvc_paged4* c);

#ifdef __cplusplus
}
#endif
#endif /* KVC_PAGED4_H_ */
