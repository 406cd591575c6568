/*
 * kvc_paged.h — a paged K/V cache and the attentions that read it, on one NVIDIA GB300
 * (sm_103a).  C ABI of libkvc.so, beside kvc.h, whose conventions hold here: device
 * buffers are the caller's, every call only enqueues work on the given stream, none reads
 * device data on the host (so a step can be captured in a CUDA graph and replayed), host
 * checks that fail enqueue nothing, and bad device data (a length, an offset, a page
 * number) never faults: it is skipped, and a bit of the error word says so.
 *
 * Store.  K and V live in pools of pages, [n_pages, page_size, Hkv, D] each.  Slot p of
 * row b (its p-th token) is slot p % page_size of page d_table[b][p / page_size].  The
 * caller allots pages and keeps two device arrays, which every call reads on the device:
 *   d_table   int32 [batch, max_pages]  page numbers; entries past a row's length are not read
 *   d_kv_len  int32 [batch]             tokens of each row, those of the current step included
 * A step raises d_kv_len by each row's new tokens, appends them, and attends: the appended
 * tokens take the last positions, kv_len - n .. kv_len - 1.  No call changes either array, so
 * a step can be repeated, and the layers of a model can share both.
 *
 * Rows of a call.  n_tokens token rows stand one behind another, row b's at
 * [d_cu[b], d_cu[b + 1]) (int32 [batch + 1], not decreasing, at most n_tokens); d_cu = NULL
 * means n_tokens / batch for every row.  A row may have none.  Nothing is written for tokens behind
 * the last row's, and what their rows of q, k and v hold does not matter (attentions may read it).
 *
 * Order.  Calls on one handle share its workspace: the caller orders them (one stream, or
 * events).  Attentions that may run at the same time need a handle and a workspace each; the
 * pools, the table and the lengths may be shared.  The same holds for captured graphs that
 * may be replayed at the same time.
 */
#ifndef KVC_PAGED_H_
#define KVC_PAGED_H_

#include "kvc.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvc_paged_config {
  int32_t batch;       /* rows, 1 .. 1024                                            */
  int32_t heads;       /* H query heads                                              */
  int32_t kv_heads;    /* Hkv; H % Hkv == 0, query head h reads kv head h / (H/Hkv)  */
  int32_t head_dim;    /* D: 64 or 128                                               */
  int32_t page_size;   /* 16, 32, 64 or 128 slots                                    */
  int32_t n_pages;     /* pages of the pool                                          */
  int32_t max_pages;   /* columns of d_table; max_pages * page_size <= 2^30          */
  int32_t max_tokens;  /* most n_tokens of a kvc_paged_attend_shared call (>= 1)     */
  int32_t dtype;       /* kvc_dtype                                                  */
  float softmax_scale; /* 0 => 1/sqrt(head_dim)                                      */
} kvc_paged_config;

typedef struct kvc_paged kvc_paged;

enum {
  KVC_DEV_BAD_PAGE = 128    /* a page number outside [0, n_pages): its slots are left out  */
};

/* Flags of kvc_paged_append. */
enum {
  KVC_ROPE_HALF = 1         /* pairs (x[j], x[j + D/2]) instead of (x[2j], x[2j+1])        */
};

/* Bytes of the workspace (error word, split partials, counters, 8 bytes per row, kv head and column for
 * scores where max_pages is at most 32768); 0 for a config that kvc_paged_create would refuse. */
size_t kvc_paged_workspace_bytes(const kvc_paged_config* cfg);

/* Create a handle.
 *  k_pages, v_pages: [n_pages, page_size, Hkv, D]; d_table, d_kv_len: as above (4-byte aligned).
 *  bounds: NULL, or the key bounds that kvc_paged_attend_sparse scores pages by, [n_pages,
 *    Hkv, 2, D] of the store's type: channelwise maximum, then minimum, over a page's filled
 *    slots (NaN where one of the keys is).  kvc_paged_append keeps them.
 *  workspace: kvc_paged_workspace_bytes(cfg) bytes; its counters and error word are zeroed on `stream`.
 *  The handle belongs to the current device; calls with another one current are KVC_ERR_ARG.
 *  Errors: KVC_ERR_ARG, KVC_ERR_UNSUPPORTED (head_dim, page_size or batch not listed above), KVC_ERR_CUDA. */
int kvc_paged_create(const kvc_paged_config* cfg, void* k_pages, void* v_pages, void* bounds,
                     const int32_t* d_table, const int32_t* d_kv_len, void* workspace, void* stream,
                     kvc_paged** out);

/* Append new tokens: row b's n_b tokens go to slots kv_len_b - n_b .. kv_len_b - 1.
 *  k, v: n_tokens rows of [Hkv, D], rows kv_stride elements apart (>= Hkv * D; a multiple of
 *    16 bytes), so that they may be slices of a joint projection.
 *  d_rope: NULL (keys are stored as they come), or fp32 (cos, sin) [rope_positions][D/2][2], 16-byte aligned:
 *    the key at position p is turned by the angles of row p first, and the store holds the
 *    exact rotation rounded once to nearest-even (finite inputs), as kvc_write_rope's does.
 *    Without KVC_ROPE_HALF pair j is (x[2j], x[2j+1]), with it (x[j], x[j + D/2]).
 *  q, q_out: NULL, or queries of the same tokens (rows of [H, D], q_stride elements apart;
 *    needs d_rope) and where their rotation goes, [n_tokens, H, D]; q_out may be q where
 *    q_stride is H * D.
 *  Bounds, if the handle has them: a page whose slot 0 is written starts anew from the tokens
 *    written; one that is continued widens.  (After kv_len was taken back, a continued page's
 *    bounds still cover the tokens given up: wider than need be, never too narrow.)
 *  Two rows must not append to one page in one call.
 *  Device errors: KVC_DEV_BAD_CUSEQ (that row is skipped; where offsets go back, tokens of the rows before may be left
 *  out too), KVC_DEV_BAD_KVLEN (kv_len outside
 *  [0, max_pages * page_size], or less than the row's new tokens: skipped), KVC_DEV_BAD_PAGE
 *  (those slots are not written), KVC_DEV_BAD_POS (a position outside the rope table: that token is
 *  not written, its query neither).
 *  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged_append(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                     int64_t q_stride, void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope,
                     int32_t rope_positions, uint32_t flags, void* stream);

/* out = softmax(scale q k^T) v of every token over its row's slots [0, kv_len).
 *  q, out: [n_tokens, H, D], dense, 16-byte aligned, apart from one another; d_lse: NULL or fp32 [n_tokens, H],
 *    the natural log-sum-exp of the scaled scores.
 *  max_q: most tokens a row has (with d_cu; ignored without it); a row with more is
 *    KVC_DEV_BAD_CUSEQ.  It chooses the kernel, as lengths are on the device: single tokens under a large max_q run
 *    in the chunks' kernel.  So do the columns of the table for 17 to 32 query rows a group (tokens x heads / kv_heads), which
 *    the streaming kernel takes only where batch x kv_heads x max_pages x page_size is at most 128 K.
 *  flags: KVC_CAUSAL (token i of a row's n sees the slots up to its own, kv_len - n + i),
 *    KVC_KERNEL_SIMT (the fp32-FMA kernel for any type, a cross-check).
 *  Slots behind a row's length may hold anything.  The values of the slots that it has must be finite where a token must
 *  not see them either (causal): a weight of 0 times infinity is NaN.
 *  A token that sees no slot (kv_len 0, or causal with more tokens than slots) gets out 0 and
 *  lse -inf.  A row with a bad offset (KVC_DEV_BAD_CUSEQ) or length (KVC_DEV_BAD_KVLEN) is left
 *  unwritten; the slots of a bad page (KVC_DEV_BAD_PAGE) are left out of the softmax.
 *  More work than 2^31 tiles of 64 slots is KVC_DEV_OVERFLOW, and nothing is written.
 *  The result of a call depends on its inputs alone: the same call gives the same bits.
 *  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged_attend(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_tokens, const int32_t* d_cu,
                     int32_t max_q, uint32_t flags, void* stream);

/* kvc_paged_attend for rows whose first slots are the same pages (a common prompt): slots
 * [0, P) are read from d_prefix_pages, once for all rows' tokens together (short lists of few rows, up to 96 MB of
 * reads in all by prefix_pages, once per row), and slots [P, kv_len) from each row's own table at their usual columns (the columns below P / page_size are not read).
 *  d_prefix_pages: int32 [prefix_pages] page numbers; d_prefix_len: int32 [1] on the device, P, a
 *    multiple of page_size, 0 <= P <= prefix_pages * page_size (else KVC_DEV_BAD_KVLEN, nothing written).
 *  A row with kv_len < P sees the first kv_len slots of the prefix.  All P slots must hold finite values, also where every
 *  row is shorter: the prefix is read as one row of its own.
 *  n_tokens <= cfg.max_tokens, and tokens x heads x prefix within what 32 bits count in tiles (KVC_ERR_RANGE).  The
 *  rest as kvc_paged_attend. */
int kvc_paged_attend_shared(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_tokens,
                            const int32_t* d_cu, int32_t max_q, const int32_t* d_prefix_pages,
                            int32_t prefix_pages, const int32_t* d_prefix_len, uint32_t flags, void* stream);

/* Attention of one token per row over n_select of its pages, chosen per kv head.
 *  A page's score is the largest that any key within its bounds could have with any query
 *  of the head's group: max over g of sum_d max(q_gd hi_d, q_gd lo_d).  The first `first` pages and
 *  the newest `recent` ones are always taken (first + recent <= n_select), then those with the
 *  largest scores, of equal scores the lower column.  Scores that fp32 cannot tell apart are taken in twice its precision
 *  (off by some 2^-44 of the sum of their terms' magnitudes), so no fp32 rounding decides.
 *  A query element of 0 adds 0, whatever the bounds; a page whose score is NaN comes before all others.
 *  A row with at most n_select pages attends all of them.
 *  q, out: [batch, H, D]; d_lse: NULL or fp32 [batch, H].
 *  d_selected: int32 [batch, Hkv, n_select], written: the columns taken, ascending, then -1.
 *  A row with kv_len 0 gets out 0, lse -inf and -1 throughout; one with a bad length is left unwritten.
 *  Errors: KVC_ERR_UNSUPPORTED without bounds, KVC_ERR_RANGE for max_pages above 32768, KVC_ERR_ARG,
 *  KVC_ERR_CUDA. */
int kvc_paged_attend_sparse(kvc_paged* c, const void* q, void* out, float* d_lse, int32_t n_select, int32_t first,
                            int32_t recent, int32_t* d_selected, uint32_t flags, void* stream);

/* As kvc_get_error: synchronise `stream`, report and clear the handle's error word.  KVC_DEV_TIMEOUT in it (a wait in an
 * attention ran out, 0.5 s) means that the outputs of every call on the handle since the last kvc_paged_get_error are
 * undefined: a kernel that gave up may leave counters behind by which later calls join the parts of a row too soon or not at
 * all (nothing hangs or faults by it).  This call puts the counters right, so what follows it is sound. */
int kvc_paged_get_error(kvc_paged* c, void* stream, int32_t* bits);

/* Testing hook, as kvc_debug_stall_waits. */
int kvc_paged_debug_stall_waits(kvc_paged* c, uint64_t ns);

/* Free the host handle.  Device buffers stay with the caller. */
int kvc_paged_destroy(kvc_paged* c);

#ifdef __cplusplus
}
#endif
#endif /* KVC_PAGED_H_ */
