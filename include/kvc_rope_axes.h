/*
 * kvc_rope_axes.h — rotary positions with several axes (time, height, width of images and video) for the paged
 * cache of kvc_paged.h, whose conventions hold here.
 *
 * A token has one position per axis, and each of its head's D/2 rotated pairs goes by one axis: pair j of a token at
 * positions p is turned by row p[pair_axis[j]] of the table of angles, column j.  With one axis these are plain positions
 * that need not be slot numbers (after images, whose tokens share positions, or in a store that has given up slots).
 */
#ifndef KVC_ROPE_AXES_H_
#define KVC_ROPE_AXES_H_

#include "kvc_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvc_rope_axes {
  int32_t n_axes;          /* 1 .. 4                                                       */
  uint8_t pair_axis[64];   /* axis of pair j, < n_axes; the first head_dim / 2 are looked at */
} kvc_rope_axes;

/* kvc_paged_append with keys and queries turned at given positions.
 *  axes: on the host, read by the call itself.
 *  d_positions: int32 [n_tokens, axes->n_axes] on the device (4-byte aligned), by the call's token rows.
 *  d_rope: needed.  Slots, bounds and all else as kvc_paged_append has them; in particular tokens go to slots
 *    kv_len - n .. kv_len - 1 whatever their positions.
 *  Device errors: as kvc_paged_append; KVC_DEV_BAD_POS for a token with a position outside [0, rope_positions): that
 *    token is not written, its query neither, and it adds nothing to its page's bounds (a page that none of the call's
 *    tokens is written to keeps its bounds).
 *  Errors: KVC_ERR_ARG, KVC_ERR_CUDA. */
int kvc_paged_append_axes(kvc_paged* c, const void* k, const void* v, int64_t kv_stride, const void* q,
                          int64_t q_stride, void* q_out, int32_t n_tokens, const int32_t* d_cu, const float* d_rope,
                          int32_t rope_positions, const kvc_rope_axes* axes, const int32_t* d_positions, uint32_t flags,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KVC_ROPE_AXES_H_ */
