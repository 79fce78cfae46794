/*
 * attn_rotary.h - C ABI of rotary positions: queries and keys turned by their
 * tokens' positions, in one pass over them. Part of libattn_fwd.so; status
 * codes, streams and error texts are attn_fwd.h's.
 *
 * Of each head's D depths the first R = rotary_dim are turned, in R / 2 pairs
 * (x1, x2): depths (i, i + R / 2), or with `interleaved` (2 i, 2 i + 1). With
 * c = table[p][i] and s = table[p][R / 2 + i] for a token at position p
 *     y1 = x1 c - x2 s,   y2 = x2 c + x1 s      (inverse: s negated)
 * in fp32, every product and sum rounded, and y rounded once to bf16. The other
 * depths are copied. The table holds what the model wants there (cosines and
 * sines of frequencies scaled in whatever way, times an amplitude). Rotating
 * back (inverse) is also the gradient of a rotation.
 *
 * Position of token i of the n_b tokens of sequence b: positions[row], or, if
 * positions is NULL, seqlens[b] - n_b + i (seqlens counts the new tokens too),
 * or, if that is NULL as well, i.
 *
 * Every pointer is a DEVICE pointer owned by the caller; the library
 * allocates nothing. The call enqueues on `stream` and returns without
 * synchronising; invalid arguments are reported before anything is enqueued.
 * What only the device can see, positions outside the table and offsets out of
 * order, is reported through attn_fwd_check(workspace): rows at such positions
 * are not written, and none of them where offsets decrease.
 */
#ifndef ATTN_ROTARY_H
#define ATTN_ROTARY_H

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_rotary_params {
  const void *q;               /* bf16: fixed [B][S][Hq][D] / packed [T][Hq][D] */
  const void *k;               /* the same with Hk heads; NULL: none (num_heads_k = 0) */
  void *q_out;                 /* bf16, q's shape, written; may be q itself with q's strides, and
                                  else shares no memory with q or k (rows of other strides may
                                  not even lie among q's), nor its rows with one another */
  void *k_out;
  const float *table;          /* [num_positions][rotary_dim] contiguous, 16-byte aligned: cosines,
                                  then sines */
  const int32_t *positions;    /* fixed [B][S] / packed [T], contiguous; or NULL */
  const int32_t *seqlens;      /* [B], or NULL */
  const int32_t *cu_seqlens;   /* packed: [B + 1] offsets of the rows. Rows in front of
                                  cu_seqlens[0] and from cu_seqlens[B] on are left as they are */
  void *workspace;             /* ATTN_FWD_WORKSPACE_BYTES, as attn_fwd_params.workspace: the
                                  device error record */
  int64_t q_stride[3];         /* elements: [0] batch (unused when packed), [1] token, [2] head;
                                  multiples of 16 bytes, depth contiguous */
  int64_t k_stride[3];
  int64_t q_out_stride[3];
  int64_t k_out_stride[3];
  int32_t batch;               /* B */
  int32_t seqlen;              /* fixed: S */
  int32_t total;               /* packed: T */
  int32_t num_heads_q;
  int32_t num_heads_k;
  int32_t head_dim;            /* D, a multiple of 8 up to 4096 */
  int32_t num_positions;
  int32_t rotary_dim;          /* R, even, 2 to D */
  int32_t interleaved;
  int32_t inverse;
} attn_rotary_params;

/* sizeof(attn_rotary_params) as compiled into the library (binding check). */
size_t attn_rotary_params_size(void);

/* Validates `p` and enqueues the rotation. */
attn_status attn_rotary(const attn_rotary_params *p, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_ROTARY_H */
