/*
 * attn_paged.h - C ABI of the paged key/value cache: writing new tokens into
 * it, reading sequences back out of it, and attention over it. Part of
 * libattn_fwd.so; status codes, streams and error texts are attn_fwd.h's.
 *
 * The cache keeps K and V of many sequences in pages of page_size tokens:
 * position j of sequence b is slot j % page_size of page
 * block_table[b][j / page_size]. It holds bf16, or float8_e4m3fn with one fp32
 * scale per (token, head): the cached value is code * scale.
 *
 *   append  token i of the Lq_b new tokens of sequence b goes to position
 *           seqlens_k[b] - Lq_b + i (seqlens_k counts the new tokens too).
 *           e4m3: with a the largest finite |x_d| of the (token, head) vector,
 *           scale = the smallest power of two s >= 2^-126 with a / s <= 448
 *           (1 if a = 0) and code_d = x_d / s rounded to nearest even. A
 *           power of two makes x / s exact and costs no accuracy (a floating
 *           code has the same relative error at any scale). Infinities become
 *           +-448 s, NaN stays NaN.
 *   read    positions 0 .. cu_seqlens_k[b+1] - cu_seqlens_k[b] - 1 of sequence
 *           b, as packed bf16 rows (e4m3: code * scale, rounded once).
 *   attend  for new token i of sequence b and query head h, hk = h / (Hq / Hkv):
 *             J_i   = { j < Lk_b : !causal || j <= Lk_b - Lq_b + i }
 *             s_ij  = scale * (q_i . K_j)
 *             LSE_i = ln sum_{j in J_i} exp(s_ij)
 *             O_i   = sum_{j in J_i} exp(s_ij - LSE_i) * V_j     bf16, rounded once
 *           (the causal mask is aligned to the END of the keys: the new
 *           tokens are the last ones cached). The weights are rounded to bf16
 *           before the P.V product, as in attn_fwd (to f16 where an e4m3 cache
 *           allows); sums and the softmax statistics are fp32. Over an e4m3 cache,
 *           calls of more than 32 rows (seqlen_q * Hq / Hkv) round more:
 *             V: code * scale, to bf16, once.
 *             K, D = 64: the same.
 *             K, D = 128: the same where the sequences have 512 rows or more in the
 *               mean and the bf16 copy of them that is then made takes 1 GiB at
 *               most (4 * Hkv * D bytes for each of B * seqlen_k tokens, seqlen_k
 *               rounded up to 128). Else K is exact, and q is 2^e (q1 + q2) with
 *               e4m3 q1 and q2: exact for values above 2^-9 of the row's largest,
 *               within 2^-17 of the largest below.
 *           Rounding code * scale to bf16 changes nothing when scales are powers of
 *           two, as append's are (but for products below bf16's subnormals, 2^-133);
 *           other scales move a score by up to 2^-8 of scale * sum_d |q_id K_jd|.
 *           Rows with an empty J_i get O_i = 0 and
 *           LSE_i = -inf. Slots at or past position Lk_b are never used, they
 *           may hold anything; cached values in front of Lk_b that the causal
 *           mask hides must be finite (their weight is zero).
 *
 * Every pointer is a DEVICE pointer owned by the caller; the library
 * allocates nothing. Calls enqueue on `stream` and return without
 * synchronising; invalid arguments are reported before anything is enqueued.
 * What only the device can see is checked there and reported through
 * attn_fwd_check(workspace): lengths out of range, offsets out of order, page
 * numbers outside the cache. Such a call touches no memory outside the
 * tensors: append and read skip the rows concerned (all rows, where offsets
 * decrease), attend computes them from other data (nothing of that call's output
 * can be trusted). A call without rows enqueues nothing, and nothing is checked.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes at the start of attn_paged_fwd's workspace that are zero before its
 * first use and after every call (and its least size). */
#define ATTN_PAGED_ZEROED_BYTES 8192

typedef struct attn_kv_cache {
  void *k;                    /* [P][page_size][Hkv][D], bf16 or e4m3 (dtype), 16-byte aligned */
  void *v;                    /* the same shape and type */
  float *k_scale;             /* e4m3 only: [P][Hkv][page_size] contiguous, 16-byte aligned */
  float *v_scale;
  const int32_t *block_table; /* [B][max_pages], row stride table_stride, entries contiguous */
  int64_t k_stride[3];        /* elements: [0] page, [1] token, [2] head; depth contiguous;
                                 multiples of 16 bytes, positive where the dimension is
                                 larger than 1 */
  int64_t v_stride[3];
  int64_t table_stride;       /* elements between the rows of block_table */
  int32_t dtype;              /* attn_dtype of k and v */
  int32_t num_pages;          /* P */
  int32_t page_size;          /* a power of two, 16 to 65536 */
  int32_t max_pages;          /* columns of block_table */
  int32_t num_heads_kv;       /* Hkv */
  int32_t head_dim;           /* D, 64 or 128 */
  int32_t batch;              /* B, sequences */
} attn_kv_cache;

typedef struct attn_cache_append_params {
  attn_kv_cache cache;
  const void *k;               /* bf16 new rows: fixed [B][Sq][Hkv][D] / packed [Tq][Hkv][D] */
  const void *v;
  const int32_t *seqlens_k;    /* [B]: tokens in the cache, the new ones included */
  const int32_t *cu_seqlens_q; /* packed only: [B+1] offsets of the new rows; rows in front of
                                  cu_seqlens_q[0] and from cu_seqlens_q[B] on are ignored */
  void *workspace;             /* ATTN_FWD_WORKSPACE_BYTES, as attn_fwd_params.workspace: the
                                  device error record */
  int64_t k_stride[3];         /* elements: [0] batch (unused when packed), [1] token, [2] head */
  int64_t v_stride[3];
  int32_t seqlen_q;            /* fixed: Sq */
  int32_t total_q;             /* packed: Tq */
} attn_cache_append_params;

typedef struct attn_cache_read_params {
  attn_kv_cache cache;
  void *k;                     /* bf16 rows, written: [Tk][Hkv][D] */
  void *v;
  const int32_t *cu_seqlens_k; /* [B+1] offsets of each sequence's rows; rows in front of
                                  cu_seqlens_k[0] and from cu_seqlens_k[B] on are left as
                                  they are */
  void *workspace;             /* the device error record, see append */
  int64_t k_stride[2];         /* elements: [0] token, [1] head */
  int64_t v_stride[2];
  int32_t total_k;             /* Tk */
} attn_cache_read_params;

typedef struct attn_paged_params {
  attn_kv_cache cache;
  const void *q;               /* bf16: fixed [B][Sq][Hq][D] / packed [Tq][Hq][D] */
  void *o;                     /* bf16, the same shape, written */
  float *lse;                  /* fixed [B][Hq][Sq] / packed [Hq][Tq] contiguous, written; may be NULL */
  const int32_t *seqlens_k;    /* [B]: Lk_b */
  const int32_t *cu_seqlens_q; /* packed only: [B+1]; rows of o in front of cu_seqlens_q[0] and
                                  from cu_seqlens_q[B] on are left as they are */
  void *workspace;             /* >= attn_paged_workspace_bytes(p), 256-byte aligned; its first
                                  ATTN_PAGED_ZEROED_BYTES zero-filled once before its first use
                                  (every call leaves them zeroed). Calls that share a workspace
                                  must not overlap. */
  size_t workspace_bytes;
  int64_t q_stride[3];         /* elements: [0] batch (unused when packed), [1] token, [2] head;
                                  multiples of 16 bytes */
  int64_t o_stride[3];
  int32_t seqlen_q;            /* fixed: Sq; packed: an upper bound of every Lq_b */
  int32_t seqlen_k;            /* an upper bound of every Lk_b, at most max_pages * page_size */
  int32_t total_q;             /* packed: Tq */
  int32_t num_heads_q;         /* Hq, a multiple of Hkv */
  int32_t causal;
  float softmax_scale;         /* > 0 */
} attn_paged_params;

/* sizeof of the three parameter structs as compiled into the library
 * (binding check): which = 0 append, 1 read, 2 attend. */
size_t attn_paged_params_size(int32_t which);

/* Validates `p` and enqueues the write of its new rows. Two rows must not go
 * to the same slot (sequences that share a page may only append behind it). */
attn_status attn_cache_append(const attn_cache_append_params *p, attn_stream_t stream);

/* Validates `p` and enqueues the read. */
attn_status attn_cache_read(const attn_cache_read_params *p, attn_stream_t stream);

/* Validates `p` and enqueues the attention. */
attn_status attn_paged_fwd(const attn_paged_params *p, attn_stream_t stream);

/* Workspace bytes attn_paged_fwd needs for `p` on the current device (an
 * invalid `p` or NULL gives ATTN_PAGED_ZEROED_BYTES). Depends on sizes only,
 * never on device data. */
size_t attn_paged_workspace_bytes(const attn_paged_params *p);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PAGED_H */
