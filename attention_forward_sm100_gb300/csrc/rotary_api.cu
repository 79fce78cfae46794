// Host side of the C ABI declared in include/attn_rotary.h.
#include <string.h>

#include "rotary.h"
#include "rows_host.h"

namespace {

using af::report_error;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status check_rows(const char* what, const void* p, const int64_t* stride, int first) {
  if (p == nullptr || !aligned(p, 16))
    return report_error(ATTN_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", what);
  for (int i = first; i < 3; ++i)
    if (stride[i] < 0 || (stride[i] * 2) % 16)
      return report_error(ATTN_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", what);
  return ATTN_OK;
}

bool no_rows(const attn_rotary_params* p) {
  return p->batch == 0 || (p->cu_seqlens != nullptr ? p->total : p->seqlen) == 0 || p->num_heads_q + p->num_heads_k == 0;
}

attn_status check(const attn_rotary_params* p) {
  if (p == nullptr) return report_error(ATTN_ERR_INVALID_ARG, "params is NULL");
  if (p->batch < 0 || p->seqlen < 0 || p->total < 0 || p->num_heads_q < 0 || p->num_heads_k < 0 || p->num_positions < 0)
    return report_error(ATTN_ERR_INVALID_ARG, "negative size");
  if (p->num_heads_q > 16384 || p->num_heads_k > 16384) return report_error(ATTN_ERR_UNSUPPORTED, "more than 16384 heads");
  if (p->head_dim <= 0 || p->head_dim > 4096 || p->head_dim % 8)
    return report_error(ATTN_ERR_UNSUPPORTED, "head_dim %d is not a multiple of 8 up to 4096", p->head_dim);
  if (p->rotary_dim < 2 || p->rotary_dim > p->head_dim || p->rotary_dim % 2)
    return report_error(ATTN_ERR_INVALID_ARG, "rotary_dim %d is not an even number from 2 to head_dim", p->rotary_dim);
  const bool packed = p->cu_seqlens != nullptr;
  if (!packed && (int64_t)p->batch * p->seqlen > 0x7fffffffll)
    return report_error(ATTN_ERR_UNSUPPORTED, "more than 2^31 tokens");
  if (no_rows(p)) return ATTN_OK;
  attn_status st;
  const int first = packed ? 1 : 0;
  if (p->num_heads_q > 0) {
    if ((st = check_rows("q", p->q, p->q_stride, first)) != ATTN_OK) return st;
    if ((st = check_rows("q_out", p->q_out, p->q_out_stride, first)) != ATTN_OK) return st;
  }
  if (p->num_heads_k > 0) {
    if ((st = check_rows("k", p->k, p->k_stride, first)) != ATTN_OK) return st;
    if ((st = check_rows("k_out", p->k_out, p->k_out_stride, first)) != ATTN_OK) return st;
  }
  const int64_t n0 = packed ? 1 : p->batch, n1 = packed ? p->total : p->seqlen;
  const af::RowsAt q(p->q, n0, n1, p->num_heads_q, p->q_stride, p->head_dim),
      k(p->k, n0, n1, p->num_heads_k, p->k_stride, p->head_dim),
      q_out(p->q_out, n0, n1, p->num_heads_q, p->q_out_stride, p->head_dim),
      k_out(p->k_out, n0, n1, p->num_heads_k, p->k_out_stride, p->head_dim);
  if (const char* wrong = af::misplaced(q_out, q, {k, k_out}))
    return report_error(ATTN_ERR_INVALID_ARG, "q_out %s", wrong);
  if (const char* wrong = af::misplaced(k_out, k, {q, q_out}))
    return report_error(ATTN_ERR_INVALID_ARG, "k_out %s", wrong);
  if (p->num_positions > 0 && (p->table == nullptr || !aligned(p->table, 16)))
    return report_error(ATTN_ERR_INVALID_ARG, "table must be non-NULL and 16-byte aligned");
  if (!aligned(p->positions, 4) || !aligned(p->seqlens, 4) || !aligned(p->cu_seqlens, 4))
    return report_error(ATTN_ERR_INVALID_ARG, "positions, seqlens and cu_seqlens must be 4-byte aligned");
  if (p->workspace == nullptr || !aligned(p->workspace, 256))
    return report_error(ATTN_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  return ATTN_OK;
}

}  // namespace

extern "C" {

size_t attn_rotary_params_size(void) { return sizeof(attn_rotary_params); }

attn_status attn_rotary(const attn_rotary_params* p, attn_stream_t stream) {
  report_error(ATTN_OK, "%s", "");
  const attn_status st = check(p);
  if (st != ATTN_OK) return st;
  if (no_rows(p)) return ATTN_OK;
  const bool packed = p->cu_seqlens != nullptr;
  af::RotaryParams a;
  memset(&a, 0, sizeof(a));
  const int64_t* in[2] = {p->q_stride, p->k_stride};
  const int64_t* out[2] = {p->q_out_stride, p->k_out_stride};
  a.in[0] = static_cast<const uint8_t*>(p->q);
  a.in[1] = static_cast<const uint8_t*>(p->k);
  a.out[0] = static_cast<uint8_t*>(p->q_out);
  a.out[1] = static_cast<uint8_t*>(p->k_out);
  for (int i = 0; i < 2; ++i) {
    a.in_b[i] = packed ? 0 : in[i][0] * 2;
    a.in_t[i] = in[i][1] * 2;
    a.in_h[i] = in[i][2] * 2;
    a.out_b[i] = packed ? 0 : out[i][0] * 2;
    a.out_t[i] = out[i][1] * 2;
    a.out_h[i] = out[i][2] * 2;
  }
  a.positions = p->positions;
  a.seqlens = p->seqlens;
  a.cu = p->cu_seqlens;
  a.ws = static_cast<uint32_t*>(p->workspace);
  a.tokens = packed ? p->total : (int64_t)p->batch * p->seqlen;
  a.heads[0] = p->num_heads_q;
  a.heads[1] = p->num_heads_k;
  a.batch = p->batch;
  a.seqlen = p->seqlen;
  a.num_positions = p->num_positions;
  const cudaError_t e = af::rotary_launch(a, p->head_dim, p->rotary_dim, p->interleaved != 0, p->inverse != 0, p->table,
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "rotary launch failed: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // extern "C"
