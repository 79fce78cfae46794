"""Paged key/value cache: the Python calls of the operators in attn_paged.h.

``cache_append`` writes the keys and values of new tokens into the pages of a
cache, ``cache_read`` takes sequences back out as packed tensors (the layout
``forward`` takes), and ``paged_forward`` is the attention of each sequence's
newest tokens (one, a few, or a prompt chunk) over everything it has cached.
There is no CPU path.

The cache of many sequences is two tensors ``[pages, page_size, Hkv, D]``
(any strides that are multiples of 16 bytes, so a head-major cache is a
transposed view), bf16 or float8_e4m3fn. Position j of sequence b is slot
``j % page_size`` of page ``block_table[b, j // page_size]``. An e4m3 cache
has an fp32 scale per (token, head), ``[pages, Hkv, page_size]``; the cached
value is code * scale.

Lengths, offsets and page numbers live on the device and may change between
replays of a captured call. What is wrong with them is found there: nothing
outside the tensors is touched, and ``check`` raises. Scratch memory is kept
per device and stream (up to 128 MiB; what a call needs beyond that goes back
to torch's allocator with the call), so calls on different streams may overlap;
a captured call takes its own from the graph's memory, and what its replays
find wrong is only seen by ``check`` if the call was given a ``workspace``: a
contiguous tensor that is zero before its first use and that calls which may
overlap do not share (what a call needs is in the error that refuses too small
a one).

Arguments are checked and marshalled by the extension module _paged_native
(csrc/python_paged.cpp).
"""
from __future__ import annotations

import torch

from . import _binding
from ._binding import AttnError, last_error


def _on(stream, tensor):
    """The context that makes ``stream`` (a torch stream or a handle) current."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=tensor.device)
    elif getattr(tensor, "is_cuda", False) and stream.device != tensor.device:
        raise ValueError("stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _result(r):
    """The outputs, unless the library refused the call (its status)."""
    if r.__class__ is int and r != _binding.ATTN_OK:
        raise AttnError(r, last_error())
    return r


def cache_append(k, v, k_cache, v_cache, block_table, seqlens_k, *, k_scale=None, v_scale=None, cu_seqlens_q=None,
                 workspace=None, stream=None):
    """Writes the new tokens' keys and values into the cache, in place.

    ``k`` and ``v`` are bf16, [B, Sq, Hkv, D], or packed [T, Hkv, D] with int32
    ``cu_seqlens_q`` (rows in front of the first sequence and behind the last
    one are ignored).
    ``seqlens_k`` (int32 [B]) counts each sequence's tokens with the new ones:
    token i of Lq goes to position seqlens_k - Lq + i. Into an e4m3 cache each
    (token, head) vector is rounded with its own scale, the smallest power of
    two s with amax / s <= 448, which goes to ``k_scale`` / ``v_scale``. Two
    new tokens must not share a slot. A token whose position or page is out
    of range is not written and reported by ``check``. Asynchronous on
    ``stream`` (default: the current torch stream).
    """
    native = _binding.paged_native()
    if stream is not None:
        with _on(stream, k_cache):
            return cache_append(k, v, k_cache, v_cache, block_table, seqlens_k, k_scale=k_scale, v_scale=v_scale,
                                cu_seqlens_q=cu_seqlens_q, workspace=workspace)
    _result(native.cache_append(k, v, k_cache, v_cache, block_table, seqlens_k, k_scale, v_scale, cu_seqlens_q,
                                workspace))


def cache_read(k_cache, v_cache, block_table, cu_seqlens_k, *, total_k=None, k_scale=None, v_scale=None, out_k=None,
               out_v=None, workspace=None, stream=None):
    """Reads sequences out of the cache; returns packed bf16 (k, v), [Tk, Hkv, D].

    Rows ``cu_seqlens_k[b]`` to ``cu_seqlens_k[b + 1]`` (int32 [B + 1]) receive
    positions 0, 1, ... of sequence b; an e4m3 cache gives code * scale,
    rounded once. ``total_k`` is the number of rows to allocate; or pass
    ``out_k`` and ``out_v``, whose rows in front of the first sequence and behind
    the last one stay as they are. A row whose position or page is out of range is not written and
    reported by ``check``. Asynchronous on ``stream`` (default: the current
    torch stream).
    """
    native = _binding.paged_native()
    if stream is not None:
        with _on(stream, k_cache):
            return cache_read(k_cache, v_cache, block_table, cu_seqlens_k, total_k=total_k, k_scale=k_scale,
                              v_scale=v_scale, out_k=out_k, out_v=out_v, workspace=workspace)
    return _result(native.cache_read(k_cache, v_cache, block_table, cu_seqlens_k, total_k, k_scale, v_scale, out_k,
                                     out_v, workspace))


def paged_forward(q, k_cache, v_cache, block_table, seqlens_k, *, causal=True, softmax_scale=None, k_scale=None,
                  v_scale=None, cu_seqlens_q=None, max_seqlen_q=None, max_seqlen_k=None, out=None, lse=None,
                  return_lse=True, workspace=None, stream=None):
    """Attention of new tokens over the paged cache; returns (O, LSE).

    ``q`` is bf16, [B, Sq, Hq, D] -> O [B, Sq, Hq, D] bf16, LSE [B, Hq, Sq]
    fp32; or packed [T, Hq, D] with int32 ``cu_seqlens_q`` and ``max_seqlen_q``
    (an upper bound of every sequence's new tokens) -> O [T, Hq, D], LSE
    [Hq, T] (rows in front of the first sequence and behind the last one stay as
    they are). ``seqlens_k`` (int32 [B]) counts each sequence's cached tokens, the
    new ones included (append them first). ``causal``: new token i of Lq sees
    positions up to seqlens_k - Lq + i; otherwise all. Rows that see nothing get
    O = 0 and LSE = -inf. D is 64 or 128; D ** -0.5 is the default
    ``softmax_scale``. Slots past a sequence's length may hold anything; cached
    values that the causal mask hides must be finite.

    ``max_seqlen_k`` bounds the cached lengths (default: what block_table can
    hold). The launch is planned for it: under a table much wider than the
    lengths, a tight bound makes short sequences up to 1.8 times as fast, and
    long e4m3 chunks up to 1.3 times.

    More than 32 rows (new tokens times Hq / Hkv) over an e4m3 cache round
    code * scale of V to bf16, and of K too with D = 64, or where the sequences
    have 512 rows or more in the mean and a bf16 copy of them fits 1 GiB of scratch
    memory (4 * Hkv * D bytes times B times ``max_seqlen_k``): without effect for
    scales that are powers of two, as ``cache_append`` writes them.

    Asynchronous on ``stream`` (default: the current torch stream).
    """
    native = _binding.paged_native()
    if stream is not None:
        with _on(stream, k_cache):
            return paged_forward(q, k_cache, v_cache, block_table, seqlens_k, causal=causal,
                                 softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale,
                                 cu_seqlens_q=cu_seqlens_q, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
                                 out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    return _result(native.paged_forward(q, k_cache, v_cache, block_table, seqlens_k, causal, softmax_scale, k_scale,
                                        v_scale, cu_seqlens_q, max_seqlen_q, max_seqlen_k, out, lse, return_lse,
                                        workspace))
