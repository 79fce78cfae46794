"""Paged key/value cache: ctypes binding of the operators in attn_paged.h.

``cache_append`` writes the keys and values of new tokens into the pages of a
cache, ``cache_read`` takes sequences back out as packed tensors (the layout
``forward`` takes), and ``paged_forward`` is the attention of each sequence's
newest tokens (one, a few, or a prompt chunk) over everything it has cached.
As in ``_binding``, this module only checks and marshals arguments; there is
no CPU path.

The cache of many sequences is two tensors ``[pages, page_size, Hkv, D]``
(any strides that are multiples of 16 bytes, so a head-major cache is a
transposed view), bf16 or float8_e4m3fn. Position j of sequence b is slot
``j % page_size`` of page ``block_table[b, j // page_size]``. An e4m3 cache
has an fp32 scale per (token, head), ``[pages, Hkv, page_size]``; the cached
value is code * scale.

Lengths, offsets and page numbers live on the device and may change between
replays of a captured call. What is wrong with them is found there: nothing
outside the tensors is touched, and ``check`` raises.
"""
from __future__ import annotations

import struct

import torch

from . import _binding
from ._binding import ATTN_OK, DTYPES, WORKSPACE_BYTES, AttnError, last_error, lib

# attn_kv_cache, then the rest of each parameter struct (native alignment)
_CACHE = "5P7q7i4x"
_APPEND = struct.Struct("@" + _CACHE + "5P6q2i")
_READ = struct.Struct("@" + _CACHE + "4P4qi4x")
_PAGED = struct.Struct("@" + _CACHE + "6PN6q5if")

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

_checked_layout = False
_bytes_by_sizes = {}


def _library():
    global _checked_layout
    L = lib()
    if not _checked_layout:
        for which, s in enumerate((_APPEND, _READ, _PAGED)):
            if L.attn_paged_params_size(which) != s.size:
                raise RuntimeError("attn_paged.h layout mismatch between the binding and the library")
        _checked_layout = True
    return L


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _strides(t):
    """Element strides without the last dimension's; 0 where a dimension has size 1."""
    return [0 if n == 1 else s for n, s in zip(t.shape[:-1], t.stride())]


def _int32(name, t, shape):
    _need(t.dtype == torch.int32 and t.is_contiguous(), f"{name} must be a contiguous int32 tensor")
    _need(tuple(t.shape) == shape, f"{name} shape {tuple(t.shape)} != {shape}")


def _check_cache(k_cache, v_cache, block_table, k_scale, v_scale):
    """Checks the cache tensors; returns the fields of attn_kv_cache."""
    _need(k_cache.dim() == 4 and k_cache.shape == v_cache.shape,
          "k_cache and v_cache must be [pages, page_size, Hkv, D] of one shape")
    _need(k_cache.dtype in DTYPES, f"unsupported cache dtype {k_cache.dtype}")
    _need(k_cache.dtype == v_cache.dtype, "k_cache and v_cache must have one dtype")
    pages, page_size, heads, dim = k_cache.shape
    _need(k_cache.stride(3) == 1 and v_cache.stride(3) == 1, "the cache's depth must be contiguous")
    _need(block_table.dim() == 2 and block_table.dtype == torch.int32, "block_table must be an int32 [B, max_pages] tensor")
    batch, width = block_table.shape
    _need(width <= 1 or block_table.stride(1) == 1, "the rows of block_table must be contiguous")
    scales = (0, 0)
    if k_cache.dtype == torch.float8_e4m3fn:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t is not None, f"an e4m3 cache needs {name}")
            _need(t.dtype == torch.float32 and t.is_contiguous() and tuple(t.shape) == (pages, heads, page_size),
                  f"{name} must be a contiguous fp32 [pages, Hkv, page_size] tensor")
        scales = (k_scale.data_ptr(), v_scale.data_ptr())
    else:
        _need(k_scale is None and v_scale is None, "a bf16 cache takes no scales")
    return (k_cache.data_ptr(), v_cache.data_ptr(), *scales, block_table.data_ptr(), *_strides(k_cache),
            *_strides(v_cache), 0 if batch == 1 else block_table.stride(0), DTYPES[k_cache.dtype], pages, page_size,
            width, heads, dim, batch)


def _check_device(tensors):
    """All on one CUDA device; returns its index."""
    index = None
    for name, t in tensors:
        if t is None:
            continue
        i = t.get_device()
        _need(i >= 0, f"{name} must be a CUDA tensor (this library has no CPU path)")
        _need(index is None or i == index, f"{name} is on another device than the other tensors")
        index = i
    return index


def _elsewhere(index, stream):
    """A context that makes device ``index`` and ``stream`` current, or None if they are."""
    if stream is not None:
        return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else
                                 torch.cuda.ExternalStream(int(stream), device=index))
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return None


def _workspace(index, handle, nbytes):
    """Scratch of a call on stream ``handle``: one buffer per device and
    stream that grows with need, so calls on different streams do not share
    it. A captured call gets its own from the graph's memory (two graphs never
    share one); its device error record is then not seen by ``check``, pass a
    workspace to keep it."""
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
        ws[:WORKSPACE_BYTES].zero_()
        return ws
    key = (index, handle)
    ws = _binding._paged_workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        grown = torch.empty(max(nbytes, WORKSPACE_BYTES), dtype=torch.uint8, device=torch.device("cuda", index))
        if ws is None:
            grown[:WORKSPACE_BYTES].zero_()
        else:
            grown[:WORKSPACE_BYTES].copy_(ws[:WORKSPACE_BYTES])   # keep an error that nobody has read yet
        _binding._paged_workspaces[key] = ws = grown
    return ws


def _check_workspace(ws):
    _need(ws.is_contiguous() and ws.numel() * ws.element_size() >= WORKSPACE_BYTES,
          f"workspace must be contiguous and hold at least {WORKSPACE_BYTES} bytes")


def _raise_unless_ok(st):
    if st != ATTN_OK:
        raise AttnError(st, last_error())


def cache_append(k, v, k_cache, v_cache, block_table, seqlens_k, *, k_scale=None, v_scale=None, cu_seqlens_q=None,
                 workspace=None, stream=None):
    """Writes the new tokens' keys and values into the cache, in place.

    ``k`` and ``v`` are bf16, [B, Sq, Hkv, D], or packed [T, Hkv, D] with int32
    ``cu_seqlens_q`` (rows behind the last sequence are not read).
    ``seqlens_k`` (int32 [B]) counts each sequence's tokens with the new ones:
    token i of Lq goes to position seqlens_k - Lq + i. Into an e4m3 cache each
    (token, head) vector is rounded with its own scale, the smallest power of
    two s with amax / s <= 448, which goes to ``k_scale`` / ``v_scale``. Two
    new tokens must not share a slot. A token whose position or page is out
    of range is not written and reported by ``check``. Asynchronous on
    ``stream`` (default: the current torch stream).
    """
    L = _library()
    packed = cu_seqlens_q is not None
    cache = _check_cache(k_cache, v_cache, block_table, k_scale, v_scale)
    batch, heads, dim = cache[-1], cache[-3], cache[-2]
    _need(k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16, "new keys and values must be bf16")
    _need(k.dim() == (3 if packed else 4) and k.shape == v.shape,
          "k and v must be [B, Sq, Hkv, D], or [T, Hkv, D] with cu_seqlens_q, of one shape")
    _need(tuple(k.shape[-2:]) == (heads, dim), "k and v must have the cache's heads and depth")
    _need(k.stride(-1) == 1 and v.stride(-1) == 1, "the depth of k and v must be contiguous")
    _int32("seqlens_k", seqlens_k, (batch,))
    if packed:
        _int32("cu_seqlens_q", cu_seqlens_q, (batch + 1,))
        seqlen_q, total_q = 0, k.shape[0]
        strides = (0, *_strides(k), 0, *_strides(v))
    else:
        _need(k.shape[0] == batch, "k and block_table batch sizes differ")
        seqlen_q, total_q = k.shape[1], 0
        strides = (*_strides(k), *_strides(v))
    if workspace is not None:
        _check_workspace(workspace)
    index = _check_device((("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache),
                           ("block_table", block_table), ("seqlens_k", seqlens_k), ("k_scale", k_scale),
                           ("v_scale", v_scale), ("cu_seqlens_q", cu_seqlens_q), ("workspace", workspace)))
    ctx = _elsewhere(index, stream)
    if ctx is not None:
        with ctx:
            return cache_append(k, v, k_cache, v_cache, block_table, seqlens_k, k_scale=k_scale, v_scale=v_scale,
                                cu_seqlens_q=cu_seqlens_q, workspace=workspace)
    handle = _raw_stream(index)
    ws = workspace if workspace is not None else _workspace(index, handle, WORKSPACE_BYTES)
    p = _APPEND.pack(*cache, k.data_ptr(), v.data_ptr(), seqlens_k.data_ptr(),
                     cu_seqlens_q.data_ptr() if packed else 0, ws.data_ptr(), *strides, seqlen_q, total_q)
    _raise_unless_ok(L.attn_cache_append(p, handle))


def cache_read(k_cache, v_cache, block_table, cu_seqlens_k, *, total_k=None, k_scale=None, v_scale=None, out_k=None,
               out_v=None, workspace=None, stream=None):
    """Reads sequences out of the cache; returns packed bf16 (k, v), [Tk, Hkv, D].

    Rows ``cu_seqlens_k[b]`` to ``cu_seqlens_k[b + 1]`` (int32 [B + 1]) receive
    positions 0, 1, ... of sequence b; an e4m3 cache gives code * scale,
    rounded once. ``total_k`` is the number of rows to allocate; or pass
    ``out_k`` and ``out_v``, whose rows behind the last sequence stay as they
    are. A row whose position or page is out of range is not written and
    reported by ``check``. Asynchronous on ``stream`` (default: the current
    torch stream).
    """
    L = _library()
    cache = _check_cache(k_cache, v_cache, block_table, k_scale, v_scale)
    batch, heads, dim = cache[-1], cache[-3], cache[-2]
    _int32("cu_seqlens_k", cu_seqlens_k, (batch + 1,))
    _need((out_k is None) == (out_v is None), "out_k and out_v go together")
    if out_k is None:
        _need(total_k is not None and total_k >= 0, "total_k (the rows to allocate) or out_k and out_v are needed")
    else:
        rows = out_k.shape[0] if out_k.dim() else 0
        _need(total_k is None or total_k == rows, "total_k differs from the rows of out_k")
        total_k = rows
        for name, t in (("out_k", out_k), ("out_v", out_v)):
            _need(t.dtype == torch.bfloat16 and tuple(t.shape) == (rows, heads, dim) and t.stride(2) == 1,
                  f"{name} must be a bf16 [Tk, Hkv, D] tensor with contiguous depth")
    if workspace is not None:
        _check_workspace(workspace)
    index = _check_device((("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table),
                           ("cu_seqlens_k", cu_seqlens_k), ("k_scale", k_scale), ("v_scale", v_scale),
                           ("out_k", out_k), ("out_v", out_v), ("workspace", workspace)))
    ctx = _elsewhere(index, stream)
    if ctx is not None:
        with ctx:
            return cache_read(k_cache, v_cache, block_table, cu_seqlens_k, total_k=total_k, k_scale=k_scale,
                              v_scale=v_scale, out_k=out_k, out_v=out_v, workspace=workspace)
    if out_k is None:
        out_k = torch.empty((total_k, heads, dim), dtype=torch.bfloat16, device=k_cache.device)
        out_v = torch.empty_like(out_k)
    handle = _raw_stream(index)
    ws = workspace if workspace is not None else _workspace(index, handle, WORKSPACE_BYTES)
    p = _READ.pack(*cache, out_k.data_ptr(), out_v.data_ptr(), cu_seqlens_k.data_ptr(), ws.data_ptr(),
                   *_strides(out_k), *_strides(out_v), total_k)
    _raise_unless_ok(L.attn_cache_read(p, handle))
    return out_k, out_v


def paged_forward(q, k_cache, v_cache, block_table, seqlens_k, *, causal=True, softmax_scale=None, k_scale=None,
                  v_scale=None, cu_seqlens_q=None, max_seqlen_q=None, max_seqlen_k=None, out=None, lse=None,
                  return_lse=True, workspace=None, stream=None):
    """Attention of new tokens over the paged cache; returns (O, LSE).

    ``q`` is bf16, [B, Sq, Hq, D] -> O [B, Sq, Hq, D] bf16, LSE [B, Hq, Sq]
    fp32; or packed [T, Hq, D] with int32 ``cu_seqlens_q`` and ``max_seqlen_q``
    (an upper bound of every sequence's new tokens) -> O [T, Hq, D], LSE
    [Hq, T] (rows behind the last sequence stay as they are). ``seqlens_k``
    (int32 [B]) counts each sequence's cached tokens, the new ones included
    (append them first). ``causal``: new token i of Lq sees positions up to
    seqlens_k - Lq + i; otherwise all. Rows that see nothing get O = 0 and
    LSE = -inf. ``max_seqlen_k`` bounds the cached lengths (default: what
    block_table can hold); a tighter bound only helps to plan the launch.
    D is 64 or 128; D ** -0.5 is the default ``softmax_scale``. Slots past a
    sequence's length may hold anything. Asynchronous on ``stream`` (default:
    the current torch stream).
    """
    L = _library()
    packed = cu_seqlens_q is not None
    cache = _check_cache(k_cache, v_cache, block_table, k_scale, v_scale)
    batch, heads, dim, width, page_size = cache[-1], cache[-3], cache[-2], cache[-4], cache[-5]
    _need(q.dtype == torch.bfloat16, "q must be bf16")
    _need(q.dim() == (3 if packed else 4), "q must be [B, Sq, Hq, D], or [T, Hq, D] with cu_seqlens_q")
    _need(q.shape[-1] == dim, "q and the cache have different depths")
    _need(q.stride(-1) == 1, "the depth of q must be contiguous")
    _int32("seqlens_k", seqlens_k, (batch,))
    hq = q.shape[-2]
    if packed:
        _int32("cu_seqlens_q", cu_seqlens_q, (batch + 1,))
        _need(max_seqlen_q is not None and max_seqlen_q >= 0, "packed q needs max_seqlen_q")
        total_q = q.shape[0]
        seqlen_q = min(int(max_seqlen_q), total_q)
        lse_shape = (hq, total_q)
    else:
        _need(q.shape[0] == batch, "q and block_table batch sizes differ")
        seqlen_q, total_q = q.shape[1], 0
        lse_shape = (batch, hq, seqlen_q)
    seqlen_k = width * page_size if max_seqlen_k is None else min(int(max_seqlen_k), width * page_size)
    _need(seqlen_k >= 0, "max_seqlen_k must not be negative")
    if out is not None:
        _need(out.dtype == torch.bfloat16 and out.shape == q.shape and out.stride(-1) == 1,
              "out must be a bf16 tensor of q's shape with contiguous depth")
    if lse is not None:
        _need(lse.dtype == torch.float32 and tuple(lse.shape) == lse_shape and lse.is_contiguous(),
              f"lse must be a contiguous fp32 tensor of shape {lse_shape}")
    if workspace is not None:
        _check_workspace(workspace)
    index = _check_device((("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table),
                           ("seqlens_k", seqlens_k), ("k_scale", k_scale), ("v_scale", v_scale),
                           ("cu_seqlens_q", cu_seqlens_q), ("out", out), ("lse", lse), ("workspace", workspace)))
    ctx = _elsewhere(index, stream)
    if ctx is not None:
        with ctx:
            return paged_forward(q, k_cache, v_cache, block_table, seqlens_k, causal=causal,
                                 softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale,
                                 cu_seqlens_q=cu_seqlens_q, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
                                 out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    scale = float(softmax_scale if softmax_scale is not None else dim ** -0.5)
    handle = _raw_stream(index)
    q_strides, o_strides = _strides(q), _strides(out)
    if packed:
        q_strides, o_strides = (0, *q_strides), (0, *o_strides)
    rows = (q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), seqlens_k.data_ptr(),
            cu_seqlens_q.data_ptr() if packed else 0)
    rest = (*q_strides, *o_strides, seqlen_q, seqlen_k, total_q, hq, 1 if causal else 0, scale)
    if workspace is None:
        # the size is a function of these numbers and the device alone
        sizes = (index, seqlen_q, seqlen_k, total_q, hq, causal, *cache[-7:])
        nbytes = _bytes_by_sizes.get(sizes)
        if nbytes is None:
            nbytes = int(L.attn_paged_workspace_bytes(_PAGED.pack(*cache, *rows, 0, 0, *rest)))
            if len(_bytes_by_sizes) >= 256:
                _bytes_by_sizes.clear()
            _bytes_by_sizes[sizes] = nbytes
        workspace = _workspace(index, handle, nbytes)
    p = _PAGED.pack(*cache, *rows, workspace.data_ptr(), workspace.numel() * workspace.element_size(), *rest)
    _raise_unless_ok(L.attn_paged_fwd(p, handle))
    return out, lse
