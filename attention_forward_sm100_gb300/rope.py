"""Rotary positions: the Python calls of the operator in attn_rotary.h.

``rotary`` turns queries and keys by their tokens' positions before they go to
``forward``, ``cache_append`` or ``paged_forward`` (``cache_append`` can do it
on the way). The angles come in a table that a program makes once for its model:
``rotary_table`` from the frequencies of ``rotary_frequencies``, or any other
cosines and sines.
"""
from __future__ import annotations

import math

import torch

from . import _binding
from .paged import _on, _result


def rotary_frequencies(dim, *, base=10000.0, factor=1.0, original_length=None, slow_turns=1.0, fast_turns=32.0,
                       ramp="log"):
    """Angle per position of each of the ``dim // 2`` pairs, float64 [dim // 2].

    Pair i turns by base ** (-2 i / dim). For contexts ``factor`` times as long
    as a model was trained for: without ``original_length`` all frequencies are
    divided by ``factor`` (interpolated positions). With it, pairs that make
    ``fast_turns`` turns or more over the original length stay as they are, those
    that make ``slow_turns`` or fewer are divided, and between them the two are
    mixed, in a way that a model was trained with and that ``ramp`` names:

    - ``"log"``: in proportion to the logarithm of the turns;
    - ``"turns"``: in proportion to the turns;
    - ``"pairs"``: in proportion to i, between whole numbers: the last i with
      ``fast_turns`` or more (0 at least) and the first with ``slow_turns`` or fewer
      (dim - 1 at most), turns taken as a function of any real i.

    With dim 128, base 10000, factor 32 and an original length of 4096, ``"log"``
    and ``"pairs"`` are up to 2.1 times apart. (Scaling by a larger
    ``base`` needs nothing else.)
    """
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and at least 2")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if ramp not in ("log", "turns", "pairs"):
        raise ValueError("ramp must be 'log', 'turns' or 'pairs'")
    own = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if original_length is None:
        if ramp != "log":
            raise ValueError("ramp goes with original_length")
        return own / factor
    if not (original_length > 0 and 0 < slow_turns < fast_turns):
        raise ValueError("original_length must be positive, and 0 < slow_turns < fast_turns")
    turns = original_length * own / (2 * math.pi)
    if ramp == "log":
        keep = ((turns / slow_turns).log() / math.log(fast_turns / slow_turns)).clamp(0, 1)
    elif ramp == "turns":
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
    else:
        if base <= 1:
            raise ValueError("a ramp over pairs needs a base above 1: their turns must fall")
        fast, slow = (dim * math.log(original_length / (2 * math.pi * n)) / (2 * math.log(base))
                      for n in (fast_turns, slow_turns))   # i where a pair makes n turns
        fast, slow = max(math.floor(fast), 0), min(math.ceil(slow), dim - 1)
        i = torch.arange(dim // 2, dtype=torch.float64)
        keep = ((slow - i) / (slow - fast)).clamp(0, 1) if slow > fast else (i <= fast).double()
    return own * keep + own / factor * (1 - keep)


def rotary_table(frequencies, length, *, amplitude=1.0, first=0, device="cuda"):
    """fp32 [length, 2 * len(frequencies)]: cosines, then sines, of positions
    ``first``, ``first`` + 1, ... times ``amplitude``. Angles are computed in
    float64 (in fp32 they would lose 2^-24 of themselves: a whole 0.01 at position
    131072), each value is rounded once."""
    frequencies = torch.as_tensor(frequencies, dtype=torch.float64).to(device)
    if frequencies.dim() != 1 or length < 0:
        raise ValueError("frequencies must be one-dimensional and length not negative")
    angle = torch.arange(first, first + length, dtype=torch.float64, device=device)[:, None] * frequencies
    return (torch.cat([angle.cos(), angle.sin()], 1) * amplitude).float()


def rotary(q, k, table, *, positions=None, seqlens=None, cu_seqlens=None, interleaved=False, inverse=False, out_q=None,
           out_k=None, workspace=None, stream=None):
    """Turns the first R depths of every head by its token's position; returns (q, k).

    ``q`` and ``k`` are bf16, [B, S, H, D], or packed [T, H, D] with int32
    ``cu_seqlens`` ([T, H, D] without it: one sequence); ``k`` may be None. Depths
    (i, i + R / 2), with ``interleaved`` (2 i, 2 i + 1), form pair i < R / 2 and
    become (x1 c - x2 s, x2 c + x1 s) with c = table[p, i], s = table[p, R / 2 + i]
    (``table`` fp32 [positions, R], R <= D), computed in fp32 and rounded once.
    The other depths are copied. ``inverse`` turns back (s negated), which is also
    the gradient of the rotation.

    p is ``positions`` (int32, [B, S] or [T]); or, with ``seqlens`` (int32 [B]:
    each sequence's tokens, these included), seqlens[b] - S + i for token i; or i.
    A row at a position outside the table is not written and reported by
    ``check``; rows in front of the first packed sequence and behind the last one
    stay as they are.

    ``out_q`` and ``out_k`` may be ``q`` and ``k`` themselves, or parts of their memory with the
    same strides that no row of the call uses; any other overlap is refused. Strides are multiples
    of 16 bytes and D a multiple of 8. Tables whose R is a multiple of 16 (8 with
    ``interleaved``) are read 16 bytes at a time, others value by value.
    Asynchronous on ``stream`` (default: the current torch stream).
    """
    native = _binding.paged_native()
    if stream is not None:
        with _on(stream, q):
            return rotary(q, k, table, positions=positions, seqlens=seqlens, cu_seqlens=cu_seqlens,
                          interleaved=interleaved, inverse=inverse, out_q=out_q, out_k=out_k, workspace=workspace)
    return _result(native.rotary(q, k, table, positions, seqlens, cu_seqlens, interleaved, inverse, out_q, out_k,
                                 workspace))
