"""Frequencies of scaled positions, and rows that a rotation writes and where they may
lie, without a GPU. (Calls that would be taken have no workspace, which is looked at
last.)"""
import math
import random

import pytest
import torch

import test_paged4_cpu as C4
import test_paged_cpu as C
import test_rotary_cpu as T
from test_rotary_cpu import pkg  # noqa: F401


def _verdict(L, status):
    assert status == 1
    text = L.attn_fwd_last_error().decode()
    return None if "workspace" in text else text


def _rows(at, n, stride, dim):
    """Addresses, in units of 16 bytes, of rows of dim bf16 each."""
    return {(at + 2 * (i * stride[0] + j * stride[1] + h * stride[2])) // 16 + c
            for i in range(n[0]) for j in range(n[1]) for h in range(n[2]) for c in range(dim // 8)}


def test_rows_that_share_memory_are_refused(pkg):  # noqa: F811
    """Against the sets of addresses: random views of one buffer, in place, between the
    input's rows, and across them."""
    L = T._library(pkg)
    g = random.Random(3)
    seen = dict(same=0, apart=0, meet=0, other=0)
    for _ in range(3000):
        dim = g.choice((8, 16, 64))
        n = (g.choice((1, 2, 3)), g.choice((1, 2, 5)), g.choice((1, 2, 3)))

        def strides():
            head = dim * g.choice((1, 2, 3))
            token = head * n[2] * g.choice((1, 1, 2))
            out = [token * n[1] * g.choice((1, 2)), token, head]
            return tuple([out[1], out[0], out[2]] if g.random() < 0.1 and n[0] == 1 else out)

        sq = strides()
        so = sq if g.random() < 0.7 else strides()
        base, at = 1 << 20, (1 << 20) + 16 * g.choice((0, 0, 1, dim // 8, g.randrange(-400, 400)))
        got = _verdict(L, L.attn_rotary(T._params(
            q=base, q_out=at, k=0, k_out=0, ws=0, q_stride=sq, q_out_stride=so, k_stride=(0, 0, 0), k_out_stride=(0, 0, 0),
            batch=n[0], seqlen=n[1], heads_q=n[2], heads_k=0, dim=dim, rot=8), None))
        a, b = _rows(base, n, sq, dim), _rows(at, n, so, dim)
        alike = all(x == y for x, y, m in zip(sq, so, n) if m > 1)
        if at == base and alike:
            kind = "same"
            assert got is None
        elif not a & b and (alike or min(a) > max(b) or min(b) > max(a)):
            kind = "apart"
            assert got is None, (n, sq, so, at - base, dim)
        elif a & b:
            kind = "meet"
            assert got is not None and "q_out shares memory" in got, (n, sq, so, at - base, dim)
        else:
            kind = "other"   # rows of other strides among q's
            assert got is not None and "q_out shares memory" in got
        seen[kind] += 1
    assert min(seen.values()) > 30, seen


FUSED = dict(q_stride=(1 << 12, 512, 64), k_stride=(1 << 12, 512, 64), q_out_stride=(1 << 12, 512, 64),
             k_out_stride=(1 << 12, 512, 64), q=1 << 20, q_out=1 << 20, k=(1 << 20) + 256, k_out=(1 << 20) + 256, ws=0)


@pytest.mark.parametrize("change,bad", [
    ({}, None), (dict(q_out=1 << 22, k_out=1 << 23), None), (dict(k_out=1 << 20), "q_out"), (dict(q_out=(1 << 20) + 512), None),
    (dict(q_out=(1 << 20) + 256), "q_out"), (dict(q_out=(1 << 20) + 384), "q_out"), (dict(k_out=(1 << 20) + 512), None),
    (dict(q_out=1 << 22, k_out=(1 << 20) + 128), "k_out"), (dict(q_out=1 << 22, k_out=1 << 22), "q_out"),
    (dict(q_out=1 << 22, q_out_stride=(1 << 12, 512, 0)), "q_out has rows in one place"),
    (dict(q_out=1 << 22, q_out_stride=(0, 512, 64)), "q_out has rows in one place"),
    (dict(k_out=1 << 22, k_out_stride=(1 << 12, 0, 64)), "k_out has rows in one place"),
    (dict(q_out=1 << 22, q_out_stride=(0, 512, 64), batch=1), None)], ids=str)
def test_queries_and_keys_of_one_projection(pkg, change, bad):  # noqa: F811
    L = T._library(pkg)
    got = _verdict(L, L.attn_rotary(T._params(**{**FUSED, **change}), None))
    assert (got is None) == (bad is None) and (bad is None or bad in got)


@pytest.mark.parametrize("change,bad", [
    ({}, None), (dict(q_out=14 << 20), None), (dict(q_out=(14 << 20) + 128), "q_out"),
    (dict(q_out=14 << 20, out_stride=(1024, 256, 64)), "q_out"), (dict(q_out=4 << 20), "q_out"), (dict(q_out=5 << 20), "q_out"),
    (dict(out_stride=(0, 256, 64)), "q_out has rows in one place"), (dict(q_out=0, heads=0), None)], ids=str)
def test_queries_of_an_append(pkg, change, bad):  # noqa: F811
    """Two sequences, one new token, two heads of keys and four of queries, 64 deep."""
    L = C4._library(pkg)
    for cache, blocks in (({}, None), (C4.FP4, C4.GOOD)):
        p = C.APPEND.pack(*C._cache(**cache), 4 << 20, 5 << 20, 6 << 20, 0, 0, *(256, 128, 64) * 2, 1, 0)
        got = _verdict(L, L.attn_cache_append_blocks(p, blocks, C4._turn(**change), None))
        assert (got is None) == (bad is None) and (bad is None or bad in got)


@pytest.mark.parametrize("dim,base,length,slow,fast", [
    (128, 10000.0, 4096, 1.0, 32.0), (64, 1e6, 64, 0.5, 4.0), (64, 10000.0, 100, 1.0, 32.0), (128, 500000.0, 8192, 1.0, 4.0),
    (8, 10.0, 12, 1.0, 1.25), (16, 1e4, 1 << 40, 1.0, 32.0), (32, 1e4, 3, 1.0, 32.0)])
def test_ramps_between_kept_and_divided_frequencies(pkg, dim, base, length, slow, fast):  # noqa: F811
    """Pair by pair with Python's own arithmetic; the bounds over pairs by counting."""
    factor = 32.0

    def turns(i):
        return length * base ** (-2 * i / dim) / (2 * math.pi)

    lo = max((i for i in range(-4 * dim, 4 * dim) if turns(i) >= fast), default=0)
    hi = min((i for i in range(-4 * dim, 4 * dim) if turns(i) <= slow), default=dim - 1)
    lo, hi = max(lo, 0), min(hi, dim - 1)
    for ramp in ("log", "turns", "pairs"):
        got = pkg.rotary_frequencies(dim, base=base, factor=factor, original_length=length, slow_turns=slow, fast_turns=fast,
                                     ramp=ramp)
        assert got.dtype == torch.float64 and got.shape == (dim // 2,)
        for i in range(dim // 2):
            w, t = base ** (-2 * i / dim), turns(i)
            keep = {"log": math.log(t / slow) / math.log(fast / slow), "turns": (t - slow) / (fast - slow),
                    "pairs": (hi - i) / (hi - lo) if hi > lo else float(i <= lo)}[ramp]
            keep = min(max(keep, 0.0), 1.0)
            # both terms are doubles of a few roundings each; of the shares, the logarithms' quotient most
            assert abs(got[i].item() - (w * keep + w / factor * (1 - keep))) <= 2.0 ** -44 * w
    same = pkg.rotary_frequencies(dim, base=base, factor=factor, original_length=length, slow_turns=slow, fast_turns=fast)
    assert torch.equal(same, pkg.rotary_frequencies(dim, base=base, factor=factor, original_length=length, slow_turns=slow,
                                                    fast_turns=fast, ramp="log"))


def test_ramps_differ_as_documented(pkg):  # noqa: F811
    f = [pkg.rotary_frequencies(128, factor=32.0, original_length=4096, ramp=r) for r in ("log", "pairs", "turns")]
    assert 2.1 < (f[1] / f[0]).max().item() < 2.15
    assert all(bool((x[:20] == f[0][:20]).all()) and bool((x[48:] * 32 / f[0][48:] / 32 - 1).abs().max() < 1e-12) for x in f)
    for bad in (dict(ramp="linear"), dict(ramp="pairs"), dict(ramp="turns"),
                dict(ramp="pairs", original_length=64, base=1.0), dict(ramp="pairs", original_length=64, base=0.5)):
        with pytest.raises(ValueError):
            pkg.rotary_frequencies(8, **bad)
