"""Calls of the paged-cache operators at the edges of what they accept."""
import math

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


# ---------------------------------------------------------------- tiny value scales
TINY = {
    "smallest": lambda n: torch.full((n,), 2.0 ** -126),
    "2^-121": lambda n: torch.full((n,), 2.0 ** -121),
    "2^-120": lambda n: torch.full((n,), 2.0 ** -120),
    "mixed": lambda n: torch.exp2(-126.0 + torch.arange(n) % 30),
    "then_ordinary": lambda n: torch.where(torch.arange(n) < 3 * n // 4, 2.0 ** -126, 2.0 ** -8),
    "after_ordinary": lambda n: torch.where(torch.arange(n) < n // 4, 2.0 ** -8, 2.0 ** -124),
}


@pytest.mark.parametrize("lens_k", [[1, 17], [1500, 700]], ids=["short", "long"])
@pytest.mark.parametrize("dim,hq,new", [(128, 4, 1), (64, 4, 1), (128, 4, 3), (64, 4, 3), (128, 20, 1), (64, 20, 1)])
@pytest.mark.parametrize("name", list(TINY))
def test_tiny_value_scales(pkg, name, dim, hq, new, lens_k):
    """Rows of up to 32 share the cached values: O within the roundings of the
    weights and of O, and half a step of bf16's subnormals (2^-134)."""
    p = R.make(lens_k, [new] * 2, hq, 1, dim, 16, fp8=True, seed=41)
    for b, n in enumerate(lens_k):
        s = TINY[name](n)
        at = torch.arange(n)
        p.v_scale[p.table[b].cpu()[at // 16].long(), 0, at % 16] = s.float().cuda()
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 2.0 ** -134
        assert ((o[b].double() - ro).abs() <= bound).all()
        seen = torch.isfinite(rl)
        assert torch.equal(torch.isfinite(lse[b]), seen)
        assert ((lse[b].double() - rl)[seen].abs() <= 5e-5).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_zero_vectors_with_the_smallest_scale(pkg, dim):
    """A quantiser that clamps its scales at the smallest normal float writes
    2^-126 for a vector of zeros: O = 0, whatever the length."""
    p = R.make([1, 40, 1000], [1] * 3, 4, 1, dim, 16, fp8=True, seed=42)
    held = ~torch.isnan(p.v_scale)
    p.v_scale[held] = 2.0 ** -126
    p.v_cache.view(torch.uint8)[held.transpose(1, 2)] = 0
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    assert bool((o == 0).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("size", [-118, -122, -126, -131])
def test_attend_to_what_append_wrote_for_tiny_values(pkg, size):
    p = R.make([5, 300], [5, 5], 4, 2, 128, 16, fp8=True, seed=43)
    p.v_new.copy_((p.v_new.double() * 2.0 ** size).to(torch.bfloat16))
    table, lens = p.table, p.seqlens
    pkg.cache_append(p.k_new, p.v_new, *p.cache, **p.scales)
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 2.0 ** -134
        assert ((o[b].double() - ro).abs() <= bound).all()


# ---------------------------------------------------------------- offsets
def _reported(pkg):
    with pytest.raises(pkg.AttnError, match="paged cache"):
        pkg.check()
    pkg.check()


WRONG = {
    # offsets, rows there are, sequences that are right all the same
    "decreasing_inside": ([0, 10, 5, 20], 20, []),
    "decreasing_at_the_end": ([0, 10, 15, 5], 20, []),
    "last_wholly_past_the_rows": ([0, 3, 5, 11], 5, [0, 1]),
    "last_two_past_the_rows": ([0, 5, 9, 11], 5, [0]),
    "below_zero": ([-5, 0, 4, 10], 10, [1, 2]),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(WRONG))
def test_append_reports_wrong_offsets(pkg, name, fp8):
    """Out of order: nothing is written. Past the rows or below zero: the
    sequences concerned are not written, the others are."""
    cu, rows, right = WRONG[name]
    lens = [max(0, cu[b + 1] - cu[b]) if b in right else 0 for b in range(3)]
    p = R.make([40, 30, 50], lens, 2, 2, 64, 16, fp8=fp8, packed=True, seed=44)
    g = torch.Generator(device="cuda").manual_seed(45)
    k, v = (torch.randn(rows, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    p.k_new, p.v_new = (torch.cat([x[cu[b]:cu[b + 1]] for b in right] + [x[:0]]) for x in (k, v))
    want = R.append(p)
    pkg.cache_append(k, v, *p.cache, cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), **p.scales)
    _reported(pkg)
    for got, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
        assert got is None or torch.equal(R.bits(got), R.bits(w))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["decreasing_inside", "decreasing_at_the_end", "below_zero"])
def test_read_reports_wrong_offsets(pkg, name, fp8):
    cu, rows, right = WRONG[name]
    p = R.make([40, 30, 50], [0] * 3, 2, 2, 64, 16, fp8=fp8, packed=True, seed=46)
    out = [torch.full((rows, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [x.clone() for x in out]
    for b in right:
        for w, x in zip(want, R.gather(p, b)):
            w[cu[b]:cu[b + 1]] = x[:cu[b + 1] - cu[b]].to(torch.bfloat16)
    pkg.cache_read(p.k_cache, p.v_cache, p.table, torch.tensor(cu, dtype=torch.int32, device="cuda"), out_k=out[0],
                   out_v=out[1], **p.scales)
    _reported(pkg)
    assert torch.equal(R.bits(out[0]), R.bits(want[0])) and torch.equal(R.bits(out[1]), R.bits(want[1]))


def test_wrong_offsets_among_many_sequences(pkg):
    """Found wherever they are, and by calls whose rows all lie in front of them."""
    n = 300
    p = R.make([20] * n, [1] * n, 1, 1, 64, 16, packed=True, seed=47)
    before = p.k_cache.clone()
    cu = p.cu_q.clone()
    cu[277] = 3
    pkg.cache_append(p.k_new, p.v_new, *p.cache, cu_seqlens_q=cu)
    with pytest.raises(pkg.AttnError, match="sequence 276"):
        pkg.check()
    pkg.cache_append(p.k_new[:7], p.v_new[:7], *p.cache, cu_seqlens_q=cu)
    _reported(pkg)
    assert torch.equal(R.bits(p.k_cache), R.bits(before))
    out = torch.full((n, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, out_k=out, out_v=out.clone())
    _reported(pkg)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_rows_in_front_of_the_first_sequence(pkg, fp8):
    """Offsets that start late (a part of a larger batch): the rows in front of
    them belong to nobody, as those behind the last sequence."""
    p = R.make([70, 9, 200], [70, 1, 30], 4, 2, 64, 16, fp8=fp8, packed=True, seed=48)
    want = R.append(p)
    pad = torch.full((13, 2, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    cu = p.cu_q + 13
    pkg.cache_append(torch.cat([pad, p.k_new]), torch.cat([pad, p.v_new]), *p.cache, cu_seqlens_q=cu, **p.scales)
    pkg.check()
    for got, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
        assert got is None or torch.equal(R.bits(got), R.bits(w))
    lens = p.lens_k
    cu_k = torch.tensor([13 + sum(lens[:b]) for b in range(4)], dtype=torch.int32, device="cuda")
    out = [torch.full((13 + sum(lens) + 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkg.cache_read(p.k_cache, p.v_cache, p.table, cu_k, out_k=out[0], out_v=out[1], **p.scales)
    pkg.check()
    both = [torch.cat(x).to(torch.bfloat16) for x in zip(*(R.gather(p, b) for b in range(3)))]
    for got, w in zip(out, both):
        assert torch.equal(got[13:-2], w) and bool((got[:13] == 7.0).all()) and bool((got[-2:] == 7.0).all())
    q = torch.cat([torch.full((13, 4, 64), math.nan, dtype=torch.bfloat16, device="cuda"), p.q])
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, q.shape[0]), 7.0, device="cuda")
    for most in (70, 200):
        pkg.paged_forward(q, *p.cache, cu_seqlens_q=cu, max_seqlen_q=most, out=o, lse=lse, **p.scales)
        pkg.check()
        R.check_attend(p, o[13:], lse[:, 13:], True)
        assert bool((o[:13] == 7.0).all()) and bool((lse[:, :13] == 7.0).all())


def test_a_bound_of_no_new_tokens(pkg):
    """max_seqlen_q = 0 where sequences have new tokens is a wrong bound like any other."""
    p = R.make([40, 30], [2, 3], 4, 2, 64, 16, packed=True, seed=49)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=p.cu_q, max_seqlen_q=0, out=out)
    _reported(pkg)
    out.fill_(7.0)
    pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=torch.zeros_like(p.cu_q), max_seqlen_q=0, out=out)
    pkg.check()
    assert bool((out == 7.0).all())


# ---------------------------------------------------------------- NaN
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dim,new,lens_k", [(64, 3, [900, 300]), (128, 3, [900, 300]), (64, 130, [900, 300]),
                                            (128, 130, [900, 300]), (128, 160, [9000, 300]), (64, 600, [2500, 600])])
def test_nan_stays_in_its_rows(pkg, dim, new, lens_k, fp8):
    """A NaN in q makes its (token, head) NaN, O and LSE; a NaN among the keys that
    every row sees makes its KV head's rows NaN. All others are as ever."""
    hq, hkv = 4, 2
    p = R.make(lens_k, [new] * 2, hq, hkv, dim, 16, fp8=fp8, seed=50)
    p.q[0, 1, 2, 5] = math.nan
    p.q[1, new - 1, 0, 0] = math.nan
    p.k_cache[p.table[1, 0].long(), 3, 1, 7] = math.nan     # KV head 1: query heads 2 and 3
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    bad = torch.zeros(2, hq, new, dtype=torch.bool, device="cuda")
    bad[0, 2, 1] = bad[1, 0, new - 1] = True
    bad[1, 2:] = (torch.arange(new, device="cuda") + lens_k[1] - new >= 3)
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(o).any(-1).transpose(1, 2), bad) and torch.equal(torch.isnan(o).all(-1).transpose(1, 2), bad)
    p.q = p.q.nan_to_num(0.0)
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        ok = ~bad[b]
        off = (o[b].double() - ro).abs() / (2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 1e-6)
        assert (off.transpose(0, 1)[ok] <= 1.0).all()
        assert ((lse[b].double() - rl)[ok & torch.isfinite(rl)].abs() <= 5e-5).all()


# ---------------------------------------------------------------- scratch memory
def _long_chunk():
    """e4m3, 600 rows to a KV head, a table of 131072 tokens: a copy of 512 MiB."""
    p = R.make([3000, 900], [300] * 2, 8, 4, 128, 64, fp8=True, seed=54)
    table = torch.full((2, 131072 // 64), -1, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = p.table
    return p, table


def test_a_long_chunk_keeps_no_large_scratch(pkg):
    """Its memory goes back to the allocator with the call; results, and the
    calls after it, are as ever."""
    p, table = _long_chunk()
    small = R.make([700, 90], [1] * 2, 8, 2, 64, 16, seed=55)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = pkg.paged_forward(small.q, *small.cache)
        held = torch.cuda.memory_allocated()
        o, lse = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, **p.scales)
        grown = torch.cuda.memory_allocated() - held - o.nbytes - lse.nbytes
        assert torch.cuda.max_memory_allocated() - held > 512 << 20      # (the copy was made)
        got = pkg.paged_forward(small.q, *small.cache)
        o2, lse2 = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, **p.scales)
        pkg.check()
    R.check_attend(p, o, lse, True)
    assert torch.equal(R.bits(o), R.bits(o2)) and torch.equal(R.bits(lse), R.bits(lse2))
    for x, y in zip(want, got):
        assert torch.equal(R.bits(x), R.bits(y))
    assert grown <= 128 << 20


def test_what_a_long_chunk_finds_wrong_is_reported(pkg):
    """Its own errors, and one that nobody has read when it starts."""
    p, table = _long_chunk()
    bad = table.clone()
    bad[1, 2] = -3
    pkg.paged_forward(p.q, p.k_cache, p.v_cache, bad, p.seqlens, **p.scales)
    with pytest.raises(pkg.AttnError, match="sequence 1"):
        pkg.check()
    pkg.check()
    small = R.make([700, 90], [1] * 2, 8, 2, 64, 16, seed=55)
    small.table[0, 0] = -1
    pkg.paged_forward(small.q, *small.cache)
    o, lse = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, **p.scales)
    with pytest.raises(pkg.AttnError, match="sequence 0"):
        pkg.check()
    pkg.check()
    R.check_attend(p, o, lse, True)


# ---------------------------------------------------------------- scales that are no powers of two, in chunks
def _score_error(p, b, scale, split):
    """Bound of a score's error: fp32 products and sums in steps of 16 depths (a
    tensor core may truncate, 2^-23 a step), the exponent's two roundings, and
    where q is split in two e4m3 parts 2^-17 of a row's largest value on the
    values below 2^-9 of it."""
    k, _ = R.gather(p, b)
    q = R.rows_of(p, p.q, b).double()
    group = q.shape[1] // k.shape[1]
    worst = 0.0
    for h in range(q.shape[1]):
        kh = k[:, h // group].abs()
        size = (q[:, h].abs() @ kh.t()).max().item() * scale
        ds = (q.shape[2] / 16 + 6) * 2.0 ** -23 * size
        if split:
            top = q[:, h].abs().amax(-1, keepdim=True)
            lost = torch.where(q[:, h].abs() < 2.0 ** -9 * top, 2.0 ** -17 * top, 0.0)
            ds += (lost @ kh.t()).max().item() * scale
        worst = max(worst, ds)
    return worst


@pytest.mark.parametrize("wide_table", [False, True], ids=["tight", "wide"])
@pytest.mark.parametrize("dim,new", [(128, 100), (128, 140), (64, 100), (64, 140)])
def test_chunks_over_scales_of_any_value(pkg, dim, new, wide_table):
    """Scales as amax / 448 gives them. code * scale of V is rounded to bf16
    (2^-8 of every value), that of K with D = 64, and with D = 128 where 512 rows
    or more (four query heads: 128 new tokens) read a bf16 copy, which a bound on
    the lengths that asks for more than 1 GiB turns off; a score then moves by
    at most 2^-8 * scale * sum |q k|."""
    p = R.make([new, 700], [new] * 2, 8, 2, dim, 16, fp8=True, seed=52)
    g = torch.Generator().manual_seed(53)
    for s, factor in ((p.k_scale, 2.0 ** -7), (p.v_scale, 2.0 ** -6)):
        held = ~torch.isnan(s)
        s[held] = ((torch.rand(int(held.sum()), generator=g) + 0.5) * factor).cuda()
    table = p.table
    if wide_table:
        table = torch.full((2, (1 << 21) // 16), -1, dtype=torch.int32, device="cuda")
        table[:, :p.table.shape[1]] = p.table
    o, lse = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, **p.scales)
    pkg.check()
    rounds_k = dim == 64 or (new * 4 >= 512 and not wide_table)
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        ds = 0.0
        if rounds_k:
            k, _ = R.gather(p, b)
            ds = max(2.0 ** -8 * dim ** -0.5 * (p.q[b, :, h].double().abs() @ k[:, h // 4].abs().t()).max().item()
                     for h in range(8))
        else:
            ds = _score_error(p, b, dim ** -0.5, True)
        grow = math.expm1(2 * ds)
        bound = 2.0 ** -8 * ro.abs() + (2 * 2.0 ** -8 + 2.0 ** -14 + grow) * ra * (1 + grow) + 1e-6
        assert ((o[b].double() - ro).abs() <= bound).all()
        assert (lse[b].double() - rl).abs().max().item() <= 5e-5 + ds


# ---------------------------------------------------------------- large scores
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dim,new,lens_k", [(64, 3, [700, 90]), (128, 3, [700, 90]), (64, 10, [1700, 90]),
                                            (64, 130, [700, 130]), (128, 130, [700, 130]), (128, 200, [9000, 200]),
                                            (64, 600, [2500, 600]), (128, 600, [2500, 600])])
def test_values_under_large_scores(pkg, dim, new, lens_k, fp8):
    """Scores in the thousands, in random order: every move of the running
    maximum has to rescale what is summed so far, by a power of two with hundreds
    for its exponent. O and LSE within the bound that the score's error (2 ds in
    the exponent; ds is 0.02, or 0.3 where q is split) and the roundings imply."""
    p = R.make(lens_k, [new] * 2, 4, 2, dim, 16, fp8=fp8, seed=51)
    p.q *= 200
    o, lse = pkg.paged_forward(p.q, *p.cache, softmax_scale=1.0, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True, 1.0)):
        ds = _score_error(p, b, 1.0, fp8 and dim == 128)
        grow = math.expm1(2 * ds)
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14 + grow) * ra * (1 + grow) + 1e-6
        assert ((o[b].double() - ro).abs() <= bound).all()
        assert ((lse[b].double() - rl).abs() <= ds + 2.0 ** -20 + 2.0 ** -23 * rl.abs()).all()


# ---------------------------------------------------------------- many sequences, a wide table
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_many_short_sequences_under_a_wide_table(pkg, fp8):
    """1100 sequences of 32 KV heads in a table of 2^22 tokens each: more key tiles
    than 32 bits count, were they full. All share one page."""
    batch, heads, dim, page, longest = 1100, 32, 64, 65536, 300
    g = torch.Generator(device="cuda").manual_seed(61)
    cache = [torch.full((1, page, heads, dim), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x in cache:
        x[0, :longest] = torch.randn(longest, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    scales = {}
    if fp8:
        cache = [x.to(R.E4M3) for x in cache]
        scales = {n: torch.ones(1, heads, page, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.zeros(batch, 64, dtype=torch.int32, device="cuda")
    lens = 1 + torch.arange(batch, dtype=torch.int32, device="cuda") * 7919 % longest
    q = torch.randn(batch, 1, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    o, lse = pkg.paged_forward(q, *cache, table, lens, **scales)
    pkg.check()
    k, v = (x[0, :longest].double() for x in cache)
    s = torch.einsum("bhd,khd->bhk", q[:, 0].double(), k) * dim ** -0.5
    s = torch.where(torch.arange(longest, device="cuda") < lens[:, None, None], s, -math.inf)
    w = torch.softmax(s, -1)
    ro, ra = torch.einsum("bhk,khd->bhd", w, v), torch.einsum("bhk,khd->bhd", w, v.abs())
    assert ((o[:, 0].double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 1e-6).all()
    assert ((lse[:, :, 0].double() - torch.logsumexp(s, -1)).abs() <= 5e-5).all()
