"""The paged-cache operators on the GPU against their definitions in 64 bits:
writing (bit for bit), reading back (bit for bit), attention (every element
within the bound its roundings imply), what only the device can refuse, and
runs of them together. Slots that no sequence holds are NaN throughout, and
table columns past a sequence's pages hold numbers outside the cache."""
import math
import types

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


# ---------------------------------------------------------------- append
APPEND = {
    # lens_k, lens_q, Hkv, D, page, packed, head-major
    "one_token": ([1], [1], 1, 64, 16, False, False),
    "step": ([5, 16, 17, 300], [1] * 4, 8, 128, 16, False, False),
    "chunk_crosses_pages": ([40, 100], [37, 37], 2, 128, 16, False, True),
    "packed_ragged": ([70, 9, 200, 33], [70, 1, 0, 30], 3, 64, 32, True, False),
    "packed_first_empty": ([8, 0, 130, 4], [0, 0, 129, 0], 5, 128, 64, True, True),
    "many_sequences": ([3 + b % 40 for b in range(300)], [1 + b % 3 for b in range(300)], 1, 64, 16, True, False),
    "long": ([5000, 4097], [4090, 4090], 4, 128, 128, False, False),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(APPEND))
def test_append_writes_exactly_its_slots(pkg, name, fp8):
    lens_k, lens_q, hkv, dim, page, packed, head_major = APPEND[name]
    p = R.make(lens_k, lens_q, hkv, hkv, dim, page, fp8=fp8, packed=packed, head_major=head_major, seed=3)
    want = R.append(p)
    pkg.cache_append(p.k_new, p.v_new, *p.cache, cu_seqlens_q=p.cu_q, **p.scales)
    pkg.check()
    got = (p.k_cache, p.v_cache, p.k_scale, p.v_scale)
    for g, w in zip(got, want):
        assert (g is None) == (w is None)
        if g is not None:
            assert torch.equal(R.bits(g), R.bits(w))


def test_append_e4m3_of_special_values(pkg):
    """Zeros, subnormals, the largest finite values, ties, infinities and NaN."""
    p = R.make([24], [24], 2, 2, 64, 16, fp8=True, seed=5)
    x = p.k_new
    x[0, 0] = 0.0
    x[0, 1] = 2.0 ** -133                      # the smallest bf16
    x[0, 2, 0] = 2.0 ** -126
    x[0, 3] = torch.finfo(torch.bfloat16).max
    x[0, 4, 0, 3] = math.inf
    x[0, 5, 1, 7] = -math.inf
    x[0, 6, 0, 9] = math.nan
    x[0, 7] = math.inf
    x[0, 8] = math.nan
    x[0, 9] = 448.0
    x[0, 10] = 450.0                           # just past 448: the next scale
    x[0, 11] = torch.linspace(-447, 447, 64).to(torch.bfloat16)
    x[0, 12] = (torch.arange(64) * 0.0625 + 16).to(torch.bfloat16)   # ties of the 3-bit mantissa
    x[0, 13, :, 0] = 3.0e38
    want = R.append(p)
    pkg.cache_append(p.k_new, p.v_new, *p.cache, **p.scales)
    pkg.check()
    for g, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
        if g.dtype == R.E4M3:   # NaN has two codes
            g, w = g.float(), w.float()
            assert torch.equal(torch.isnan(g), torch.isnan(w))
            g, w = g.nan_to_num(-1.0), w.nan_to_num(-1.0)
        assert torch.equal(R.bits(g), R.bits(w))


def test_append_leaves_rows_behind_the_last_sequence(pkg):
    p = R.make([20, 30], [5, 7], 2, 2, 64, 16, packed=True, seed=6)
    want = R.append(p)
    tail = torch.full((9, 2, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    pkg.cache_append(torch.cat([p.k_new, tail]), torch.cat([p.v_new, tail]), *p.cache, cu_seqlens_q=p.cu_q)
    pkg.check()
    assert torch.equal(R.bits(p.k_cache), R.bits(want[0])) and torch.equal(R.bits(p.v_cache), R.bits(want[1]))


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens_k,hkv,dim,page,head_major", [
    ([1], 1, 64, 16, False), ([33, 0, 64, 1, 250], 3, 128, 32, True), ([3000, 2049], 8, 128, 64, False),
    ([1 + b % 7 for b in range(200)], 2, 64, 16, False)])
def test_read_gives_the_cached_values(pkg, lens_k, hkv, dim, page, head_major, fp8):
    p = R.make(lens_k, [0] * len(lens_k), hkv, hkv, dim, page, fp8=fp8, packed=True, head_major=head_major, seed=7)
    total = sum(lens_k)
    cu = torch.tensor([sum(lens_k[:b]) for b in range(len(lens_k) + 1)], dtype=torch.int32, device="cuda")
    k, v = pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, total_k=total, **p.scales)
    # strided outputs with rows behind the last sequence
    both = torch.full((total + 5, 2, hkv, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, out_k=both[:, 0], out_v=both[:, 1], **p.scales)
    pkg.check()
    want = [torch.cat(x).to(torch.bfloat16) for x in zip(*(R.gather(p, b) for b in range(len(lens_k))))]
    assert torch.equal(R.bits(k), R.bits(want[0])) and torch.equal(R.bits(v), R.bits(want[1]))
    assert torch.equal(R.bits(both[:total, 0]), R.bits(want[0])) and torch.equal(R.bits(both[:total, 1]), R.bits(want[1]))
    assert bool((both[total:] == 7.0).all())


# ---------------------------------------------------------------- attend
ATTEND = {
    # lens_k, lens_q, Hq, Hkv, D, page, packed, head-major
    "one_key": ([1], [1], 1, 1, 64, 16, False, False),
    "short": ([7, 16, 17, 63], [1] * 4, 8, 2, 128, 16, False, False),
    "two_tiles": ([64, 65, 128, 129], [1] * 4, 4, 4, 64, 32, False, True),
    "decode": ([1000, 3, 2049, 777], [1] * 4, 32, 8, 128, 64, False, False),
    "decode_mha": ([515, 2000], [1, 1], 16, 16, 64, 16, False, False),
    "decode_mqa": ([4000], [1], 16, 1, 128, 128, False, False),
    "decode_group_5": ([333, 1200], [1, 1], 15, 3, 128, 32, False, True),
    "decode_group_20": ([900, 40], [1, 1], 20, 1, 64, 16, False, False),
    "decode_group_71": ([700], [1], 71, 1, 64, 64, False, False),
    "verify_5": ([300, 5, 1111], [5] * 3, 8, 4, 128, 16, False, False),
    "verify_more_new_than_cached": ([3, 1, 20], [6] * 3, 4, 2, 64, 16, False, False),
    "rows_33_of_64": ([500, 70], [11, 11], 3, 1, 128, 32, False, False),
    "empty_cache": ([0, 10, 0], [1] * 3, 4, 2, 64, 16, False, False),
    "packed_ragged": ([600, 0, 33, 1025, 64], [3, 0, 1, 9, 0], 8, 2, 128, 16, True, False),
    "packed_empty_keys": ([0, 40], [4, 4], 2, 2, 64, 16, True, False),
    "chunk_100": ([100, 260], [100, 100], 4, 2, 128, 64, False, False),
    "chunk_whole_prompt": ([257], [257], 8, 2, 64, 16, False, True),
    "chunk_packed": ([400, 1300, 129], [129, 1, 128], 6, 2, 128, 32, True, False),
    "chunk_late": ([3000], [200], 8, 1, 128, 128, False, False),
    "chunk_more_new_than_cached": ([150, 300, 1], [300] * 3, 4, 2, 128, 16, False, False),
    "many_sequences": ([1 + 13 * b % 700 for b in range(150)], [1] * 150, 4, 2, 64, 16, False, False),
    "chunk_group_5": ([200, 333], [55, 55], 10, 2, 128, 16, False, False),
    "chunk_group_7": ([90, 20, 400], [90, 0, 31], 7, 1, 64, 32, True, False),
    "chunk_group_130": ([150], [3], 130, 1, 128, 64, False, False),
    "chunk_group_12": ([700, 100], [23, 23], 24, 2, 64, 16, False, True),
    "large_page": ([5000, 1], [2, 2], 8, 8, 128, 4096, False, False),
}


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(ATTEND))
def test_attend(pkg, name, fp8, causal):
    lens_k, lens_q, hq, hkv, dim, page, packed, head_major = ATTEND[name]
    p = R.make(lens_k, lens_q, hq, hkv, dim, page, fp8=fp8, packed=packed, head_major=head_major, seed=11)
    o, lse = pkg.paged_forward(p.q, *p.cache, causal=causal, cu_seqlens_q=p.cu_q,
                               max_seqlen_q=max(lens_q) if packed else None, **p.scales)
    pkg.check()
    R.check_attend(p, o, lse, causal)
    again, lse2 = pkg.paged_forward(p.q, *p.cache, causal=causal, cu_seqlens_q=p.cu_q,
                                    max_seqlen_q=max(lens_q) if packed else None, **p.scales)
    assert torch.equal(R.bits(o), R.bits(again)) and torch.equal(R.bits(lse), R.bits(lse2))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_attend_long_context_of_few_rows(pkg, fp8):
    """One KV head over 70000 keys: every CTA holds a part of one segment."""
    p = R.make([70000], [1], 2, 1, 128, 64, fp8=fp8, seed=12)
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    R.check_attend(p, o, lse, True)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens_k,hkv,group,new,dim", [
    ([9000, 1], 32, 1, 1, 64),              # a CTA has more heads than one
    ([5000, 700, 2600], 12, 2, 3, 128),     # a grid that the heads do not divide
    ([4000, 0, 3000], 17, 1, 1, 128),       # no divisor
    ([40000], 6, 16, 2, 128),               # segments cut into many parts, 32 rows
    ([30000, 20000], 2, 24, 1, 64)])        # row tiles and heads
def test_attend_many_kv_heads(pkg, lens_k, hkv, group, new, dim, fp8):
    """How heads are dealt to CTAs, and who joins the parts of which segment."""
    p = R.make(lens_k, [min(new, n) for n in lens_k], hkv * group, hkv, dim, 32, fp8=fp8, packed=True, seed=31)
    o, lse = pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=p.cu_q, max_seqlen_q=new, **p.scales)
    pkg.check()
    R.check_attend(p, o, lse, True)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("batch,hkv,group,new,longest", [
    (75, 8, 1, 1, 1000),     # two segments to a CTA, none cut
    (75, 3, 4, 2, 3000),     # more than one window of 32 lengths, segments cut
    (300, 2, 2, 1, 90),      # many short ones
    (1100, 1, 2, 1, 40),     # more than 1024 lengths
    (2300, 1, 1, 3, 700)])
def test_attend_many_sequences(pkg, batch, hkv, group, new, longest, fp8):
    """How the kernel finds its sequences among many, empty ones between them."""
    lens_k = [0 if b % 5 == 3 or 40 <= b < 80 and batch > 200 else 1 + (b * 7919) % longest for b in range(batch)]
    lens_k[batch // 2] = longest
    p = R.make(lens_k, [min(new, n) for n in lens_k], hkv * group, hkv, 64, 16, fp8=fp8, packed=True, seed=32)
    o, lse = pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=p.cu_q, max_seqlen_q=new, **p.scales)
    pkg.check()
    R.check_attend(p, o, lse, True)


def test_attend_large_scores(pkg):
    """Scores of both signs in the thousands: the running maximum has to move
    and no exponential may overflow. (The reference bound for LSE assumes
    ordinary scores: here it is one ulp of the score's magnitude, 2^-11, times
    the few roundings on its way.)"""
    p = R.make([700, 90], [3, 3], 4, 2, 64, 16, seed=13)
    p.q *= 200
    o, lse = pkg.paged_forward(p.q, *p.cache, softmax_scale=1.0)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True, 1.0)):
        assert torch.isfinite(lse[b]).all() and torch.isfinite(o[b].float()).all()
        assert (lse[b].double() - rl).abs().max() <= 8 * 2.0 ** -24 * rl.abs().max() * 8


def test_attend_views_and_scale(pkg):
    """q inside a fused projection, out inside a wider tensor, a table that is
    a view of a larger one, a bound on the lengths, no LSE."""
    p = R.make([130, 70], [2, 2], 8, 2, 128, 32, seed=14)
    fused = torch.randn(2, 2, 12, 128, device="cuda").to(torch.bfloat16)
    fused[:, :, 2:10] = p.q
    wide = torch.zeros(2, 2, 8, 256, dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, 40), -5, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = p.table
    o, lse = pkg.paged_forward(fused[:, :, 2:10], p.k_cache, p.v_cache, table[:, :p.table.shape[1]], p.seqlens,
                               softmax_scale=0.3, max_seqlen_k=130, out=wide[..., 128:], return_lse=False)
    pkg.check()
    assert lse is None and bool((wide[..., :128] == 0).all())
    _, l = pkg.paged_forward(p.q, *p.cache, softmax_scale=0.3)
    R.check_attend(p, o, l, True, 0.3)


def test_attend_leaves_rows_behind_the_last_sequence(pkg):
    for lens_q, hq in (([2, 1], 4), ([150, 90], 4)):
        p = R.make([300, 95], lens_q, hq, 2, 64, 16, packed=True, seed=15)
        n = sum(lens_q)
        q = torch.cat([p.q, torch.full((6, hq, 64), math.nan, dtype=torch.bfloat16, device="cuda")])
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((hq, n + 6), 7.0, device="cuda")
        pkg.paged_forward(q, *p.cache, cu_seqlens_q=p.cu_q, max_seqlen_q=max(lens_q), out=out, lse=lse)
        pkg.check()
        assert bool((out[n:] == 7.0).all()) and bool((lse[:, n:] == 7.0).all())
        R.check_attend(p, out[:n], lse[:, :n], True)


@pytest.mark.parametrize("new", [1, 200])
def test_cache_beyond_32_bit_offsets(pkg, new):
    """Pages whose element offsets pass 2^31 (a 4.4 GB K cache)."""
    p = R.make([new + 40], [new], 4, 2, 128, 64, seed=16, high_pages=(1 << 31) // (64 * 2 * 128) + 3)
    pkg.cache_append(p.k_new, p.v_new, *p.cache)
    o, lse = pkg.paged_forward(p.q, *p.cache)
    pkg.check()
    R.check_attend(p, o, lse, True)
    k, _ = R.gather(p, 0)
    assert torch.equal(k[-new:], p.k_new[0].double())
    cu = torch.tensor([0, new + 40], dtype=torch.int32, device="cuda")
    kr, _ = pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, total_k=new + 40)
    assert torch.equal(kr.double(), k)


# ---------------------------------------------------------------- what only the device sees
def _bad(pkg, p, **kw):
    with pytest.raises(pkg.AttnError, match="paged cache"):
        pkg.check()
    pkg.check()   # reported once


@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("what", ["page_high", "page_negative", "length_high", "length_negative", "offsets"])
def test_bad_device_values_are_reported(pkg, what, new):
    """Reported by check(); rows of the other sequence are right, nothing faults."""
    packed = what == "offsets"
    p = R.make([200, 150], [new] * 2, 4, 2, 64, 16, packed=packed, seed=17)
    table, seqlens, cu = p.table.clone(), p.seqlens.clone(), p.cu_q
    if what == "page_high":
        table[1, 3] = p.k_cache.shape[0]
    elif what == "page_negative":
        table[1, 0] = -1
    elif what == "length_high":
        seqlens[1] = 1 << 30
    elif what == "length_negative":
        seqlens[1] = -4
    else:
        cu = torch.tensor([0, new, new - 1], dtype=torch.int32, device="cuda")
    before = p.k_cache.clone()
    o, lse = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, seqlens, cu_seqlens_q=cu,
                               max_seqlen_q=new if packed else None)
    _bad(pkg, p)
    (ro, rl, ra) = R.attend(p, True)[0]
    got = o[:new] if packed else o[0]
    assert ((got.double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 1e-6).all()
    # append: pages that no longer hold sequence 1 are not written
    if what != "offsets":
        if what.startswith("page"):
            table[1] = -1 if what == "page_negative" else p.k_cache.shape[0]
        pkg.cache_append(p.k_new, p.v_new, p.k_cache, p.v_cache, table, seqlens)
        _bad(pkg, p)
        for b, c in ((1, c) for c in range(10)):
            at = int(p.table[b, c])
            assert torch.equal(R.bits(p.k_cache[at]), R.bits(before[at]))


def test_bad_reads_are_reported(pkg):
    p = R.make([40, 30], [1, 1], 2, 2, 64, 16, seed=18)
    out = torch.full((70, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    long = torch.tensor([0, 40, 40 + 16 * p.table.shape[1] + 1], dtype=torch.int32, device="cuda")
    n = int(long[-1])
    big = torch.full((n, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    table = p.table.clamp(max=p.k_cache.shape[0] - 1)   # every column names a page
    pkg.cache_read(p.k_cache, p.v_cache, table, long, out_k=big, out_v=big.clone())
    _bad(pkg, p)
    assert bool((big[n - 1] == 7.0).all())
    table = p.table.clone()
    table[1, 1] = -7
    cu = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    pkg.cache_read(p.k_cache, p.v_cache, table, cu, out_k=out, out_v=out.clone())
    _bad(pkg, p)
    assert bool((out[40 + 16:] == 7.0).all())
    assert torch.equal(out[:40].double(), R.gather(p, 0)[0])


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_prompt_chunks_then_steps_match_contiguous_attention(pkg, fp8):
    """Two prompts enter the cache in chunks, tokens follow one by one; every
    output matches forward()'s causal attention over what cache_read returns
    (both round the same quantities, so their difference is at most twice the
    bound of one)."""
    hq, hkv, dim, page, n = 8, 2, 128, 32, 333
    g = torch.Generator(device="cuda").manual_seed(20)
    q, k, v = (torch.randn(2, n, h, dim, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    pages = 2 * (-(-n // page))
    dt = R.E4M3 if fp8 else torch.bfloat16
    kc, vc = (torch.zeros(pages, page, hkv, dim, device="cuda").to(dt) for _ in range(2))
    sc = dict(k_scale=torch.zeros(pages, hkv, page, device="cuda"),
              v_scale=torch.zeros(pages, hkv, page, device="cuda")) if fp8 else {}
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(2, -1)
    outs, lses, at = [], [], 0
    for step in (150, 150, 17, 9, 1, 1, 1, 1, 1, 1, 1):
        lens = torch.full((2,), at + step, dtype=torch.int32, device="cuda")
        new = slice(at, at + step)
        pkg.cache_append(k[:, new], v[:, new], kc, vc, table, lens, **sc)
        o, lse = pkg.paged_forward(q[:, new], kc, vc, table, lens, **sc)
        outs.append(o)
        lses.append(lse)
        at += step
    assert at == n
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    kr, vr = pkg.cache_read(kc, vc, table, cu, total_k=2 * n, **sc)
    kr, vr = kr.view(2, n, hkv, dim), vr.view(2, n, hkv, dim)
    o_ref, lse_ref = pkg.forward(q, kr, vr, causal=True)
    pkg.check()
    if not fp8:
        assert torch.equal(R.bits(kr), R.bits(k)) and torch.equal(R.bits(vr), R.bits(v))
    o, lse = torch.cat(outs, 1), torch.cat(lses, 2)
    _, _, absv = zip(*_contiguous(q, kr, vr))
    bound = 2 * (2.0 ** -8 * o_ref.double().abs() + (2.0 ** -8 + 2.0 ** -14) * torch.stack(absv) + 1e-6)
    assert bool(((o.double() - o_ref.double()).abs() <= bound).all())
    assert (lse - lse_ref).abs().max().item() <= 1e-4


def _contiguous(q, k, v):
    n, (hq, dim), hkv = q.shape[1], q.shape[2:], k.shape[2]
    p = R.Problem(k, v, None, None, torch.arange(q.shape[0])[:, None], None, [n] * q.shape[0], [n] * q.shape[0], None,
                  q, k, v)
    return R.attend(p, True)


def _graph(pkg, p, out, lse, o2=None):
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        pkg.cache_append(p.k_new, p.v_new, *p.cache, cu_seqlens_q=p.cu_q, **p.scales)
        pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=p.cu_q,
                          max_seqlen_q=None if p.cu_q is None else max(p.lens_q), out=out, lse=lse, **p.scales)
    return graph


@pytest.mark.parametrize("new,hq", [(1, 8), (160, 8)])
def test_captured_step_follows_the_lengths(pkg, new, hq):
    """A captured append + attention replayed with other lengths on the device
    (a serving loop) gives what eager calls give; two such graphs replayed at
    once on two streams do not disturb each other. The first use of the
    library on a stream may be the capture itself."""
    graphs = []
    for seed in (21, 22):
        p = R.make([new + 900, new + 500], [new] * 2, hq, 2, 128, 32, seed=seed, poison=False)
        out, lse = torch.empty_like(p.q), torch.empty(2, hq, new, device="cuda")
        graphs.append((p, out, lse, _graph(pkg, p, out, lse)))
    streams = [torch.cuda.Stream() for _ in graphs]
    for lens in ([new + 900, new + 500], [new, new + 333], [new + 17, new + 400]):
        want = []
        for p, out, lse, _ in graphs:
            p.seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
            p.lens_k[:] = lens
        torch.cuda.synchronize()
        for _ in range(5):
            for s, (p, out, lse, graph) in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for p, out, lse, _ in graphs:
            o, l = pkg.paged_forward(p.q, *p.cache)
            pkg.check()
            assert torch.equal(R.bits(o), R.bits(out)) and torch.equal(R.bits(l), R.bits(lse))
            R.check_attend(p, out, lse, True)


def test_two_streams_at_once(pkg):
    """Calls of different sizes on two streams share no workspace."""
    ps = [R.make([3000, 2000], [n] * 2, 8, 2, 128, 64, seed=s) for n, s in ((1, 23), (1, 24), (140, 25))]
    want = [pkg.paged_forward(p.q, *p.cache) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for _ in range(10):
        got = [pkg.paged_forward(p.q, *p.cache, stream=s) for s, p in zip(streams, ps)]
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(R.bits(o), R.bits(wo)) and torch.equal(R.bits(l), R.bits(wl))
    for s in streams:
        pkg.check(stream=s)
    o, l = pkg.paged_forward(ps[0].q, *ps[0].cache, stream=streams[1].cuda_stream)   # a bare handle
    pkg.check(stream=streams[1])
    assert torch.equal(R.bits(o), R.bits(want[0][0])) and torch.equal(R.bits(l), R.bits(want[0][1]))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 130])
def test_sequences_that_share_pages(pkg, new, fp8):
    """A common prefix in the same pages, and a page that a sequence names twice."""
    p = R.make([2000, 2000], [new] * 2, 4, 2, 64, 16, fp8=fp8, seed=34)
    p.table[1, :124] = p.table[0, :124]
    p.table[:, 7] = p.table[:, 3]
    p.q[1] = p.q[0]
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    R.check_attend(p, o, lse, True)
    p.table[1] = p.table[0]
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    R.check_attend(p, o, lse, True)
    cu = torch.tensor([0, 2000, 4000], dtype=torch.int32, device="cuda")
    k, v = pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, total_k=4000, **p.scales)
    pkg.check()
    assert torch.equal(R.bits(k[:2000]), R.bits(k[2000:])) and torch.equal(R.bits(v[:2000]), R.bits(v[2000:]))
    assert torch.equal(R.bits(k[48:64]), R.bits(k[112:128]))


def test_offsets_past_the_rows_are_reported(pkg):
    """Fewer rows than the offsets claim: what is there of the other sequences is right."""
    p = R.make([40, 30], [5, 6], 2, 2, 64, 16, packed=True, seed=35)
    want = R.append(p)
    before = p.k_cache.clone()
    pkg.cache_append(p.k_new[:-1], p.v_new[:-1], *p.cache, cu_seqlens_q=p.cu_q)
    _bad(pkg, p)
    pages = p.table[0, :3].long()
    assert torch.equal(R.bits(p.k_cache[pages]), R.bits(want[0][pages]))
    pages = p.table[1, :2].long()
    assert torch.equal(R.bits(p.k_cache[pages]), R.bits(before[pages]))
    cu = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    k, _ = pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, total_k=69)
    _bad(pkg, p)
    assert torch.equal(k[:40].double(), R.gather(p, 0)[0])


def test_append_with_a_length_far_below_zero(pkg):
    """lk - lq must not wrap around to a position that exists."""
    page, n = 65536, 70000
    k_cache = torch.full((1, page, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    v_cache = k_cache.clone()
    table = torch.zeros(1, 0x7fff0000 // page, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), -2 ** 31, dtype=torch.int32, device="cuda")
    new = torch.zeros(1, n, 1, 64, dtype=torch.bfloat16, device="cuda")
    pkg.cache_append(new, new, k_cache, v_cache, table, lens)
    with pytest.raises(pkg.AttnError, match="out of range"):
        pkg.check()
    assert bool((k_cache == 3.0).all()) and bool((v_cache == 3.0).all())


def test_stream_of_another_device_is_refused(pkg):
    p = R.make([20], [1], 2, 2, 64, 16, seed=33)
    other = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="another device"):
        pkg.cache_append(p.k_new, p.v_new, *p.cache, stream=other)
    with pytest.raises(ValueError, match="another device"):
        pkg.paged_forward(p.q, *p.cache, stream=other)


def test_own_workspace(pkg):
    p = R.make([1300, 40], [1, 1], 8, 2, 64, 16, seed=26)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    pkg.cache_append(p.k_new, p.v_new, *p.cache, workspace=ws)
    o, lse = pkg.paged_forward(p.q, *p.cache, workspace=ws)
    pkg.check(workspace=ws)
    R.check_attend(p, o, lse, True)
    with pytest.raises(pkg.AttnError, match="workspace"):
        pkg.paged_forward(p.q, *p.cache, workspace=ws[:256])
    table = p.table.clone()
    table[0, 0] = -1
    pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, workspace=ws)
    with pytest.raises(pkg.AttnError, match="sequence 0"):
        pkg.check(workspace=ws)


def test_no_rows(pkg):
    p = R.make([20], [1], 2, 2, 64, 16, seed=27)
    o, lse = pkg.paged_forward(p.q[:, :0], *p.cache)
    assert o.shape == (1, 0, 2, 64) and lse.shape == (1, 2, 0)
    o, lse = pkg.paged_forward(p.q[:0], p.k_cache, p.v_cache, p.table[:0], p.seqlens[:0])
    assert o.shape == (0, 1, 2, 64)
    pkg.cache_append(p.k_new[:0], p.v_new[:0], p.k_cache, p.v_cache, p.table[:0], p.seqlens[:0])
    k, v = pkg.cache_read(p.k_cache, p.v_cache, p.table, torch.zeros(2, dtype=torch.int32, device="cuda"), total_k=0)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    pkg.check()


def test_overlapping_offsets_are_reported(pkg):
    """Offsets that go back and forth claim more rows than there are: no list
    or scratch is overrun, and check() says so."""
    p = R.make([400] * 6, [0, 0, 0, 0, 0, 240], 4, 2, 64, 16, packed=True, seed=28)
    cu = torch.tensor([0, 240, 0, 240, 0, 240, 240], dtype=torch.int32, device="cuda")
    pkg.paged_forward(p.q, *p.cache, cu_seqlens_q=cu, max_seqlen_q=240)
    _bad(pkg, p)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens_k,lens_q,hq,hkv,dim,page", [
    ([9000], [256], 4, 4, 128, 64),                      # few tiles, each cut in many pieces
    ([5000], [300], 16, 2, 64, 128),                     # pieces across tile borders
    ([4100, 1300, 2600, 1029], [200, 900, 1, 130], 8, 2, 128, 32),   # ragged, whole tiles and cut ones
    ([1200] * 40, [70] * 40, 6, 2, 64, 16),              # several waves, heads in pairs
    ([1500, 0, 1100, 3], [40, 5, 0, 100], 32, 1, 64, 16),
])
def test_attend_chunks_that_are_cut(pkg, lens_k, lens_q, hq, hkv, dim, page, fp8):
    p = R.make(lens_k, lens_q, hq, hkv, dim, page, fp8=fp8, packed=True, seed=29)
    for causal in (True, False):
        kw = dict(causal=causal, cu_seqlens_q=p.cu_q, max_seqlen_q=max(lens_q), **p.scales)
        o, lse = pkg.paged_forward(p.q, *p.cache, **kw)
        pkg.check()
        R.check_attend(p, o, lse, causal)
        o2, lse2 = pkg.paged_forward(p.q, *p.cache, **kw)
        assert torch.equal(R.bits(o), R.bits(o2)) and torch.equal(R.bits(lse), R.bits(lse2))


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens_k,lens_q,hq,hkv,dim,page,head_major", [
    ([700, 0, 129, 1300], [600, 0, 129, 900], 2, 1, 64, 16, True),     # empty, one past a tile, whole prompts
    ([2500, 333], [200, 333], 12, 3, 128, 32, False),
    ([65, 1], [65, 1], 32, 1, 128, 128, False),                        # a bare tile
    ([5000], [1030], 4, 4, 128, 256, False)])
def test_attend_e4m3_chunks_widened_or_not(pkg, lens_k, lens_q, hq, hkv, dim, page, head_major, causal):
    """Long chunks read a bf16 copy of the sequences, unless a bound on the
    lengths asks for too much scratch memory; the exact copy of the writer's
    values keeps the bound either way."""
    p = R.make(lens_k, lens_q, hq, hkv, dim, page, fp8=True, packed=True, head_major=head_major, seed=36)
    wide = torch.full((len(lens_k), (1 << 21) // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :p.table.shape[1]] = p.table
    for table in (p.table, wide):
        o, lse = pkg.paged_forward(p.q, p.k_cache, p.v_cache, table, p.seqlens, causal=causal, cu_seqlens_q=p.cu_q,
                                   max_seqlen_q=max(lens_q), **p.scales)
        pkg.check()
        R.check_attend(p, o, lse, causal)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_rows_on_16_byte_boundaries_only(pkg, fp8):
    """New rows, outputs and q whose strides are odd multiples of 16 bytes."""
    p = R.make([90, 40], [30, 30], 4, 2, 64, 16, fp8=fp8, seed=30)
    wide = torch.full((2, 30, 2, 3 * 72 + 8), 3.0, dtype=torch.bfloat16, device="cuda")[..., 8:]
    k, v = wide[..., :64], wide[..., 72:136]
    k.copy_(p.k_new)
    v.copy_(p.v_new)
    want = R.append(p)
    pkg.cache_append(k, v, *p.cache, **p.scales)
    for g, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
        assert g is None or torch.equal(R.bits(g), R.bits(w))
    cu = torch.tensor([0, 90, 130], dtype=torch.int32, device="cuda")
    out = torch.full((130, 2, 152), 5.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, out_k=out[..., 8:72], out_v=out[..., 80:144], **p.scales)
    both = [torch.cat(x).to(torch.bfloat16) for x in zip(*(R.gather(p, b) for b in range(2)))]
    assert torch.equal(out[..., 8:72], both[0]) and torch.equal(out[..., 80:144], both[1])
    assert bool((out[..., :8] == 5.0).all()) and bool((out[..., 72:80] == 5.0).all()) and bool((out[..., 144:] == 5.0).all())
    for n in (30, 4):   # either attention kernel
        q = torch.zeros(2, n, 4, 72, dtype=torch.bfloat16, device="cuda")[..., 8:]
        q.copy_(p.q[:, 30 - n:])
        o = torch.full((2, n, 4, 88), 5.0, dtype=torch.bfloat16, device="cuda")
        _, lse = pkg.paged_forward(q, *p.cache, out=o[..., 8:72], **p.scales)
        p2 = R.Problem(p.k_cache, p.v_cache, p.k_scale, p.v_scale, p.table, p.seqlens, p.lens_k, [n, n], None, q, None, None)
        R.check_attend(p2, o[..., 8:72], lse, True)
        assert bool((o[..., :8] == 5.0).all()) and bool((o[..., 72:] == 5.0).all())
    pkg.check()


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("spread", ["powers", "any", "growing", "zero_and_negative"])
def test_attend_e4m3_scales_that_differ(pkg, spread, new):
    """Value scales over many orders of magnitude, in any order, not only powers
    of two; zero vectors, zero and negative scales. The chunk kernel (60 rows)
    may round code * scale to bf16 once more: 2^-8 of every value, and as much
    of every key, which moves the scores by less than 2^-8 * scale * sum |q k|."""
    p = R.make([1500, 700], [new] * 2, 4, 1, 64, 16, fp8=True, seed=31)
    g = torch.Generator().manual_seed(32)
    for s, c in ((p.k_scale, p.k_cache), (p.v_scale, p.v_cache)):
        held = ~torch.isnan(s)
        n = int(held.sum())
        if spread == "powers":
            x = torch.exp2(torch.randint(-40, 11, (n,), generator=g).double())
        elif spread == "any":
            x = torch.exp2(torch.rand(n, generator=g).double() * 12 - 14) * 1.2345
        elif spread == "growing":
            x = torch.exp2(torch.linspace(-30, 5, n).double())
        else:
            x = torch.exp2(torch.randint(-8, -4, (n,), generator=g).double()) * torch.randint(-1, 2, (n,), generator=g)
        if s is p.k_scale:   # scores stay ordinary
            x = x.sign() * x.abs().clamp(max=2.0 ** -7)
        s[held] = x.float().cuda()
    p.v_cache[p.table[0, 3].long(), 5] = 0.0
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        wide = new * 4 > 32 and spread in ("any", "growing")
        k, _ = R.gather(p, b)
        q = p.q[b].double()
        ds = 2.0 ** -8 * 64 ** -0.5 * (q.abs() @ k[:, 0].abs().t()).max().item() if wide else 0.0
        grow = math.expm1(2 * ds)
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14 + (2.0 ** -8 if wide else 0.0) + grow) * ra * (1 + grow) + 1e-6 * ra.max()
        assert ((o[b].double() - ro).abs() <= bound).all()
        assert (lse[b].double() - rl).abs().max().item() <= 5e-5 + ds
