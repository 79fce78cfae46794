"""The 4-bit paged cache on the GPU: writing (bit for bit, with and without
rotation), reading back (bit for bit), attention (every element within the bound
its roundings imply), what only the device can refuse, and runs of them together.
Slots that no sequence holds have NaN scales throughout."""
import math

import pytest
import torch

import paged4_reference as R4
import paged_reference as R
import test_gpu_paged as G
import test_gpu_rotary as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("name", list(G.APPEND))
def test_append_writes_exactly_its_slots(pkg, name):
    lens_k, lens_q, hkv, dim, page, packed, head_major = G.APPEND[name]
    p = R4.make(lens_k, lens_q, hkv, hkv, dim, page, packed=packed, head_major=head_major, seed=3)
    want = R4.append(p)
    pkg.cache_append(p.p.k_new, p.p.v_new, *p.cache, cu_seqlens_q=p.p.cu_q, **p.scales)
    pkg.check()
    R4.same(p.all(), want)


@pytest.mark.parametrize("name", list(T.APPEND))
def test_append_with_rotation(pkg, name):
    lens_k, lens_q, hq, hkv, dim, page, packed, rot, inter = T.APPEND[name]
    p = R4.make(lens_k, lens_q, hq, hkv, dim, page, packed=packed, seed=4)
    table = R4.angles(max(lens_k), rot)
    want = R4.append(p, table, interleaved=inter)
    q2 = pkg.cache_append(p.p.k_new, p.p.v_new, *p.cache, cu_seqlens_q=p.p.cu_q, rotary_table=table, interleaved=inter,
                          q=p.p.q, **p.scales)
    pkg.check()
    R4.same(p.all(), want)
    at = torch.cat([torch.arange(k - q, k) for k, q in zip(lens_k, lens_q)]).cuda()
    T.check_turned(q2.reshape(-1, hq, dim), p.p.q.reshape(-1, hq, dim), table, at, inter)


def test_append_of_special_values(pkg):
    """Zeros, subnormals, the largest finite values, ties, infinities and NaN; every
    quotient that a bf16 value and a block scale can give near a border."""
    p = R4.make([80], [80], 2, 2, 64, 16, seed=5)
    x = p.p.k_new
    x[0, 0] = 0.0
    x[0, 1] = 2.0 ** -133                      # the smallest bf16
    x[0, 2, 0] = 2.0 ** -126
    x[0, 3] = torch.finfo(torch.bfloat16).max
    x[0, 4, 0, 3] = math.inf
    x[0, 5, 1, 7] = -math.inf
    x[0, 6, 0, 9] = math.nan
    x[0, 7] = math.inf
    x[0, 8] = math.nan
    x[0, 9] = 2688.0
    x[0, 10] = 2704.0                          # just past 6 * 448: the next scale
    x[0, 11] = torch.linspace(-6, 6, 64).to(torch.bfloat16)
    x[0, 12, :, 0] = 3.0e38
    x[0, 13, 0, 16:] = 0.0                     # empty blocks
    x[0, 14, 0, 16:32] *= 2.0 ** -17           # block scales below e4m3's normal range
    x[0, 14, 0, 32:48] *= 2.0 ** -20
    x[0, 15] = -0.0
    # a block's largest value 6 * 2^8 * m makes its scale an e4m3 value: the others sit on the codes' borders
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0])
    for i in range(64):
        size = (8 + i % 8) * 2.0 ** (i // 8 - 6)
        x[0, 16 + i] = torch.cat([borders * size, torch.tensor([6.0 * size])]).repeat(4).to(torch.bfloat16)
        assert bool((x[0, 16 + i, 0, :15].double().cpu() == borders.double() * size).all())
    p.p.v_new[0, :, 1] = x[0, :, 0]
    want = R4.append(p)
    pkg.cache_append(x, p.p.v_new, *p.cache, **p.scales)
    pkg.check()
    R4.same(p.all(), want)


@pytest.mark.parametrize("lens_k,hkv,dim,page,head_major", [
    ([1], 1, 64, 16, False), ([33, 0, 64, 1, 250], 3, 128, 32, True), ([3000, 2049], 8, 128, 64, False),
    ([1 + b % 7 for b in range(400)], 2, 64, 16, False)])
@pytest.mark.parametrize("as_type", [torch.uint8, torch.float4_e2m1fn_x2])
def test_read_gives_the_cached_values(pkg, lens_k, hkv, dim, page, head_major, as_type):
    p = R4.make(lens_k, [0] * len(lens_k), hkv, hkv, dim, page, packed=True, head_major=head_major, seed=7)
    total = sum(lens_k)
    cu = torch.tensor([sum(lens_k[:b]) for b in range(len(lens_k) + 1)], dtype=torch.int32, device="cuda")
    kc, vc = p.k_cache.view(as_type), p.v_cache.view(as_type)
    k, v = pkg.cache_read(kc, vc, p.p.table, cu, total_k=total, **p.scales)
    both = torch.full((total + 5, 2, hkv, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_read(kc, vc, p.p.table, cu, out_k=both[:, 0], out_v=both[:, 1], **p.scales)
    pkg.check()
    want = [torch.cat(x).to(torch.bfloat16) for x in zip(*(R.gather(p.p, b) for b in range(len(lens_k))))]
    assert torch.equal(R.bits(k), R.bits(want[0])) and torch.equal(R.bits(v), R.bits(want[1]))
    assert torch.equal(R.bits(both[:total, 0]), R.bits(want[0])) and torch.equal(R.bits(both[:total, 1]), R.bits(want[1]))
    assert bool((both[total:] == 7.0).all())


# ---------------------------------------------------------------- attend
def _attend(pkg, p, causal=True, **kw):
    if p.p.cu_q is not None:
        kw = dict(dict(cu_seqlens_q=p.p.cu_q, max_seqlen_q=max(p.p.lens_q)), **kw)
    return pkg.paged_forward(p.p.q, *p.cache, causal=causal, **p.scales, **kw)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name", list(G.ATTEND))
def test_attend(pkg, name, causal):
    lens_k, lens_q, hq, hkv, dim, page, packed, head_major = G.ATTEND[name]
    p = R4.make(lens_k, lens_q, hq, hkv, dim, page, packed=packed, head_major=head_major, seed=11)
    o, lse = _attend(pkg, p, causal)
    pkg.check()
    R.check_attend(p.p, o, lse, causal)
    again, lse2 = _attend(pkg, p, causal)
    assert torch.equal(R.bits(o), R.bits(again)) and torch.equal(R.bits(lse), R.bits(lse2))


def test_attend_long_context_of_few_rows(pkg):
    p = R4.make([70000], [1], 2, 1, 128, 64, seed=12)
    o, lse = _attend(pkg, p)
    pkg.check()
    R.check_attend(p.p, o, lse, True)


@pytest.mark.parametrize("lens_k,hkv,group,new,dim", [
    ([9000, 1], 32, 1, 1, 64), ([5000, 700, 2600], 12, 2, 3, 128), ([4000, 0, 3000], 17, 1, 1, 128),
    ([40000], 6, 16, 2, 128), ([30000, 20000], 2, 24, 1, 64), ([6000, 31], 4, 16, 2, 64)])
def test_attend_many_kv_heads(pkg, lens_k, hkv, group, new, dim):
    p = R4.make(lens_k, [min(new, n) for n in lens_k], hkv * group, hkv, dim, 32, packed=True, seed=31)
    o, lse = _attend(pkg, p, max_seqlen_q=new)
    pkg.check()
    R.check_attend(p.p, o, lse, True)


@pytest.mark.parametrize("batch,hkv,group,new,longest", [
    (75, 8, 1, 1, 1000), (75, 3, 4, 2, 3000), (300, 2, 2, 1, 90), (1100, 1, 2, 1, 40), (1500, 1, 1, 3, 300)])
def test_attend_many_sequences(pkg, batch, hkv, group, new, longest):
    lens_k = [0 if b % 5 == 3 or 40 <= b < 80 and batch > 200 else 1 + (b * 7919) % longest for b in range(batch)]
    lens_k[batch // 2] = longest
    p = R4.make(lens_k, [min(new, n) for n in lens_k], hkv * group, hkv, 64, 16, packed=True, seed=32)
    o, lse = _attend(pkg, p, max_seqlen_q=new)
    pkg.check()
    R.check_attend(p.p, o, lse, True)


@pytest.mark.parametrize("lens_k,lens_q,hq,hkv,dim,page", [
    ([9000], [256], 4, 4, 128, 64), ([5000], [300], 16, 2, 64, 128),
    ([4100, 1300, 2600, 1029], [200, 900, 1, 130], 8, 2, 128, 32), ([1200] * 40, [70] * 40, 6, 2, 64, 16),
    ([1500, 0, 1100, 3], [40, 5, 0, 100], 32, 1, 64, 16), ([1700, 90, 33], [12, 9, 16], 8, 2, 128, 16),
    ([2100, 12], [33, 12], 2, 2, 64, 128)])
def test_attend_chunks_over_the_copy_and_without_it(pkg, lens_k, lens_q, hq, hkv, dim, page):
    """More than 64 rows read a bf16 copy, or, where a bound on the lengths asks for
    too much scratch memory, go over the cache 32 rows at a time."""
    p = R4.make(lens_k, lens_q, hq, hkv, dim, page, packed=True, seed=29)
    wide = torch.full((len(lens_k), (1 << 23) // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :p.p.table.shape[1]] = p.p.table
    for causal in (True, False):
        for table in (p.p.table, wide):
            o, lse = pkg.paged_forward(p.p.q, p.k_cache, p.v_cache, table, p.p.seqlens, causal=causal,
                                       cu_seqlens_q=p.p.cu_q, max_seqlen_q=max(lens_q), **p.scales)
            pkg.check()
            R.check_attend(p.p, o, lse, causal)


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("spread", ["powers", "any", "growing", "zero_and_negative"])
def test_attend_scales_that_differ(pkg, spread, new):
    """Scales over many orders of magnitude, not only powers of two, zero and negative
    ones. The copy that 60 tokens read may round code * block scale * scale: 2^-8 of
    every value, and as much of every key, which moves the scores by less than
    2^-8 * scale * sum |q k|."""
    p = R4.make([1500, 700], [new] * 2, 4, 1, 64, 16, seed=31)
    g = torch.Generator().manual_seed(32)
    for s in (p.k_scale, p.v_scale):
        held = ~torch.isnan(s)
        n = int(held.sum())
        if spread == "powers":
            x = torch.exp2(torch.randint(-40, 11, (n,), generator=g).double())
        elif spread == "any":
            x = torch.exp2(torch.rand(n, generator=g).double() * 12 - 17) * 1.2345
        elif spread == "growing":
            x = torch.exp2(torch.linspace(-30, 2, n).double())
        else:
            x = torch.exp2(torch.randint(-11, -7, (n,), generator=g).double()) * torch.randint(-1, 2, (n,), generator=g)
        if s is p.k_scale:   # scores stay ordinary
            x = x.sign() * x.abs().clamp(max=2.0 ** -10)
        s[held] = x.float().cuda()
    p.refresh()
    o, lse = _attend(pkg, p)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p.p, True)):
        wide = new * 4 > 32 and spread in ("any", "growing")
        k, _ = R.gather(p.p, b)
        q = p.p.q[b].double()
        ds = 2.0 ** -8 * 64 ** -0.5 * (q.abs() @ k[:, 0].abs().t()).max().item() if wide else 0.0
        grow = math.expm1(2 * ds)
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14 + (2.0 ** -8 if wide else 0.0) + grow) * ra * (1 + grow) + 1e-6 * ra.max()
        assert ((o[b].double() - ro).abs() <= bound).all()
        assert (lse[b].double() - rl).abs().max().item() <= 5e-5 + ds


@pytest.mark.parametrize("new", [1, 60])
def test_nan_blocks(pkg, new):
    """A key with a NaN makes its row NaN in O and LSE; a value with one only its block's depths."""
    p = R4.make([300, 200], [new] * 2, 4, 1, 64, 16, seed=33)
    at, slot = int(p.p.table[0, 5]), 3
    p.v_block[at, 0, slot, 1] = math.nan
    at, _ = int(p.p.table[1, 2]), 0
    p.k_block[at, 0, 0, 2] = math.nan
    o, lse = _attend(pkg, p)
    pkg.check()
    assert bool(torch.isnan(o[0, ..., 16:32]).all())
    assert not bool(torch.isnan(o[0, ..., :16]).any()) and not bool(torch.isnan(o[0, ..., 32:]).any())
    assert not bool(torch.isnan(lse[0]).any()) and bool(torch.isnan(lse[1]).all()) and bool(torch.isnan(o[1]).all())


def test_attend_views_bound_and_scale(pkg):
    p = R4.make([130, 70], [2, 2], 8, 2, 128, 32, seed=14)
    fused = torch.randn(2, 2, 12, 128, device="cuda").to(torch.bfloat16)
    fused[:, :, 2:10] = p.p.q
    wide = torch.zeros(2, 2, 8, 256, dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, 40), -5, dtype=torch.int32, device="cuda")
    table[:, :p.p.table.shape[1]] = p.p.table
    room = torch.zeros(p.k_cache.shape[0], 32, 2, 160, dtype=torch.uint8, device="cuda")   # K and V beside each other
    room[..., :64], room[..., 80:144] = p.k_cache, p.v_cache
    o, lse = pkg.paged_forward(fused[:, :, 2:10], room[..., :64], room[..., 80:144], table[:, :p.p.table.shape[1]],
                               p.p.seqlens, softmax_scale=0.3, max_seqlen_k=130, out=wide[..., 128:], return_lse=False,
                               **p.scales)
    pkg.check()
    assert lse is None and bool((wide[..., :128] == 0).all())
    _, l = _attend(pkg, p, softmax_scale=0.3)
    R.check_attend(p.p, wide[..., 128:], l, True, 0.3)


def test_attend_leaves_rows_behind_the_last_sequence(pkg):
    for lens_q, hq in (([2, 1], 4), ([150, 90], 4)):
        p = R4.make([300, 95], lens_q, hq, 2, 64, 16, packed=True, seed=15)
        n = sum(lens_q)
        q = torch.cat([p.p.q, torch.full((6, hq, 64), math.nan, dtype=torch.bfloat16, device="cuda")])
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((hq, n + 6), 7.0, device="cuda")
        pkg.paged_forward(q, *p.cache, cu_seqlens_q=p.p.cu_q, max_seqlen_q=max(lens_q), out=out, lse=lse, **p.scales)
        pkg.check()
        assert bool((out[n:] == 7.0).all()) and bool((lse[:, n:] == 7.0).all())
        R.check_attend(p.p, out[:n], lse[:, :n], True)


@pytest.mark.parametrize("new", [1, 200])
def test_cache_beyond_32_bit_offsets(pkg, new):
    """Pages whose byte offsets pass 2^32 in the codes and 2^31 in both kinds of scales."""
    p = R4.make([new + 40], [new], 4, 2, 128, 64, seed=16)
    high = (1 << 32) // (64 * 2 * 64) + 3
    big = []
    for x in p.all():
        y = torch.empty((high + x.shape[0],) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        y[high:] = x
        big.append(y)
    kc, vc, ks, vs, kb, vb = big
    table = p.p.table + high
    kw = dict(k_scale=ks, v_scale=vs, k_block=kb, v_block=vb)
    want = R4.append(p)
    pkg.cache_append(p.p.k_new, p.p.v_new, kc, vc, table, p.p.seqlens, **kw)
    R4.same([x[high:] for x in big], want)
    for x, y in zip(p.all(), want):
        x.copy_(y)
    p.refresh()
    o, lse = pkg.paged_forward(p.p.q, kc, vc, table, p.p.seqlens, **kw)
    pkg.check()
    R.check_attend(p.p, o, lse, True)
    cu = torch.tensor([0, new + 40], dtype=torch.int32, device="cuda")
    k, v = pkg.cache_read(kc, vc, table, cu, total_k=new + 40, **kw)
    assert torch.equal(k, R.gather(p.p, 0)[0].to(torch.bfloat16)) and torch.equal(v, R.gather(p.p, 0)[1].to(torch.bfloat16))


# ---------------------------------------------------------------- what only the device sees
@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("what", ["page_high", "page_negative", "length_high", "length_negative", "offsets"])
def test_bad_device_values_are_reported(pkg, what, new):
    packed = what == "offsets"
    p = R4.make([200, 150], [new] * 2, 4, 2, 64, 16, packed=packed, seed=17)
    table, seqlens, cu = p.p.table.clone(), p.p.seqlens.clone(), p.p.cu_q
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
    before = [x.clone() for x in p.all()]
    o, lse = pkg.paged_forward(p.p.q, p.k_cache, p.v_cache, table, seqlens, cu_seqlens_q=cu,
                               max_seqlen_q=new if packed else None, **p.scales)
    G._bad(pkg, p)
    (ro, rl, ra) = R.attend(p.p, True)[0]
    got = o[:new] if packed else o[0]
    assert ((got.double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 1e-6).all()
    if what != "offsets":
        if what.startswith("page"):
            table[1] = -1 if what == "page_negative" else p.k_cache.shape[0]
        pkg.cache_append(p.p.k_new, p.p.v_new, p.k_cache, p.v_cache, table, seqlens, **p.scales)
        G._bad(pkg, p)
        pages = p.p.table[1, :10].long()
        for x, y in zip(p.all(), before):
            assert torch.equal(R.bits(x[pages]), R.bits(y[pages]))


# ---------------------------------------------------------------- as they are used
def test_prompt_chunks_then_steps_match_contiguous_attention(pkg):
    """Two prompts enter the cache in chunks, tokens follow one by one, keys and queries
    turned on the way; every output matches forward()'s causal attention over what
    cache_read returns."""
    hq, hkv, dim, page, n = 8, 2, 128, 32, 333
    g = torch.Generator(device="cuda").manual_seed(20)
    q, k, v = (torch.randn(2, n, h, dim, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    pages = 2 * (-(-n // page))
    kc, vc = (torch.zeros(pages, page, hkv, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = {x + "_scale": torch.zeros(pages, hkv, page, device="cuda") for x in "kv"}
    sc |= {x + "_block": torch.zeros(pages, hkv, page, dim // 16, device="cuda").to(R.E4M3) for x in "kv"}
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(2, -1)
    turn = pkg.rotary_table(pkg.rotary_frequencies(64), n)
    outs, lses, at = [], [], 0
    for step in (150, 150, 17, 9, 1, 1, 1, 1, 1, 1, 1):
        lens = torch.full((2,), at + step, dtype=torch.int32, device="cuda")
        new = slice(at, at + step)
        q2 = pkg.cache_append(k[:, new], v[:, new], kc, vc, table, lens, rotary_table=turn, interleaved=True, q=q[:, new], **sc)
        o, lse = pkg.paged_forward(q2, kc, vc, table, lens, **sc)
        outs.append(o)
        lses.append(lse)
        at += step
    assert at == n
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    kr, vr = pkg.cache_read(kc, vc, table, cu, total_k=2 * n, **sc)
    kr, vr = kr.view(2, n, hkv, dim), vr.view(2, n, hkv, dim)
    q2, k2 = pkg.rotary(q, k, turn, interleaved=True)
    o_ref, lse_ref = pkg.forward(q2, kr, vr, causal=True)
    pkg.check()
    # keys come back within 4 bits of what went in: a step is at most a quarter of a block's largest value
    assert (kr.double() - k2.double()).norm() <= 0.15 * k2.double().norm()
    o, lse = torch.cat(outs, 1), torch.cat(lses, 2)
    _, _, absv = zip(*G._contiguous(q2, kr, vr))
    bound = 2 * (2.0 ** -8 * o_ref.double().abs() + (2.0 ** -8 + 2.0 ** -14) * torch.stack(absv) + 1e-6)
    assert bool(((o.double() - o_ref.double()).abs() <= bound).all())
    assert (lse - lse_ref).abs().max().item() <= 1e-4


@pytest.mark.parametrize("new,hq", [(1, 8), (40, 8)])
def test_captured_step_follows_the_lengths(pkg, new, hq):
    """Rotation, append and attention captured, replayed with other lengths, two graphs
    at once on two streams."""
    graphs = []
    turn = R4.angles(new + 900, 128)
    for seed in (21, 22):
        p = R4.make([new + 900, new + 500], [new] * 2, hq, 2, 128, 32, seed=seed, poison=False)
        out, lse, q2 = torch.empty_like(p.p.q), torch.empty(2, hq, new, device="cuda"), torch.empty_like(p.p.q)
        graph = torch.cuda.CUDAGraph()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            pkg.cache_append(p.p.k_new, p.p.v_new, *p.cache, rotary_table=turn, q=p.p.q, out_q=q2, **p.scales)
            pkg.paged_forward(q2, *p.cache, out=out, lse=lse, **p.scales)
        graphs.append((p, out, lse, q2, graph))
    streams = [torch.cuda.Stream() for _ in graphs]
    for lens in ([new + 900, new + 500], [new, new + 333], [new + 17, new + 400]):
        for p, *_ in graphs:
            p.p.seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
            p.p.lens_k[:] = lens
        torch.cuda.synchronize()
        for _ in range(5):
            for s, (*_, graph) in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for p, out, lse, q2, _ in graphs:
            o, l = pkg.paged_forward(q2, *p.cache, **p.scales)
            pkg.check()
            assert torch.equal(R.bits(o), R.bits(out)) and torch.equal(R.bits(l), R.bits(lse))
            at = (p.p.seqlens[:, None] - new + torch.arange(new, device="cuda")).flatten()
            T.check_turned(q2.flatten(0, 1), p.p.q.flatten(0, 1), turn, at)
            p.refresh()
            q, p.p.q = p.p.q, q2
            R.check_attend(p.p, out, lse, True)
            p.p.q = q


def test_two_streams_at_once(pkg):
    ps = [R4.make([3000, 2000], [n] * 2, 8, 2, 128, 64, seed=s) for n, s in ((1, 23), (1, 24), (40, 25))]
    want = [_attend(pkg, p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(10):
        got = [_attend(pkg, p, stream=s) for s, p in zip(streams, ps)]
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(R.bits(o), R.bits(wo)) and torch.equal(R.bits(l), R.bits(wl))
    for s in streams:
        pkg.check(stream=s)


def test_own_workspace(pkg):
    p = R4.make([1300, 40], [1, 1], 8, 2, 64, 16, seed=26)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    turn = R4.angles(1300, 64)
    q2 = pkg.cache_append(p.p.k_new, p.p.v_new, *p.cache, rotary_table=turn, q=p.p.q, workspace=ws, **p.scales)
    p.refresh()
    p.p.q = q2
    o, lse = _attend(pkg, p, workspace=ws)
    pkg.check(workspace=ws)
    R.check_attend(p.p, o, lse, True)
    with pytest.raises(pkg.AttnError, match="workspace"):
        _attend(pkg, p, workspace=ws[:256])


def test_no_rows(pkg):
    p = R4.make([20], [1], 2, 2, 64, 16, seed=27)
    o, lse = pkg.paged_forward(p.p.q[:, :0], *p.cache, **p.scales)
    assert o.shape == (1, 0, 2, 64) and lse.shape == (1, 2, 0)
    turn = R4.angles(20, 64)
    q = pkg.cache_append(p.p.k_new[:0], p.p.v_new[:0], p.k_cache, p.v_cache, p.p.table[:0], p.p.seqlens[:0],
                         rotary_table=turn, q=p.p.q[:0], **p.scales)
    assert q.shape == (0, 1, 2, 64)
    k, v = pkg.cache_read(p.k_cache, p.v_cache, p.p.table, torch.zeros(2, dtype=torch.int32, device="cuda"), total_k=0, **p.scales)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    pkg.check()


def test_rows_on_16_byte_boundaries_only(pkg):
    """New rows, outputs and q whose strides are odd multiples of 16 bytes."""
    p = R4.make([90, 40], [30, 30], 4, 2, 64, 16, seed=30)
    wide = torch.full((2, 30, 2, 3 * 72 + 8), 3.0, dtype=torch.bfloat16, device="cuda")[..., 8:]
    k, v = wide[..., :64], wide[..., 72:136]
    k.copy_(p.p.k_new)
    v.copy_(p.p.v_new)
    want = R4.append(p)
    pkg.cache_append(k, v, *p.cache, **p.scales)
    R4.same(p.all(), want)
    p.refresh()
    cu = torch.tensor([0, 90, 130], dtype=torch.int32, device="cuda")
    out = torch.full((130, 2, 152), 5.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_read(p.k_cache, p.v_cache, p.p.table, cu, out_k=out[..., 8:72], out_v=out[..., 80:144], **p.scales)
    both = [torch.cat(x).to(torch.bfloat16) for x in zip(*(R.gather(p.p, b) for b in range(2)))]
    assert torch.equal(out[..., 8:72], both[0]) and torch.equal(out[..., 80:144], both[1])
    assert bool((out[..., :8] == 5.0).all()) and bool((out[..., 72:80] == 5.0).all()) and bool((out[..., 144:] == 5.0).all())
    pkg.check()
