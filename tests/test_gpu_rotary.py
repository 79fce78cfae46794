"""Rotary positions on the GPU: bit for bit against fp32 products and sums, each
rounded, and within their roundings of the definition in 64 bits; rows that
belong to nobody; positions outside the table; and on the way into a cache."""
import types

import pytest
import torch

import paged4_reference as R4
import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def check_turned(got, x, table, at, interleaved=False, inverse=False):
    """Rows [T, H, D]."""
    want = R4.rotated(x, table, at, interleaved, inverse)
    assert torch.equal(R.bits(got), R.bits(want.to(torch.bfloat16)))
    # the definition: two products and a sum in fp32 (2^-24 each, relative to the
    # products' magnitudes, with the sum's at most theirs together), one rounding to bf16
    exact = R4.rotated(x, table, at, interleaved, inverse, torch.float64)
    size = R4.rotated(x.abs(), torch.cat([t.abs() * s for t, s in zip(table.chunk(2, 1), (1, -1))], 1), at, interleaved,
                      False, torch.float64)   # |x1 c| + |x2 s| in the first of a pair
    size2 = R4.rotated(x.abs(), table.abs(), at, interleaved, False, torch.float64)   # ... in the second
    bound = 2.0 ** -8 * exact.abs() + 2.0 ** -22 * torch.maximum(size, size2).abs()
    assert bool(((got.double() - exact).abs() <= bound).all())


CASES = {
    # B, S, Hq, Hk, D, R, interleaved
    "one_token": (1, 1, 1, 1, 64, 64, False),
    "step": (33, 1, 32, 8, 128, 128, False),
    "step_interleaved": (33, 1, 32, 8, 128, 128, True),
    "half_of_the_head": (2, 17, 5, 3, 128, 64, False),
    "half_interleaved": (2, 17, 5, 3, 128, 64, True),
    "quarter": (3, 9, 7, 1, 64, 16, False),
    "wide_head": (1, 40, 3, 2, 576, 64, False),
    "head_of_72": (2, 5, 4, 4, 72, 48, False),
    "value_by_value": (2, 13, 4, 2, 64, 20, False),
    "value_by_value_interleaved": (2, 13, 4, 2, 64, 20, True),
    "eight_interleaved": (2, 13, 4, 2, 40, 8, True),
    "two": (2, 3, 1, 1, 8, 2, False),
    "two_interleaved": (2, 3, 1, 1, 8, 2, True),
    "many_heads": (1, 6, 130, 71, 64, 64, False),
    "long": (2, 3000, 8, 2, 128, 128, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_rotary(pkg, name):
    b, s, hq, hk, d, rot, inter = CASES[name]
    q, k = randn(b, s, hq, d, seed=1), randn(b, s, hk, d, seed=2)
    table = R4.angles(s + 50, rot)
    at = torch.arange(s, device="cuda").repeat(b)
    kw = dict(interleaved=inter)
    q2, k2 = pkg.rotary(q, k, table, **kw)
    check_turned(q2.flatten(0, 1), q.flatten(0, 1), table, at, inter)
    check_turned(k2.flatten(0, 1), k.flatten(0, 1), table, at, inter)
    # any positions
    pos = torch.randint(0, s + 50, (b, s), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    q2, none = pkg.rotary(q, None, table, positions=pos, **kw)
    assert none is None
    check_turned(q2.flatten(0, 1), q.flatten(0, 1), table, pos.flatten(), inter)
    # behind what a sequence has already, turned back, in place
    lens = torch.tensor([s + (7 * i) % 50 for i in range(b)], dtype=torch.int32, device="cuda")
    at = (lens[:, None] - s + torch.arange(s, device="cuda")).flatten()
    want = q.clone()
    q2, k2 = pkg.rotary(q, k, table, seqlens=lens, inverse=True, out_q=q, **kw)
    assert q2 is q
    check_turned(q.flatten(0, 1), want.flatten(0, 1), table, at, inter, True)
    check_turned(k2.flatten(0, 1), k.flatten(0, 1), table, at, inter, True)
    pkg.check()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(pkg, inter):
    """The rotation's gradient is the rotation back: against autograd through the
    definition in 64 bits, and against differences along a direction."""
    q, grad = randn(2, 11, 3, 64, seed=4), randn(2, 11, 3, 64, seed=5)
    table = R4.angles(11, 32)
    at = torch.arange(11, device="cuda").repeat(2)
    got, _ = pkg.rotary(grad, None, table, interleaved=inter, inverse=True)
    x = q.double().flatten(0, 1).requires_grad_()
    y = R4.rotated(x, table, at, inter, dtype=torch.float64)
    y.backward(grad.double().flatten(0, 1))
    assert bool(((got.double().flatten(0, 1) - x.grad).abs() <= 2.0 ** -8 * x.grad.abs() + 2.0 ** -21 * 8).all())
    step = 1e-3 * torch.randn(x.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(6)).cuda()
    loss = lambda z: (R4.rotated(z, table, at, inter, dtype=torch.float64) * grad.double().flatten(0, 1)).sum()  # noqa: E731
    with torch.no_grad():
        diff = (loss(x + step) - loss(x - step)) / 2
        # a linear map: differences are exact but for the gradient's rounding to bf16
        assert abs(diff - (got.double().flatten(0, 1) * step).sum()) <= 2.0 ** -8 * (x.grad * step).abs().sum()


def test_packed_rows(pkg):
    """Ragged and empty sequences; rows of nobody in front and behind stay as they are."""
    lens = [5, 0, 1, 130, 64]
    cu = torch.tensor([3, 8, 8, 9, 139, 203], dtype=torch.int32, device="cuda")
    q, k = randn(210, 4, 64, seed=7), randn(210, 2, 64, seed=8)
    table = R4.angles(400, 64)
    for lens_k in (None, [9, 4, 1, 330, 64]):
        oq, ok = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        kw = {} if lens_k is None else dict(seqlens=torch.tensor(lens_k, dtype=torch.int32, device="cuda"))
        pkg.rotary(q, k, table, cu_seqlens=cu, out_q=oq, out_k=ok, **kw)
        pkg.check()
        at = torch.cat([torch.arange(n) + (0 if lens_k is None else m - n)
                        for n, m in zip(lens, lens_k or lens)]).cuda()
        for o, x in ((oq, q), (ok, k)):
            check_turned(o[3:203], x[3:203], table, at)
            assert bool((o[:3] == 7).all()) and bool((o[203:] == 7).all())
    pos = torch.arange(210, dtype=torch.int32, device="cuda")
    oq = torch.full_like(q, 7.0)
    pkg.rotary(q, None, table, positions=pos, cu_seqlens=cu, out_q=oq)
    check_turned(oq[3:203], q[3:203], table, pos[3:203])
    assert bool((oq[:3] == 7).all()) and bool((oq[203:] == 7).all())
    q2, _ = pkg.rotary(q, None, table)   # one sequence
    check_turned(q2, q, table, pos)
    many = [b % 3 for b in range(1500)]
    cu = torch.tensor([sum(many[:b]) for b in range(1501)], dtype=torch.int32, device="cuda")
    q = randn(sum(many), 1, 64, seed=9)
    q2, _ = pkg.rotary(q, None, table, cu_seqlens=cu)
    pkg.check()
    check_turned(q2, q, table, torch.tensor([i for n in many for i in range(n)], device="cuda"))


def test_views(pkg):
    """Heads inside a fused projection, one part of a wider head, odd multiples of 16 bytes."""
    fused = randn(3, 10, 9, 152, seed=10)
    before = fused.clone()
    table = R4.angles(10, 64)
    at = torch.arange(10, device="cuda").repeat(3)
    q, k = fused[:, :, 1:6, 72:136], fused[:, :, 7:, 8:72]
    q2, k2 = pkg.rotary(q, k, table, out_q=q, out_k=k)
    pkg.check()
    check_turned(q2.flatten(0, 1), before[:, :, 1:6, 72:136].flatten(0, 1), table, at)
    check_turned(k2.flatten(0, 1), before[:, :, 7:, 8:72].flatten(0, 1), table, at)
    q.copy_(before[:, :, 1:6, 72:136])
    k.copy_(before[:, :, 7:, 8:72])
    assert torch.equal(fused, before)
    shared = randn(1, 10, 1, 64, seed=11).expand(3, 10, 4, 64)   # broadcast inputs
    q2, _ = pkg.rotary(shared, None, table)
    check_turned(q2.flatten(0, 1), shared.flatten(0, 1), table, at)


def test_special_values(pkg):
    q = randn(1, 4, 2, 64, seed=12)
    q[0, 0, 0, 3] = float("inf")
    q[0, 1, 1, 40] = float("nan")
    q[0, 2] = torch.finfo(torch.bfloat16).max
    q[0, 3] = 2.0 ** -133
    table = R4.angles(4, 64)
    got, _ = pkg.rotary(q, None, table)
    want = R4.rotated(q[0], table, torch.arange(4, device="cuda")).to(torch.bfloat16)
    assert torch.equal(torch.isnan(got[0]), torch.isnan(want))
    assert torch.equal(got[0].nan_to_num(1.0, 2.0, 3.0), want.nan_to_num(1.0, 2.0, 3.0))


@pytest.mark.parametrize("what", ["position", "negative", "length", "offsets", "past"])
def test_bad_device_values_are_reported(pkg, what):
    q = randn(40, 2, 64, seed=13)
    table = R4.angles(30, 64)
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    kw = dict(cu_seqlens=cu)
    whole, gone = slice(0, 20), slice(20, 40)
    if what in ("position", "negative"):
        pos = torch.arange(20, dtype=torch.int32, device="cuda").repeat(2)
        pos[25] = 30 if what == "position" else -1
        kw["positions"] = pos
        gone = slice(25, 26)
    elif what == "length":
        kw["seqlens"] = torch.tensor([20, -2 ** 31], dtype=torch.int32, device="cuda")
    elif what == "offsets":
        kw["cu_seqlens"] = torch.tensor([0, 20, 10], dtype=torch.int32, device="cuda")
        whole, gone = slice(0, 0), slice(0, 40)
    else:
        kw["cu_seqlens"] = torch.tensor([0, 20, 41], dtype=torch.int32, device="cuda")
    pkg.rotary(q, None, table, out_q=out, **kw)
    with pytest.raises(pkg.AttnError, match="rotary"):
        pkg.check()
    pkg.check()
    assert bool((out[gone] == 7).all())
    check_turned(out[whole], q[whole], table, torch.arange(20, device="cuda")[whole])


def test_no_rows_and_workspace(pkg):
    table = R4.angles(4, 64)
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64), (2, 3, 0, 64)):
        q, k = pkg.rotary(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), None, table)
        assert q.shape == shape and k is None
    q = randn(2, 9, 2, 64, seed=14)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.rotary(q, None, table, workspace=ws)   # positions 4 to 8 are outside
    pkg.check()
    with pytest.raises(pkg.AttnError, match="rotary"):
        pkg.check(workspace=ws)


def test_graph_and_streams(pkg):
    """A captured rotation follows lengths on the device; calls on two streams."""
    q = randn(3, 1, 4, 128, seed=15)
    table = R4.angles(100, 128)
    lens = torch.tensor([5, 100, 1], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pkg.rotary(q, None, table, seqlens=lens, out_q=out, workspace=ws)
    for n in ([5, 100, 1], [77, 3, 50]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_turned(out[:, 0], q[:, 0], table, lens - 1)
    pkg.check(workspace=ws)
    lens.fill_(101)
    graph.replay()
    with pytest.raises(pkg.AttnError, match="rotary"):
        pkg.check(workspace=ws)
    lens.fill_(9)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [pkg.rotary(q, None, table, seqlens=lens, stream=s)[0] for s in streams]
    got.append(pkg.rotary(q, None, table, seqlens=lens, stream=streams[0].cuda_stream)[0])   # a bare handle
    torch.cuda.synchronize()
    for g in got:
        check_turned(g[:, 0], q[:, 0], table, lens - 1)
    other = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="another device"):
        pkg.rotary(q, None, table, stream=other)


def test_offsets_beyond_32_bits(pkg):
    """Rows whose element offsets pass 2^31, in views of 4.3 GB of memory."""
    n = 3
    big = torch.zeros((n - 1) * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((1, n, 2, 64), (8, 1 << 30, 64, 1))
    q.copy_(randn(1, n, 2, 64, seed=16))
    want = q.clone()
    table = R4.angles(n, 64)
    pkg.rotary(q, None, table, out_q=q)
    pkg.check()
    check_turned(q[0], want[0], table, torch.arange(n, device="cuda"))


# ---------------------------------------------------------------- on the way into a cache
APPEND = {
    # lens_k, lens_q, Hq, Hkv, D, page, packed, R, interleaved
    "one_token": ([1], [1], 1, 1, 64, 16, False, 64, False),
    "step": ([5, 16, 17, 300], [1] * 4, 32, 8, 128, 16, False, 128, False),
    "step_interleaved": ([5, 16, 17, 300], [1] * 4, 32, 8, 128, 16, False, 128, True),
    "chunk_half": ([40, 100], [37, 37], 4, 2, 128, 16, False, 64, False),
    "sixteen": ([40, 100], [37, 37], 3, 3, 64, 16, False, 16, False),
    "forty_eight": ([70, 9, 200, 33], [70, 1, 0, 30], 6, 3, 64, 32, True, 48, False),
    "forty_eight_interleaved": ([70, 9, 200, 33], [70, 1, 0, 30], 6, 3, 64, 32, True, 48, True),
    "112": ([8, 0, 130, 4], [0, 0, 129, 0], 5, 5, 128, 64, True, 112, False),
    "many_sequences": ([3 + b % 40 for b in range(300)], [1 + b % 3 for b in range(300)], 2, 1, 64, 16, True, 32, False),
    "long": ([3000, 2097], [2090, 2090], 8, 4, 128, 128, False, 128, False),
    # heads whose numbers have little in common, so that threads take other counts of q's than of the keys
    "groups": ([50, 9], [33, 9], 24, 3, 128, 16, True, 128, False),
    "groups_interleaved": ([50, 9], [33, 9], 32, 2, 64, 64, True, 16, True),
}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(APPEND))
def test_append_with_rotation(pkg, name, kind):
    """Bit for bit the append of keys that were turned in fp32 and never rounded before."""
    lens_k, lens_q, hq, hkv, dim, page, packed, rot, inter = APPEND[name]
    fp8 = kind == "e4m3"
    p = R.make(lens_k, lens_q, hq, hkv, dim, page, fp8=fp8, packed=packed, seed=41)
    table = R4.angles(max(lens_k), rot)
    at = torch.cat([torch.arange(k - q, k) for k, q in zip(lens_k, lens_q)]).cuda()
    flat = p.k_new.reshape(-1, hkv, dim)
    turned = R4.rotated(flat, table, at, inter)
    old = p.k_new
    p.k_new = (turned if fp8 else turned.to(torch.bfloat16)).view(old.shape)
    want = R.append(p)
    p.k_new = old
    q2 = pkg.cache_append(p.k_new, p.v_new, *p.cache, cu_seqlens_q=p.cu_q, rotary_table=table, interleaved=inter, q=p.q,
                          **p.scales)
    pkg.check()
    for g, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
        assert g is None or torch.equal(R.bits(g), R.bits(w))
    check_turned(q2.reshape(-1, hq, dim), p.q.reshape(-1, hq, dim), table, at, inter)
    # the rows of rotary() and its positions
    kw = dict(cu_seqlens=p.cu_q) if packed else {}
    q3, k3 = pkg.rotary(p.q, p.k_new, table, seqlens=p.seqlens, interleaved=inter, **kw)
    assert torch.equal(R.bits(q3), R.bits(q2))
    assert torch.equal(R.bits(k3.reshape(-1, hkv, dim)), R.bits(turned.to(torch.bfloat16)))


def test_append_with_positions_and_views(pkg):
    """Positions other than the cache's; q turned in place inside a fused projection; no q at all."""
    for lens_q, packed in (([6, 6], False), ([9, 3], True)):
        p = R.make([90, 40], lens_q, 4, 2, 64, 16, packed=packed, seed=42)
        rows = p.k_new.shape[:-2]
        n = sum(lens_q)
        pos = torch.randint(0, 500, rows, generator=torch.Generator().manual_seed(43)).to(torch.int32).cuda()
        table = R4.angles(500, 64)
        wide = torch.full(rows + (8, 72), 3.0, dtype=torch.bfloat16, device="cuda")
        q, k, v = wide[..., :4, 8:], wide[..., 4:6, 8:], wide[..., 6:, 8:]
        q.copy_(p.q)
        k.copy_(p.k_new)
        v.copy_(p.v_new)
        p.k_new = R4.rotated(p.k_new.reshape(n, 2, 64), table, pos.reshape(-1)).to(torch.bfloat16).view(p.k_new.shape)
        want = R.append(p)
        args = (k, v, *p.cache)
        kw = dict(cu_seqlens_q=p.cu_q, rotary_table=table, positions=pos)
        before = p.k_cache.clone()
        assert pkg.cache_append(*args, **kw) is None
        assert torch.equal(R.bits(p.k_cache), R.bits(want[0])) and torch.equal(R.bits(p.v_cache), R.bits(want[1]))
        p.k_cache.copy_(before)
        got = pkg.cache_append(*args, q=q, out_q=q, **kw)
        pkg.check()
        assert got is q and torch.equal(R.bits(p.k_cache), R.bits(want[0]))
        check_turned(q.reshape(n, 4, 64), p.q.reshape(n, 4, 64), table, pos.reshape(-1))
        assert bool((wide[..., :8] == 3.0).all()) and torch.equal(k.reshape(n, 2, 64), wide[..., 4:6, 8:].reshape(n, 2, 64))


@pytest.mark.parametrize("fp8", [False, True])
def test_append_at_bad_positions(pkg, fp8):
    """Tokens at positions outside the table, or without a page, are left out, their queries with them."""
    p = R.make([50, 33], [4, 4], 2, 2, 64, 16, fp8=fp8, seed=44)
    table = R4.angles(48, 64)   # positions 46 .. 49 and 29 .. 32: the first sequence's last two lie outside
    before = [x.clone() for x in (p.k_cache, p.v_cache)]
    out = torch.full_like(p.q, 7.0)
    tab = p.table.clone()
    tab[1, 2] = p.k_cache.shape[0]   # the second one's position 32
    pkg.cache_append(p.k_new, p.v_new, p.k_cache, p.v_cache, tab, p.seqlens, rotary_table=table, q=p.q, out_q=out, **p.scales)
    with pytest.raises(pkg.AttnError, match="rotary|paged cache"):
        pkg.check()
    assert bool((out[0, 2:] == 7).all()) and bool((out[1, 3:] == 7).all())
    check_turned(torch.cat([out[0, :2], out[1, :3]]), torch.cat([p.q[0, :2], p.q[1, :3]]), table,
                 torch.tensor([46, 47, 29, 30, 31], device="cuda"))
    last = int(p.table[0, 3])
    for x, b in zip((p.k_cache, p.v_cache), before):
        assert torch.equal(R.bits(x[last]), R.bits(b[last]))


def test_append_leaves_rows_of_nobody(pkg):
    p = R.make([20, 30], [5, 7], 4, 2, 64, 16, packed=True, seed=45)
    table = R4.angles(30, 64)
    n = 12
    pad = lambda x, m: torch.cat([x, torch.full((m,) + tuple(x.shape[1:]), 5.0, dtype=x.dtype, device="cuda")])  # noqa: E731
    out = torch.full((n + 4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pkg.cache_append(pad(p.k_new, 4), pad(p.v_new, 4), *p.cache, cu_seqlens_q=p.cu_q, rotary_table=table, q=pad(p.q, 4),
                     out_q=out)
    pkg.check()
    assert bool((out[n:] == 7).all())
    check_turned(out[:n], p.q, table, torch.cat([torch.arange(15, 20), torch.arange(23, 30)]).cuda())


def test_prompt_then_steps_match_contiguous_attention(pkg):
    """A model's use: chunks and single tokens rotated into the cache, their queries
    attended with; against forward() over queries and keys that rotary() turned."""
    hq, hkv, dim, page, n = 8, 2, 128, 32, 211
    q, k, v = (randn(2, n, h, dim, seed=s) for h, s in ((hq, 46), (hkv, 47), (hkv, 48)))
    table = pkg.rotary_table(pkg.rotary_frequencies(dim, factor=4.0, original_length=64), 256)
    kc, vc = (torch.zeros(2 * 7, page, hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.randperm(14, device="cuda").to(torch.int32).view(2, 7)
    outs, at = [], 0
    for step in (150, 57, 1, 1, 1, 1):
        lens = torch.full((2,), at + step, dtype=torch.int32, device="cuda")
        new = slice(at, at + step)
        turned = pkg.cache_append(k[:, new], v[:, new], kc, vc, bt, lens, rotary_table=table, q=q[:, new])
        outs.append(pkg.paged_forward(turned, kc, vc, bt, lens)[0])
        at += step
    q2, k2 = pkg.rotary(q, k, table)
    o, _ = pkg.forward(q2, k2, v, causal=True)
    pkg.check()
    p = R.Problem(k2, v, None, None, torch.arange(2)[:, None], None, [n] * 2, [n] * 2, None, q2, k2, v)
    _, _, absv = zip(*R.attend(p, True))
    bound = 2 * (2.0 ** -8 * o.double().abs() + (2.0 ** -8 + 2.0 ** -14) * torch.stack(absv) + 1e-6)
    assert bool(((torch.cat(outs, 1).double() - o.double()).abs() <= bound).all())


def test_table_of_far_positions(pkg):
    """Against Python's own arithmetic: angles of far positions keep their digits."""
    import math
    f = pkg.rotary_frequencies(64, base=500000.0)
    t = pkg.rotary_table(f, 3, first=1 << 20, amplitude=1.25)
    assert t.shape == (3, 64) and t.dtype == torch.float32 and t.is_cuda
    for i in (0, 1, 17, 31):
        for j in range(3):
            a = ((1 << 20) + j) * 500000.0 ** (-2 * i / 64)
            # the angle, up to 2^20, is a double: 2^-53 of it, and the frequency's power as much again
            assert abs(t[j, i].item() - 1.25 * math.cos(a)) <= 1.25 * 2.0 ** -24 + 2.0 ** -30
            assert abs(t[j, 32 + i].item() - 1.25 * math.sin(a)) <= 1.25 * 2.0 ** -24 + 2.0 ** -30
