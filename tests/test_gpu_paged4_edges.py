"""Edges of the 4-bit paged cache on the GPU: weights of a sequence's last keys,
device waits that run out."""
import ctypes

import pytest
import torch

import paged4_reference as R4
import paged_reference as R
import test_gpu_paged as G
import test_paged4_cpu as C4
import test_paged_cpu as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


def _attend(pkg, p, causal=True, **kw):
    if p.p.cu_q is not None:
        kw = dict(dict(cu_seqlens_q=p.p.cu_q, max_seqlen_q=max(p.p.lens_q)), **kw)
    return pkg.paged_forward(p.p.q, *p.cache, causal=causal, **p.scales, **kw)


@pytest.mark.parametrize("dim,page,group,new", [(128, 16, 4, 1), (128, 64, 4, 3), (64, 32, 8, 4), (64, 16, 16, 1), (128, 32, 1, 2)])
def test_weights_of_the_last_keys_keep_eleven_bits(pkg, dim, page, group, new):
    """Up to 64 rows have f16 weights to a sequence's very end, where slots behind it
    are passed over: 2^-11 of sum w |v| (half of f16's step), in place of bf16's 2^-8.
    (Weights are scaled to 2^-4 .. 2^8 of 2^7, so that f16's spacing near zero, 2^-24, is
    2^-27 of the largest weight at most, and 1000 keys' less than 2^-17; exponentials and
    sums in fp32 add less than 2^-14.) O is rounded once, 2^-8 of it."""
    lens_k = [2, 5, 31, 33, 64, 97, 200, 777]
    p = R4.make(lens_k, [min(n, new) for n in lens_k], 2 * group, 2, dim, page, packed=True, seed=51)
    for causal in (True, False):
        o, _ = _attend(pkg, p, causal)
        pkg.check()
        at = 0
        for ro, _, ra in R.attend(p.p, causal):
            got = o[at:at + ro.shape[0]].double()
            at += ro.shape[0]
            bound = 2.0 ** -8 * ro.abs() + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -17) * ra + 1e-6
            worst = ((got - ro).abs() / bound).max().item()
            assert worst <= 1.0, f"{worst:.3f} of the bound"


@pytest.mark.parametrize("lens_k,new,hq,hkv,dim,page,cut", [
    ([9000, 5000], 1, 8, 2, 128, 64, True), ([9000, 5000], 1, 4, 1, 64, 16, True), ([7000], 4, 8, 2, 128, 16, True),
    ([7000, 30], 7, 8, 2, 128, 64, True), ([60, 9], 1, 4, 1, 128, 32, False)])
def test_tile_that_never_comes(pkg, lens_k, new, hq, hkv, dim, page, cut):
    """The first CTA's first tile of keys is withheld: its waits run out, the call is
    reported, and the workspace, whose counters wait for a part that has not come, serves
    the next call, whose result has the bits of one with a workspace of its own."""
    p = R4.make(lens_k, [new] * len(lens_k), hq, hkv, dim, page, seed=52)
    o, lse = _attend(pkg, p)
    pkg.check()
    R.check_attend(p.p, o, lse, True)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    out, out_lse = torch.empty_like(o), torch.empty_like(lse)
    L = C4._library(pkg)
    L.attn_paged_fwd_withheld.argtypes = [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_void_p]
    pages, _, _, half = p.k_cache.shape
    params = C.PAGED.pack(
        p.k_cache.data_ptr(), p.v_cache.data_ptr(), p.k_scale.data_ptr(), p.v_scale.data_ptr(), p.p.table.data_ptr(),
        *p.k_cache.stride()[:3], *p.v_cache.stride()[:3], p.p.table.stride(0), 2, pages, page, p.p.table.shape[1], hkv, dim,
        len(lens_k), p.p.q.data_ptr(), out.data_ptr(), out_lse.data_ptr(), p.p.seqlens.data_ptr(), 0, ws.data_ptr(),
        ws.numel(), *p.p.q.stride()[:3], *out.stride()[:3], new, p.p.table.shape[1] * page, 0, hq, 1, dim ** -0.5)
    blocks = C4.BLOCKS.pack(p.k_block.data_ptr(), p.v_block.data_ptr())
    for _ in range(2):
        stream = torch.cuda.current_stream()
        assert L.attn_paged_fwd_withheld(params, blocks, ctypes.c_void_p(stream.cuda_stream)) == 0
        torch.cuda.synchronize()
        assert bool(ws[256:8192].any()) == cut
        with pytest.raises(pkg.AttnError) as e:
            pkg.check(workspace=ws)
        assert e.value.status == 4 and "block 0," in str(e.value)
        assert not bool(ws[:8192].any())
        got = _attend(pkg, p, workspace=ws)
        pkg.check(workspace=ws)
        assert torch.equal(R.bits(got[0]), R.bits(o)) and torch.equal(R.bits(got[1]), R.bits(lse))
        assert not bool(ws[:8192].any())


# ---------------------------------------------------------------- block scales over their range
def _any_blocks(p, seed):
    """A quarter of the held vectors get block scales of any finite code: zeros, subnormals,
    small ones, negative ones. Values stay below 2^-10 * 6 * 448 < 3, so scores stay ordinary."""
    g = torch.Generator().manual_seed(seed)
    for block, scale in ((p.k_block, p.k_scale), (p.v_block, p.v_scale)):
        pick = ~torch.isnan(scale) & (torch.rand(scale.shape, generator=g) < 0.25).cuda()
        codes = torch.randint(0, 256, block.shape, generator=g).to(torch.uint8).cuda()
        codes = torch.where((codes & 0x7f) == 0x7f, 1, codes)   # not NaN: the smallest subnormal instead
        block.view(torch.uint8)[pick] = codes[pick]
        scale[pick] = 2.0 ** -10
    p.refresh()
    return p


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name", list(G.ATTEND))
def test_attend_any_block_scales(pkg, name, causal):
    lens_k, lens_q, hq, hkv, dim, page, packed, head_major = G.ATTEND[name]
    p = _any_blocks(R4.make(lens_k, lens_q, hq, hkv, dim, page, packed=packed, head_major=head_major, seed=61), 62)
    o, lse = _attend(pkg, p, causal)
    pkg.check()
    R.check_attend(p.p, o, lse, causal)


@pytest.mark.parametrize("lens_k,lens_q,hq,hkv,dim,page", [
    ([4100, 1300, 2600, 1029], [200, 900, 1, 130], 8, 2, 128, 32), ([1500, 0, 1100, 3], [40, 5, 0, 100], 32, 1, 64, 16)])
def test_chunks_any_block_scales(pkg, lens_k, lens_q, hq, hkv, dim, page):
    """Over the copy, and 32 rows at a time where a bound on the lengths asks for too large a one."""
    p = _any_blocks(R4.make(lens_k, lens_q, hq, hkv, dim, page, packed=True, seed=63), 64)
    wide = torch.full((len(lens_k), (1 << 23) // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :p.p.table.shape[1]] = p.p.table
    for table in (p.p.table, wide):
        o, lse = pkg.paged_forward(p.p.q, p.k_cache, p.v_cache, table, p.p.seqlens, cu_seqlens_q=p.p.cu_q,
                                   max_seqlen_q=max(lens_q), **p.scales)
        pkg.check()
        R.check_attend(p.p, o, lse, True)


@pytest.mark.parametrize("dim", [64, 128])
def test_read_any_block_scales(pkg, dim):
    """Every code under every finite block scale, and random ones."""
    p = _any_blocks(R4.make([700, 33], [0, 0], 3, 3, dim, 16, packed=True, seed=65), 66)
    slots = [(int(p.p.table[0, j // 16]), j % 16) for j in range(256)]
    for j, (page, slot) in enumerate(slots):   # scale j, all sixteen codes in each block
        p.k_block.view(torch.uint8)[page, :, slot] = j if j & 0x7f != 0x7f else 1
        p.k_scale[page, :, slot] = 2.0 ** -10
        p.k_cache[page, slot] = torch.tensor([c * 0x22 + 0x10 for c in range(8)], device="cuda").to(torch.uint8).repeat(dim // 16)
    p.refresh()
    k, v = pkg.cache_read(*p.cache[:3], torch.tensor([0, 700, 733], dtype=torch.int32, device="cuda"), total_k=733, **p.scales)
    pkg.check()
    for got, want in zip((k, v), zip(*(R.gather(p.p, b) for b in range(2)))):
        assert torch.equal(R.bits(got), R.bits(torch.cat(want).to(torch.bfloat16)))


# ---------------------------------------------------------------- far pages
@pytest.mark.parametrize("new", [1, 200])
def test_scales_beyond_32_bit_offsets(pkg, new):
    """Pages behind 2^30 (token, head) vectors: both kinds of scales start 2^32 bytes
    further on, the block scales with as many entries, and the codes 2^35 bytes."""
    lens, page, hkv, dim = [new + 40], 64, 2, 64
    high = (1 << 30) // (page * hkv)
    need = high * page * hkv * 2 * (dim // 2 + 4 + dim // 16)
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("86 GB of memory needed")
    p = R4.make(lens, [new], 4, hkv, dim, page, seed=67)
    big = []
    for x in p.all():
        y = torch.empty((high + x.shape[0],) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        y[high:] = x
        big.append(y)
    kc, vc, ks, vs, kb, vb = big
    assert ks[high:].data_ptr() - ks.data_ptr() == 1 << 32 and kb[high:].data_ptr() - kb.data_ptr() == 1 << 32
    table = p.p.table + high
    kw = dict(k_scale=ks, v_scale=vs, k_block=kb, v_block=vb)
    turn = R4.angles(lens[0], 32)
    want = R4.append(p, turn)
    q = pkg.cache_append(p.p.k_new, p.p.v_new, kc, vc, table, p.p.seqlens, rotary_table=turn, q=p.p.q, **kw)
    pkg.check()
    R4.same([x[high:] for x in big], want)
    for x, y in zip(p.all(), want):
        x.copy_(y)
    p.refresh()
    p.p.q = q
    o, lse = pkg.paged_forward(q, kc, vc, table, p.p.seqlens, **kw)
    k, v = pkg.cache_read(kc, vc, table, torch.tensor([0, lens[0]], dtype=torch.int32, device="cuda"), total_k=lens[0], **kw)
    pkg.check()
    R.check_attend(p.p, o, lse, True)
    assert torch.equal(k, R.gather(p.p, 0)[0].to(torch.bfloat16)) and torch.equal(v, R.gather(p.p, 0)[1].to(torch.bfloat16))
    del big, kc, vc, ks, vs, kb, vb, kw, x, y
    torch.cuda.empty_cache()
