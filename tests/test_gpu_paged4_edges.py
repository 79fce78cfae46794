"""Edges of the 4-bit paged cache on the GPU: weights of a sequence's last keys,
device waits that run out."""
import ctypes

import pytest
import torch

import paged4_reference as R4
import paged_reference as R
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
