"""Edges of rotary positions on the GPU: rows beside one another in one buffer, and on
boundaries of 16 and 32 bytes."""
import pytest
import torch

import paged4_reference as R4
import paged_reference as R
import test_gpu_rotary as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


def test_outputs_beside_their_inputs(pkg):
    """Outputs between the inputs' rows are written there; outputs across them are refused."""
    buf = T.randn(2, 9, 12, 64, seed=31)
    before = buf.clone()
    table = R4.angles(9, 64)
    at = torch.arange(9, device="cuda").repeat(2)
    q, k, oq, ok = buf[:, :, :4], buf[:, :, 4:6], buf[:, :, 6:10], buf[:, :, 10:]
    pkg.rotary(q, k, table, out_q=oq, out_k=ok)
    pkg.check()
    for x, o, part in ((q, oq, slice(0, 4)), (k, ok, slice(4, 6))):
        assert torch.equal(x, before[:, :, part])
        T.check_turned(o.flatten(0, 1), x.flatten(0, 1), table, at)
    for out_q, out_k in ((buf[:, :, 1:5], None), (buf[:, :, 2:6], None), (None, buf[:, :, 3:5]), (oq, buf[:, :, 8:10]),
                         (buf[:, :, ::2][:, :, :4], None)):
        with pytest.raises(pkg.AttnError, match="shares memory|in one place"):
            pkg.rotary(q, k, table, out_q=out_q, out_k=out_k)
    with pytest.raises(pkg.AttnError, match="in one place"):
        pkg.rotary(q, None, table, out_q=T.randn(1, 1, 1, 64).expand(2, 9, 4, 64))
    assert torch.equal(buf[:, :, :6], before[:, :, :6])


def test_append_refuses_queries_on_other_rows(pkg):
    p = R.make([40, 30], [3, 3], 4, 2, 64, 16, seed=32)
    fused = torch.cat([p.q, p.k_new, p.v_new], 2)
    q, k, v = fused[:, :, :4], fused[:, :, 4:6], fused[:, :, 6:]
    before = [x.clone() for x in (p.k_cache, p.v_cache, fused)]
    table = R4.angles(40, 64)
    for out in (fused[:, :, 1:5], fused[:, :, 2:6], fused[:, :, 4:8]):
        with pytest.raises(pkg.AttnError, match="shares memory"):
            pkg.cache_append(k, v, *p.cache, rotary_table=table, q=q, out_q=out)
    pkg.check()
    for x, y in zip((p.k_cache, p.v_cache, fused), before):
        assert torch.equal(R.bits(x), R.bits(y))
    assert pkg.cache_append(k, v, *p.cache, rotary_table=table, q=q, out_q=q) is q
    T.check_turned(q.flatten(0, 1), p.q.flatten(0, 1), table, torch.tensor([37, 38, 39, 27, 28, 29], device="cuda"))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_append_whatever_the_rows_boundaries(pkg, kind):
    """New rows and queries on 32-byte boundaries or odd multiples of 16 bytes, each by itself."""
    lens_k, new, hq, hkv, dim, rot = [70, 33], 21, 4, 2, 128, 64
    table = R4.angles(70, rot)
    at = torch.cat([torch.arange(k - new, k) for k in lens_k]).cuda()
    wants = None
    for wide_q, wide_kv in ((True, True), (False, True), (True, False), (False, False)):
        four = kind == "e2m1"
        m = R4 if four else R
        p = m.make(lens_k, [new] * 2, hq, hkv, dim, 32, seed=33, **({} if four else dict(fp8=kind == "e4m3")))
        x = p.p if four else p

        def placed(rows, wide):
            room = torch.zeros(rows.shape[:-1] + (dim + 16,), dtype=torch.bfloat16, device="cuda")
            at = 16 if wide else 8
            room[..., at:at + dim] = rows
            return room[..., at:at + dim]

        q, k, v = placed(x.q, wide_q), placed(x.k_new, wide_kv), placed(x.v_new, wide_kv)
        assert (q.data_ptr() % 32 == 0) == wide_q and (k.data_ptr() % 32 == 0) == wide_kv
        got = pkg.cache_append(k, v, *p.cache, rotary_table=table, q=q, **p.scales)
        pkg.check()
        T.check_turned(got.flatten(0, 1), x.q.flatten(0, 1), table, at)
        held = p.all() if four else [t for t in (p.k_cache, p.v_cache, p.k_scale, p.v_scale) if t is not None]
        held = [R.bits(t) for t in held]
        wants = wants or held
        assert all(torch.equal(a, b) for a, b in zip(held, wants))


QUANTISED = {
    # lens_k, lens_q, Hkv, D, page, packed, R, interleaved
    "step": ([5, 16, 300], [1] * 3, 8, 128, 16, False, 128, False),
    "chunk_interleaved": ([40, 100], [37, 37], 2, 128, 32, False, 64, True),
    "forty_eight": ([70, 9, 200, 33], [70, 1, 0, 30], 3, 64, 32, True, 48, False),
    "sixteen_interleaved": ([70, 9, 200, 33], [70, 1, 0, 30], 1, 64, 16, True, 16, True),
    "112": ([8, 0, 130, 4], [0, 0, 129, 0], 5, 128, 64, True, 112, False),
}


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
@pytest.mark.parametrize("name", list(QUANTISED))
def test_quantised_appends_with_positions_and_without_queries(pkg, name, kind):
    """Positions other than the cache's, and keys that are turned with no queries beside
    them, into caches whose kernels turn keys by themselves; bit for bit."""
    lens_k, lens_q, hkv, dim, page, packed, rot, inter = QUANTISED[name]
    table = R4.angles(500, rot)
    for given in (True, False):
        four = kind == "e2m1"
        p = R4.make(lens_k, lens_q, hkv, hkv, dim, page, packed=packed, seed=34) if four else \
            R.make(lens_k, lens_q, hkv, hkv, dim, page, fp8=True, packed=packed, seed=34)
        x = p.p if four else p
        rows = x.k_new.shape[:-2]
        pos = torch.randint(0, 500, rows, generator=torch.Generator().manual_seed(35)).to(torch.int32).cuda()
        at = pos.reshape(-1) if given else torch.cat([torch.arange(k - n, k) for k, n in zip(lens_k, lens_q)]).cuda()
        if four:
            want = R4.append(p, table, positions=at, interleaved=inter)
        else:
            new = p.k_new
            p.k_new = R4.rotated(new.reshape(-1, hkv, dim), table, at, inter).view(new.shape)
            want = R.append(p)
            p.k_new = new
        kw = dict(rotary_table=table, interleaved=inter, cu_seqlens_q=x.cu_q, **p.scales)
        if given:
            kw["positions"] = pos
        assert pkg.cache_append(x.k_new, x.v_new, *p.cache, **kw) is None
        pkg.check()
        if four:
            R4.same(p.all(), want)
        else:
            for g, w in zip((p.k_cache, p.v_cache, p.k_scale, p.v_scale), want):
                assert torch.equal(R.bits(g), R.bits(w))
