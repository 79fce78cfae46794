"""Which form of the paged attention a call takes, told by its workspace."""
import pytest

import __graft_entry__
import test_paged_cpu as C


@pytest.fixture(scope="module")
def pkg():
    __graft_entry__.build()
    import attention_forward_sm100_gb300 as m
    return m


@pytest.mark.parametrize("dim", [64, 128])
def test_long_e4m3_chunks_are_copied_where_the_copy_fits(pkg, dim):
    """From 512 rows to a KV head (four query heads: 128 new tokens) on, up to 1 GiB."""
    L = C._library(pkg)
    row = 2 * dim

    def size(new, keys):
        cache = dict(dtype=1, k_scale=9 << 20, v_scale=10 << 20, dim=dim, k_stride=(16 * row, row, dim),
                     v_stride=(16 * row, row, dim), max_pages=-(-keys // 16))
        return L.attn_paged_workspace_bytes(C._paged(pkg, cache, q_stride=(8 * dim * new, 8 * dim, dim),
                                                     o_stride=(8 * dim * new, 8 * dim, dim), seqlen_q=new, seqlen_k=keys,
                                                     hq=8))

    def copy(keys):   # K and V as bf16: two sequences, two KV heads
        return 2 * 2 * 2 * 2 * dim * keys

    # 2000 keys: too few for a work list, so the copy and its table of 16 pages each are all there is
    assert size(127, 2000) == 8192
    assert size(128, 2000) == 8192 + 256 + copy(2048)
    most = (1 << 30) // (16 * dim)
    assert size(128, most) - size(127, most) > copy(most) - (1 << 20)
    assert size(128, most + 1) < 256 << 20
