"""The 4-bit cache without a GPU: what the calls refuse, the struct layouts of the
calls with block scales, which form of the attention a call takes, and the test
reference against its own definitions."""
import ctypes
import math
import struct

import pytest
import torch

import __graft_entry__
import paged4_reference as R4
import paged_reference as R
import test_paged_cpu as C

BLOCKS, TURN = struct.Struct("@2P"), struct.Struct("@4P6q4i")


@pytest.fixture(scope="module")
def pkg():
    __graft_entry__.build()
    import attention_forward_sm100_gb300 as m
    return m


def _library(pkg):
    L = C._library(pkg)
    L.attn_cache_append_blocks.argtypes = [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_char_p, ctypes.c_void_p]
    for f in (L.attn_cache_read_blocks, L.attn_paged_fwd_blocks):
        f.argtypes = [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_void_p]
    L.attn_cache_blocks_params_size.restype = ctypes.c_size_t
    return L


FP4 = dict(dtype=2, k_scale=9 << 20, v_scale=10 << 20, k_stride=(1024, 64, 32), v_stride=(1024, 64, 32))
GOOD = BLOCKS.pack(11 << 20, 12 << 20)


def _append(cache, seqlen=1, cu=0, total=0):
    return C.APPEND.pack(*C._cache(**cache), 4 << 20, 5 << 20, 6 << 20, cu, 7 << 20, *(128, 128, 64) * 2, seqlen, total)


def _turn(**kw):
    d = dict(table=13 << 20, positions=0, q=14 << 20, q_out=15 << 20, q_stride=(256, 256, 64), out_stride=(256, 256, 64),
             heads=4, num_positions=99, rot=64, inter=0)
    d.update(kw)
    return TURN.pack(d["table"], d["positions"], d["q"], d["q_out"], *d["q_stride"], *d["out_stride"], d["heads"],
                     d["num_positions"], d["rot"], d["inter"])


def test_struct_layouts(pkg):
    L = _library(pkg)
    assert [L.attn_cache_blocks_params_size(i) for i in range(3)] == [BLOCKS.size, TURN.size, 0]


def test_library_refuses_block_scales(pkg):
    L = _library(pkg)
    read = C.READ.pack(*C._cache(**FP4), 4 << 20, 5 << 20, 6 << 20, 7 << 20, *(128, 64) * 2, 5)
    for blocks in (None, BLOCKS.pack(0, 12 << 20), BLOCKS.pack(11 << 20, 0), BLOCKS.pack((11 << 20) + 8, 12 << 20)):
        assert L.attn_cache_append_blocks(_append(FP4), blocks, None, None) == 1
        assert L.attn_cache_read_blocks(read, blocks, None) == 1
        assert L.attn_paged_fwd_blocks(C._paged(pkg, FP4), blocks, None) == 1
    assert L.attn_paged_fwd(C._paged(pkg, FP4), None) == 1      # the calls without block scales
    assert L.attn_cache_append(_append(FP4), None) == 1 and L.attn_cache_read(read, None) == 1
    for other in ({}, dict(dtype=1, k_scale=9 << 20, v_scale=10 << 20)):   # bf16 and e4m3 have none
        assert L.attn_paged_fwd_blocks(C._paged(pkg, other), GOOD, None) == 1
        assert L.attn_cache_append_blocks(_append(other), GOOD, None, None) == 1
    assert L.attn_paged_fwd_blocks(C._paged(pkg, dict(FP4, k_scale=0)), GOOD, None) == 1
    assert L.attn_paged_fwd_blocks(C._paged(pkg, dict(FP4, k_stride=(1024, 64, 24))), GOOD, None) == 1
    for f in (L.attn_cache_append_blocks, ):
        assert f(None, GOOD, None, None) == 1
    assert L.attn_cache_read_blocks(None, GOOD, None) == 1 and L.attn_paged_fwd_blocks(None, GOOD, None) == 1
    assert L.attn_fwd_last_error()


TURN_ERRORS = [(dict(table=0), 1), (dict(table=(13 << 20) + 8), 1), (dict(positions=2), 1), (dict(q=0), 1),
               (dict(q_out=(15 << 20) + 2), 1), (dict(q_stride=(256, 250, 64)), 1), (dict(out_stride=(256, 256, 60)), 1),
               (dict(heads=-1), 1), (dict(num_positions=-1), 1), (dict(heads=16385), 2), (dict(rot=0), 2), (dict(rot=8), 2),
               (dict(rot=24), 2), (dict(rot=128), 2)]


@pytest.mark.parametrize("change,status", TURN_ERRORS, ids=[str(c[0]) for c in TURN_ERRORS])
def test_library_refuses_rotations(pkg, change, status):
    L = _library(pkg)
    assert L.attn_cache_append_blocks(_append({}), None, _turn(**change), None) == status
    assert L.attn_cache_append_blocks(_append(FP4), GOOD, _turn(**change), None) == status


def test_no_rows(pkg):
    L = _library(pkg)
    assert L.attn_cache_append_blocks(_append(FP4, seqlen=0), GOOD, _turn(q=0), None) == 0


def _problem(**kw):
    return R4.make([40, 9], [2, 2], 4, 2, 64, 16, device="cpu", **kw)


REFUSALS = {
    "cpu": ({}, "CUDA"),
    "k_block": (dict(k_block=None), "k_block"),
    "v_block": (dict(v_block=None), "v_block"),
    "k_scale": (dict(k_scale=None), "k_scale"),
    "block_dtype": (dict(k_block=lambda p: p.k_block.float()), "k_block"),
    "block_shape": (dict(k_block=lambda p: p.k_block[1:]), "k_block"),
    "block_stride": (dict(v_block=lambda p: p.v_block.transpose(1, 2).contiguous().transpose(1, 2)), "v_block"),
    "v_dtype": (dict(v_cache=lambda p: p.v_cache.view(torch.int8)), "one dtype"),
    "cache_dtype": (dict(k_cache=lambda p: p.k_cache.view(torch.int8), v_cache=lambda p: p.v_cache.view(torch.int8)), "dtype"),
}


@pytest.mark.parametrize("name", list(REFUSALS))
def test_calls_refuse(pkg, name):
    change, match = REFUSALS[name]
    p = _problem()
    a = dict(k_cache=p.k_cache, v_cache=p.v_cache, block_table=p.p.table, seqlens_k=p.p.seqlens, **p.scales)
    a.update({k: (f(p) if callable(f) else f) for k, f in change.items()})
    with pytest.raises(ValueError, match=match):
        pkg.paged_forward(p.p.q, **a)
    with pytest.raises(ValueError, match=match):
        pkg.cache_append(p.p.k_new, p.p.v_new, **a)
    lens = a.pop("seqlens_k")
    with pytest.raises(ValueError, match=match):
        pkg.cache_read(cu_seqlens_k=torch.tensor([0, 40, 49], dtype=torch.int32), total_k=49, **a)
    assert lens is not None


def test_other_caches_take_no_block_scales(pkg):
    block = torch.zeros(1, dtype=R.E4M3)
    for fp8 in (False, True):
        p = R.make([40, 9], [2, 2], 4, 2, 64, 16, device="cpu", fp8=fp8)
        with pytest.raises(ValueError, match="only an e2m1 cache"):
            pkg.paged_forward(p.q, *p.cache, k_block=block, **p.scales)


@pytest.mark.parametrize("dim", [64, 128])
def test_more_than_64_rows_are_copied_where_the_copy_fits(pkg, dim):
    """Two sequences, two KV heads, eight query heads: 17 new tokens are 68 rows."""
    L = _library(pkg)

    def size(new, keys):
        cache = dict(dtype=2, k_scale=9 << 20, v_scale=10 << 20, dim=dim, k_stride=(16 * dim, dim, dim // 2),
                     v_stride=(16 * dim, dim, dim // 2), max_pages=-(-keys // 16))
        return L.attn_paged_workspace_bytes(C._paged(pkg, cache, q_stride=(8 * dim * new, 8 * dim, dim),
                                                     o_stride=(8 * dim * new, 8 * dim, dim), seqlen_q=new, seqlen_k=keys,
                                                     hq=8))

    def copy(keys):   # K and V as bf16
        return 2 * 2 * 2 * 2 * dim * keys

    assert size(16, 200) == 8192
    assert size(17, 2000) == 8192 + 256 + copy(2048)   # too few keys for a work list
    most = (1 << 30) // (16 * dim)
    assert size(17, most) > copy(most)
    assert size(17, most + 1) < 256 << 20


# ---------------------------------------------------------------- the reference itself
def test_reference_codes():
    """Every magnitude and border, by hand."""
    y = torch.tensor([0.0, -0.0, 0.25, 0.2500001, 0.5, 0.75, 0.7499999, 1.0, 1.25, 1.2500001, 1.5, 1.75, 1.7499999, 2.0, 2.5,
                      2.5000002, 3.0, 3.5, 3.4999998, 4.0, 5.0, 5.0000005, 6.0, 100.0, -0.6, -5.5])
    want = [0, 8, 0, 1, 1, 2, 1, 2, 2, 3, 3, 4, 3, 4, 4, 5, 5, 6, 5, 6, 6, 7, 7, 7, 9, 15]
    assert R4.e2m1_codes(y).tolist() == want
    nearest = torch.tensor(R4.MAGNITUDES)
    z = torch.rand(5000, generator=torch.Generator().manual_seed(1)) * 7
    best = (z[:, None] - nearest[None]).abs().argmin(1)
    assert torch.equal(R4.e2m1_codes(z).long(), best)


def test_reference_quantiser():
    x = torch.randn(40, 64, generator=torch.Generator().manual_seed(2)) * torch.logspace(-30, 30, 40)[:, None]
    x[0] = 0
    x[1, 16:] = 0
    codes, block, scale = R4.quantise(x)
    amax = x.abs().amax(-1).double()
    assert bool((torch.frexp(scale)[0] == 0.5).all()) and bool((amax <= 2688.0 * scale.double()).all())
    assert bool(((amax > 1344.0 * scale.double()) | (amax == 0)).all())
    back = R4.values(codes, block, scale)
    # a block's largest value is at most 2^-4 off by the scale's rounding and half a step
    # of 2 in 6 by the code's; any value at most that half step, 1, of the block's scale
    size = block.double()[..., None] * scale.double()[:, None, None]
    off = (back - x.double()).unflatten(-1, (-1, 16)).abs()
    assert bool((off <= size * (1 + 6 * 2.0 ** -4) + 2.0 ** -10 * 6 * scale.double()[:, None, None]).all())
    assert bool((back[0] == 0).all()) and bool((back[1, 16:] == 0).all())
    x = torch.zeros(3, 32)
    x[0, 3], x[1, 3], x[2, 20] = math.inf, math.nan, -math.inf
    x[:, 0] = 1.0
    back = R4.values(*R4.quantise(x))
    # 1 / 2^-11 = 2048 in a scale's units: its block's scale is 341.33 rounded to 352 of them
    assert back[0, 0] == 352 * 6 * 2.0 ** -11 and back[0, 3] == back[0, 0]
    assert bool(torch.isnan(back[1, :16]).all()) and bool((back[1, 16:] == 0).all())
    assert back[2, 0] == 352 * 6 * 2.0 ** -11 and bool((back[2, 16:] == 0).all())


def test_reference_rotation():
    x = torch.randn(5, 2, 32, generator=torch.Generator().manual_seed(3))
    at = torch.tensor([0, 3, 9, 1, 700])
    table = R4.angles(701, 24, device="cpu")
    for inter in (False, True):
        y = R4.rotated(x, table, at, inter, dtype=torch.float64)
        assert torch.equal(y[..., 24:], x[..., 24:].double())
        assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1), rtol=1e-6)   # the table's own rounding
        for i in (0, 5, 11):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 12)
            w = 700 * 10000.0 ** (-2 * i / 24)
            z = complex(x[4, 1, a], x[4, 1, b]) * complex(math.cos(w), math.sin(w))
            assert abs(y[4, 1, a] - z.real) < 1e-6 and abs(y[4, 1, b] - z.imag) < 1e-6
        assert torch.allclose(R4.rotated(y, table, at, inter, True, torch.float64), x.double(), atol=1e-6)
