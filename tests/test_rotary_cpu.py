"""Rotary positions without a GPU: what the calls refuse, the header's exports and
struct layouts, frequencies and tables against closed forms."""
import ctypes
import math
import os
import re
import struct

import pytest
import torch

import __graft_entry__
import paged_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROTARY = struct.Struct("@9P12q10i")


@pytest.fixture(scope="module")
def pkg():
    __graft_entry__.build()
    import attention_forward_sm100_gb300 as m
    return m


def _library(pkg):
    L = ctypes.CDLL(pkg._binding.LIB_PATH)
    L.attn_rotary.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
    L.attn_rotary_params_size.restype = ctypes.c_size_t
    L.attn_fwd_last_error.restype = ctypes.c_char_p
    return L


def test_header(pkg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn_rotary.h")).read(), flags=re.S)
    names = re.findall(r"^\s*[A-Za-z_][\w \*]*?\b(attn_\w+)\s*\(", text, flags=re.M)
    L = _library(pkg)
    assert set(names) == {"attn_rotary", "attn_rotary_params_size"} and all(hasattr(L, n) for n in names)
    assert L.attn_rotary_params_size() == ROTARY.size


def _params(**kw):
    d = dict(q=1 << 20, k=2 << 20, q_out=3 << 20, k_out=4 << 20, table=5 << 20, positions=0, seqlens=0, cu=0, ws=6 << 20,
             q_stride=(512, 128, 64), k_stride=(512, 128, 64), q_out_stride=(512, 128, 64), k_out_stride=(512, 128, 64),
             batch=2, seqlen=4, total=0, heads_q=2, heads_k=2, dim=64, num_positions=9, rot=64, inter=0, inverse=0)
    d.update(kw)
    flat = []
    for v in d.values():
        flat += list(v) if isinstance(v, tuple) else [v]
    return ROTARY.pack(*flat)


ERRORS = [(dict(q=0), 1), (dict(k_out=(4 << 20) + 8), 1), (dict(table=0), 1), (dict(table=(5 << 20) + 4), 1),
          (dict(ws=0), 1), (dict(ws=(6 << 20) + 16), 1), (dict(positions=2), 1), (dict(cu=6, total=4), 1),
          (dict(seqlens=1), 1), (dict(batch=-1), 1), (dict(seqlen=-1), 1), (dict(heads_q=-1), 1), (dict(num_positions=-1), 1),
          (dict(heads_k=16385), 2), (dict(dim=60), 2), (dict(dim=0), 2), (dict(dim=4104), 2), (dict(rot=0), 1),
          (dict(rot=66), 1), (dict(rot=31), 1), (dict(q_stride=(512, 128, 60)), 1), (dict(k_out_stride=(512, -128, 64)), 1),
          (dict(batch=1 << 16, seqlen=1 << 16), 2)]


@pytest.mark.parametrize("change,status", ERRORS, ids=[str(c[0]) for c in ERRORS])
def test_library_refuses(pkg, change, status):
    L = _library(pkg)
    assert L.attn_rotary(_params(**change), None) == status and L.attn_fwd_last_error()
    assert L.attn_rotary(None, None) == 1


def test_library_takes_calls_without_rows(pkg):
    L = _library(pkg)
    for change in (dict(batch=0), dict(seqlen=0), dict(heads_q=0, heads_k=0), dict(cu=8, total=0)):
        assert L.attn_rotary(_params(q=0, table=0, ws=0, **change), None) == 0


BF = torch.bfloat16
REFUSALS = {
    "cpu": ({}, "CUDA"),
    "q_dtype": (dict(q=torch.zeros(2, 3, 4, 64)), "q must be bf16"),
    "q_dims": (dict(q=torch.zeros(4, 64, dtype=BF)), "q must be"),
    "packed_dims": (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), "q must be"),
    "k_rows": (dict(k=torch.zeros(2, 4, 4, 64, dtype=BF)), "k must have"),
    "k_depth": (dict(k=torch.zeros(2, 3, 4, 128, dtype=BF)), "k must have"),
    "stride": (dict(q=torch.zeros(2, 3, 64, 4, dtype=BF).transpose(2, 3)), "depth of q"),
    "table_dtype": (dict(table=torch.zeros(9, 64, dtype=torch.float64)), "table"),
    "table_dims": (dict(table=torch.zeros(9 * 64)), "table"),
    "table_stride": (dict(table=torch.zeros(64, 9).t()), "table"),
    "positions_shape": (dict(positions=torch.zeros(2, 4, dtype=torch.int32)), "positions"),
    "positions_dtype": (dict(positions=torch.zeros(2, 3, dtype=torch.int64)), "positions"),
    "seqlens": (dict(seqlens=torch.zeros(3, dtype=torch.int32)), "seqlens"),
    "both": (dict(seqlens=torch.zeros(2, dtype=torch.int32), positions=torch.zeros(2, 3, dtype=torch.int32)), "exclude"),
    "out_shape": (dict(out_q=torch.zeros(2, 3, 5, 64, dtype=BF)), "out_q"),
    "out_dtype": (dict(out_q=torch.zeros(2, 3, 4, 64)), "out_q"),
    "out_k_alone": (dict(out_k=torch.zeros(2, 3, 4, 64, dtype=BF)), "out_k"),
    "workspace": (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace"),
    "not_a_tensor": (dict(k=3), "k must be a tensor"),
}


@pytest.mark.parametrize("name", list(REFUSALS))
def test_rotary_refuses(pkg, name):
    change, match = REFUSALS[name]
    a = dict(q=torch.zeros(2, 3, 4, 64, dtype=BF), k=None, table=torch.zeros(9, 64))
    a.update(change)
    with pytest.raises(ValueError, match=match):
        pkg.rotary(**a)


APPEND_REFUSALS = {
    "cpu": ({}, "CUDA"),
    "positions_alone": (dict(rotary_table=None, q=None), "rotary_table"),
    "q_alone": (dict(rotary_table=None, positions=None), "rotary_table"),
    "interleaved_alone": (dict(rotary_table=None, positions=None, q=None, interleaved=True), "rotary_table"),
    "out_alone": (dict(q=None, out_q=torch.zeros(2, 2, 4, 64, dtype=BF)), "out_q"),
    "table": (dict(rotary_table=torch.zeros(40, 64, dtype=BF)), "rotary_table"),
    "positions": (dict(positions=torch.zeros(2, 3, dtype=torch.int32)), "positions"),
    "q_rows": (dict(q=torch.zeros(2, 3, 4, 64, dtype=BF)), "q must be"),
    "q_depth": (dict(q=torch.zeros(2, 2, 4, 128, dtype=BF)), "q must be"),
    "out_shape": (dict(out_q=torch.zeros(2, 2, 5, 64, dtype=BF)), "out_q"),
}


@pytest.mark.parametrize("name", list(APPEND_REFUSALS))
def test_append_refuses(pkg, name):
    change, match = APPEND_REFUSALS[name]
    p = R.make([40, 9], [2, 2], 4, 2, 64, 16, device="cpu")
    a = dict(rotary_table=torch.zeros(40, 64), positions=torch.zeros(2, 2, dtype=torch.int32), q=p.q)
    a.update(change)
    with pytest.raises(ValueError, match=match):
        pkg.cache_append(p.k_new, p.v_new, *p.cache, **a)


def test_frequencies(pkg):
    f = pkg.rotary_frequencies
    assert torch.equal(f(8), torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)) or \
        (f(8) - torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)).abs().max() < 1e-17
    assert (f(8, factor=4.0) * 4 - f(8)).abs().max() < 1e-17
    # by parts: over 64 positions a pair of frequency w turns 64 w / 2 pi times
    w = f(64, base=1e6)
    turns = 64 * w / (2 * math.pi)
    got = f(64, base=1e6, factor=8.0, original_length=64, slow_turns=0.5, fast_turns=4.0)
    assert bool((got[turns >= 4] == w[turns >= 4]).all()) and int((turns >= 4).sum()) > 2
    assert bool(((got * 8 - w)[turns <= 0.5].abs() < 1e-15).all()) and int((turns <= 0.5).sum()) > 2
    mid = (turns > 0.5) & (turns < 4)
    keep = torch.log2(turns[mid] / 0.5) / 3
    assert int(mid.sum()) > 2 and bool((got[mid] - w[mid] * (keep + (1 - keep) / 8)).abs().max() < 1e-15)
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, base=0), dict(dim=8, factor=0), dict(dim=8, original_length=0),
                dict(dim=8, original_length=9, slow_turns=2.0, fast_turns=1.0)):
        with pytest.raises(ValueError):
            f(**bad)


def test_table(pkg):
    t = pkg.rotary_table(pkg.rotary_frequencies(4, base=100.0), 5, first=1000, amplitude=0.5, device="cpu")
    assert t.shape == (5, 4) and t.dtype == torch.float32 and t.is_contiguous()
    for j in range(5):
        want = [0.5 * g((1000 + j) * w) for g in (math.cos, math.sin) for w in (1.0, 0.1)]
        assert max(abs(a - b) for a, b in zip(t[j].tolist(), want)) <= 2.0 ** -26   # half an ulp of at most 0.5
    assert pkg.rotary_table([1.0, 2.0], 0, device="cpu").shape == (0, 4)
    for bad in (([[1.0]], 3), ([1.0], -1)):
        with pytest.raises(ValueError):
            pkg.rotary_table(*bad, device="cpu")
