"""The paged-cache operators without a GPU: arguments they refuse (by the
binding before anything is marshalled, by the library before anything is
enqueued), the exports of the header, the workspace sizes, and the test
reference against its own definitions."""
import ctypes
import math
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import __graft_entry__
import paged_reference as R

# attn_kv_cache, then the rest of each parameter struct (native alignment)
_CACHE = "5P7q7i4x"
APPEND = struct.Struct("@" + _CACHE + "5P6q2i")
READ = struct.Struct("@" + _CACHE + "4P4qi4x")
PAGED = struct.Struct("@" + _CACHE + "6PN6q5if")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pkg():
    __graft_entry__.build()
    import attention_forward_sm100_gb300 as m
    return m


def test_header_functions_are_exported(pkg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn_paged.h")).read(), flags=re.S)
    names = re.findall(r"^\s*[A-Za-z_][\w \*]*?\b(attn_\w+)\s*\(", text, flags=re.M)
    assert {"attn_cache_append", "attn_cache_read", "attn_paged_fwd", "attn_paged_workspace_bytes"} <= set(names)
    lib = ctypes.CDLL(pkg._binding.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def _library(pkg):
    L = ctypes.CDLL(pkg._binding.LIB_PATH)
    for f in (L.attn_cache_append, L.attn_cache_read, L.attn_paged_fwd):
        f.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
    L.attn_paged_workspace_bytes.argtypes = [ctypes.c_char_p]
    L.attn_paged_workspace_bytes.restype = ctypes.c_size_t
    L.attn_fwd_last_error.restype = ctypes.c_char_p
    return L


def test_struct_layouts(pkg):
    L = _library(pkg)
    L.attn_paged_params_size.restype = ctypes.c_size_t
    assert [L.attn_paged_params_size(i) for i in range(4)] == [APPEND.size, READ.size, PAGED.size, 0]


def test_header_compiles_as_c(pkg, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "paged.c", str(tmp_path / "paged")
    src.write_text("""
#include "attn_paged.h"
#include <stdio.h>
int main(void) {
  attn_paged_params p = {0};
  p.cache.page_size = 16;
  if (attn_paged_fwd(&p, 0) != ATTN_ERR_INVALID_ARG || attn_fwd_last_error()[0] == 0) return 1;
  if (attn_paged_workspace_bytes(&p) != ATTN_PAGED_ZEROED_BYTES) return 2;
  if (attn_cache_append(0, 0) != ATTN_ERR_INVALID_ARG || attn_cache_read(0, 0) != ATTN_ERR_INVALID_ARG) return 3;
  if (attn_paged_params_size(2) != sizeof(attn_paged_params)) return 4;
  puts("ok");
  return 0;
}
""")
    lib = os.path.join(ROOT, "attention_forward_sm100_gb300")
    cmd = [cc, "-std=c99", "-Wall", "-Wextra", "-Wno-missing-field-initializers", "-Wno-missing-braces", "-Werror",
           "-pedantic", "-I", os.path.join(ROOT, "include"), str(src), "-L", lib, "-lattn_fwd", "-Wl,-rpath," + lib, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok"


def _problem(**kw):
    return R.make([40, 9], [2, 2], 4, 2, 64, 16, device="cpu", **kw)


def _attend(pkg, p, **kw):
    a = dict(q=p.q, k_cache=p.k_cache, v_cache=p.v_cache, block_table=p.table, seqlens_k=p.seqlens)
    a.update(p.scales)
    a.update(kw)
    return pkg.paged_forward(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("block_table"), a.pop("seqlens_k"),
                             **a)


ATTEND_REFUSALS = {
    "cpu": ({}, "CUDA"),
    "q_dtype": (dict(q=lambda p: p.q.float()), "bf16"),
    "q_dims": (dict(q=lambda p: p.q[0]), "q must be"),
    "q_depth": (dict(q=lambda p: p.q[..., :32]), "depth"),
    "q_stride": (dict(q=lambda p: p.q.transpose(2, 3).contiguous().transpose(2, 3)), "contiguous"),
    "batch": (dict(q=lambda p: p.q[:1]), "batch"),
    "v_shape": (dict(v_cache=lambda p: p.v_cache[1:]), "one shape"),
    "v_dtype": (dict(v_cache=lambda p: p.v_cache.float()), "one dtype"),
    "cache_dtype": (dict(k_cache=lambda p: p.k_cache.float()), "dtype"),
    "table_dtype": (dict(block_table=lambda p: p.table.long()), "int32"),
    "table_dims": (dict(block_table=lambda p: p.table[0]), "block_table"),
    "table_stride": (dict(block_table=lambda p: p.table.t().contiguous().t()), "contiguous"),
    "lengths_dtype": (dict(seqlens_k=lambda p: p.seqlens.long()), "seqlens_k"),
    "lengths_shape": (dict(seqlens_k=lambda p: p.seqlens[:1]), "seqlens_k"),
    "scales_of_bf16": (dict(k_scale=lambda p: torch.ones(1)), "no scales"),
    "packed_without_bound": (dict(q=lambda p: p.q[0], cu_seqlens_q=lambda p: torch.tensor([0, 1, 2], dtype=torch.int32)),
                             "max_seqlen_q"),
    "offsets_shape": (dict(q=lambda p: p.q[0], max_seqlen_q=2,
                           cu_seqlens_q=lambda p: torch.tensor([0, 2], dtype=torch.int32)), "cu_seqlens_q"),
    "out_shape": (dict(out=lambda p: p.q[:, :1].clone()), "out"),
    "out_dtype": (dict(out=lambda p: p.q.float()), "out"),
    "lse_shape": (dict(lse=lambda p: torch.zeros(2, 2, 4)), "lse"),
    "negative_bound": (dict(max_seqlen_k=-1), "max_seqlen_k"),
    "workspace": (dict(workspace=lambda p: torch.zeros(16, dtype=torch.uint8)), "workspace"),
}


@pytest.mark.parametrize("name", list(ATTEND_REFUSALS))
def test_paged_forward_refuses(pkg, name):
    change, match = ATTEND_REFUSALS[name]
    p = _problem()
    with pytest.raises(ValueError, match=match):
        _attend(pkg, p, **{k: (f(p) if callable(f) else f) for k, f in change.items()})


def test_e4m3_cache_needs_its_scales(pkg):
    p = _problem(fp8=True)
    for kw in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=p.k_scale.half()), dict(v_scale=p.v_scale[1:]),
               dict(k_scale=p.k_scale.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError, match="_scale"):
            _attend(pkg, p, **kw)


def test_cache_append_refuses(pkg):
    p = _problem()
    ok = dict(k=p.k_new, v=p.v_new, k_cache=p.k_cache, v_cache=p.v_cache, block_table=p.table, seqlens_k=p.seqlens)

    def call(**kw):
        pkg.cache_append(**dict(ok, **kw))

    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    for kw, match in ((dict(), "CUDA"), (dict(k=p.k_new.float()), "bf16"), (dict(v=p.v_new[:, :1]), "one shape"),
                      (dict(k=p.k_new[..., :32], v=p.v_new[..., :32]), "heads and depth"),
                      (dict(k=p.k_new[:1], v=p.v_new[:1]), "batch"), (dict(cu_seqlens_q=cu), "cu_seqlens_q"),
                      (dict(k=p.k_new[0], v=p.v_new[0], cu_seqlens_q=cu[:2]), "cu_seqlens_q"),
                      (dict(seqlens_k=p.seqlens[:1]), "seqlens_k"), (dict(k_scale=torch.ones(1)), "no scales")):
        with pytest.raises(ValueError, match=match):
            call(**kw)


def test_cache_read_refuses(pkg):
    p = _problem()
    cu = torch.tensor([0, 40, 49], dtype=torch.int32)
    out = torch.zeros(49, 2, 64, dtype=torch.bfloat16)
    for kw, match in ((dict(total_k=49), "CUDA"), (dict(), "total_k"), (dict(out_k=out), "go together"),
                      (dict(out_k=out, out_v=out[:, :1]), "out_v"), (dict(out_k=out.float(), out_v=out), "out_k"),
                      (dict(total_k=48, out_k=out, out_v=out), "total_k"), (dict(total_k=-1), "total_k")):
        with pytest.raises(ValueError, match=match):
            pkg.cache_read(p.k_cache, p.v_cache, p.table, cu, **kw)
    with pytest.raises(ValueError, match="cu_seqlens_k"):
        pkg.cache_read(p.k_cache, p.v_cache, p.table, cu[:2], total_k=49)


# ---------------------------------------------------------------- the library's own checks
CACHE = dict(k=1 << 20, v=2 << 20, k_scale=0, v_scale=0, table=3 << 20, k_stride=(2048, 128, 64), v_stride=(2048, 128, 64),
             table_stride=8, dtype=0, num_pages=10, page_size=16, max_pages=8, heads=2, dim=64, batch=2)


def _cache(**kw):
    c = dict(CACHE, **kw)
    return (c["k"], c["v"], c["k_scale"], c["v_scale"], c["table"], *c["k_stride"], *c["v_stride"], c["table_stride"],
            c["dtype"], c["num_pages"], c["page_size"], c["max_pages"], c["heads"], c["dim"], c["batch"])


def _paged(pkg, cache=None, **kw):
    d = dict(q=4 << 20, o=5 << 20, lse=6 << 20, seqlens=7 << 20, cu=0, ws=8 << 20, ws_bytes=1 << 30,
             q_stride=(256, 256, 64), o_stride=(256, 256, 64), seqlen_q=1, seqlen_k=128, total_q=0, hq=4, causal=1,
             scale=0.125)
    d.update(kw)
    return PAGED.pack(*_cache(**(cache or {})), d["q"], d["o"], d["lse"], d["seqlens"], d["cu"], d["ws"],
                                 d["ws_bytes"], *d["q_stride"], *d["o_stride"], d["seqlen_q"], d["seqlen_k"],
                                 d["total_q"], d["hq"], d["causal"], d["scale"])


CACHE_ERRORS = [(dict(k=0), 1), (dict(v=(2 << 20) + 8), 1), (dict(table=0), 1), (dict(dtype=7), 1), (dict(num_pages=0), 1),
                (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=1 << 17), 2), (dict(dim=96), 2),
                (dict(dim=256), 2), (dict(heads=0), 1), (dict(batch=-1), 1), (dict(max_pages=-1), 1),
                (dict(max_pages=1 << 28), 2), (dict(k_stride=(2048, 129, 64)), 1), (dict(v_stride=(-2048, 128, 64)), 1),
                (dict(dtype=1), 1), (dict(table_stride=-1), 1)]


@pytest.mark.parametrize("change,status", CACHE_ERRORS, ids=[str(c[0]) for c in CACHE_ERRORS])
def test_library_refuses_caches(pkg, change, status):
    L = _library(pkg)
    if "heads" not in change:   # zero heads would also divide the query heads
        assert L.attn_paged_fwd(_paged(pkg, change), None) == status
    assert L.attn_cache_append(APPEND.pack(*_cache(**change), 4 << 20, 5 << 20, 6 << 20, 0, 7 << 20,
                                                      *(128, 128, 64) * 2, 1, 0), None) == status
    assert L.attn_cache_read(READ.pack(*_cache(**change), 4 << 20, 5 << 20, 6 << 20, 7 << 20,
                                                  *(128, 64) * 2, 5), None) == status
    assert L.attn_fwd_last_error()


PAGED_ERRORS = [(dict(q=0), 1), (dict(o=(5 << 20) + 2), 1), (dict(seqlens=0), 1), (dict(lse=(6 << 20) + 2), 1),
                (dict(ws=0), 1), (dict(ws=(8 << 20) + 16), 1), (dict(ws_bytes=100), 1), (dict(hq=3), 1), (dict(hq=0), 1),
                (dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(seqlen_k=129), 1), (dict(seqlen_q=-1), 1),
                (dict(q_stride=(256, 250, 64)), 1), (dict(o_stride=(256, 256, 60)), 1), (dict(cu=(9 << 20) + 2, total_q=2), 1)]


def test_library_refuses_too_many_new_tokens(pkg):
    L = _library(pkg)
    p = APPEND.pack(*_cache(batch=1 << 16), 4 << 20, 5 << 20, 6 << 20, 0, 7 << 20, *(128, 128, 64) * 2, 1 << 16, 0)
    assert L.attn_cache_append(p, None) == 2


@pytest.mark.parametrize("change,status", PAGED_ERRORS, ids=[str(c[0]) for c in PAGED_ERRORS])
def test_library_refuses_calls(pkg, change, status):
    L = _library(pkg)
    assert L.attn_paged_fwd(_paged(pkg, **change), None) == status
    assert L.attn_fwd_last_error()
    assert L.attn_paged_fwd(None, None) == 1 and L.attn_cache_append(None, None) == 1 and L.attn_cache_read(None, None) == 1


def test_workspace_depends_on_sizes_only(pkg):
    L = _library(pkg)
    size = L.attn_paged_workspace_bytes
    assert size(None) == 8192
    assert size(_paged(pkg, dict(dim=96))) == 8192
    short, long = dict(max_pages=8), dict(max_pages=4096)
    assert size(_paged(pkg, short)) == 8192                               # nothing is split
    n = size(_paged(pkg, long, seqlen_k=65536))
    assert n > 8192
    assert n == size(_paged(pkg, long, seqlen_k=65536, ws=0, ws_bytes=0))  # asked before there is one
    assert L.attn_paged_fwd(_paged(pkg, long, seqlen_k=65536, ws_bytes=n - 1), None) == 1


# ---------------------------------------------------------------- the reference itself
def test_reference_quantiser_matches_its_definition():
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0] = 0
    x[1] = 2.0 ** -133
    codes, scale = R.quantise(x)
    assert bool((torch.frexp(scale)[0] == 0.5).all())                       # powers of two
    amax = x.float().abs().amax(-1)
    assert bool((amax / scale <= 448).all())
    assert bool(((amax / (scale / 2) > 448) | (amax == 0) | (scale == 2.0 ** -126)).all())
    assert torch.equal(codes.float(), (x.float() / scale[:, None]).to(R.E4M3).float())


def test_reference_attention_matches_the_oracle():
    """A chunk that is the whole prompt is ordinary causal attention."""
    import numpy as np

    import oracle
    p = R.make([37], [37], 4, 2, 64, 16, device="cpu", seed=2)
    k, v = R.gather(p, 0)
    o, lse, _ = R.attend(p, True)[0]
    o_ref, lse_ref = oracle.attention(p.q.double().numpy(), k[None].numpy(), v[None].numpy(), causal=True, scale=64 ** -0.5)
    assert np.abs(o.numpy() - o_ref[0]).max() < 1e-12 and np.abs(lse.numpy() - lse_ref[0]).max() < 1e-12
