"""Edges of the 4-bit paged cache without a GPU: which calls have a tile to withhold."""
import ctypes

import test_paged4_cpu as C4
import test_paged_cpu as C
from test_paged4_cpu import pkg  # noqa: F401


def test_only_streamed_e2m1_calls_have_tiles_to_withhold(pkg):  # noqa: F811
    L = C4._library(pkg)
    L.attn_paged_fwd_withheld.argtypes = [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_void_p]
    many = dict(seqlen_q=70, q_stride=(70 * 128, 128, 64), o_stride=(70 * 128, 128, 64), ws_bytes=1 << 30)
    assert L.attn_paged_fwd_withheld(C._paged(pkg), None, None) == 2
    assert L.attn_paged_fwd_withheld(C._paged(pkg, dict(dtype=1, k_scale=9 << 20, v_scale=10 << 20)), None, None) == 2
    assert L.attn_paged_fwd_withheld(C._paged(pkg, C4.FP4, **many), C4.GOOD, None) == 2
    assert b"withhold" in L.attn_fwd_last_error()
    assert L.attn_paged_fwd_withheld(C._paged(pkg, C4.FP4), None, None) == 1      # no block scales
    assert L.attn_paged_fwd_withheld(None, C4.GOOD, None) == 1
