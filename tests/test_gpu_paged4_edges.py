"""Edges of the 4-bit paged cache on the GPU: weights of a sequence's last keys."""
import pytest
import torch

import paged4_reference as R4
import paged_reference as R

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
