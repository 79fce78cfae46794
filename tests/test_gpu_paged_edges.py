"""Calls of the paged-cache operators at the edges of what they accept."""
import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import attention_forward_sm100_gb300 as m
    return m


# ---------------------------------------------------------------- tiny value scales
TINY = {
    "smallest": lambda n: torch.full((n,), 2.0 ** -126),
    "2^-121": lambda n: torch.full((n,), 2.0 ** -121),
    "2^-120": lambda n: torch.full((n,), 2.0 ** -120),
    "mixed": lambda n: torch.exp2(-126.0 + torch.arange(n) % 30),
    "then_ordinary": lambda n: torch.where(torch.arange(n) < 3 * n // 4, 2.0 ** -126, 2.0 ** -8),
    "after_ordinary": lambda n: torch.where(torch.arange(n) < n // 4, 2.0 ** -8, 2.0 ** -124),
}


@pytest.mark.parametrize("lens_k", [[1, 17], [1500, 700]], ids=["short", "long"])
@pytest.mark.parametrize("dim,hq,new", [(128, 4, 1), (64, 4, 1), (128, 4, 3), (64, 4, 3), (128, 20, 1), (64, 20, 1)])
@pytest.mark.parametrize("name", list(TINY))
def test_tiny_value_scales(pkg, name, dim, hq, new, lens_k):
    """Rows of up to 32 share the cached values: O within the roundings of the
    weights and of O, and half a step of bf16's subnormals (2^-134)."""
    p = R.make(lens_k, [new] * 2, hq, 1, dim, 16, fp8=True, seed=41)
    for b, n in enumerate(lens_k):
        s = TINY[name](n)
        at = torch.arange(n)
        p.v_scale[p.table[b].cpu()[at // 16].long(), 0, at % 16] = s.float().cuda()
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 2.0 ** -134
        assert ((o[b].double() - ro).abs() <= bound).all()
        seen = torch.isfinite(rl)
        assert torch.equal(torch.isfinite(lse[b]), seen)
        assert ((lse[b].double() - rl)[seen].abs() <= 5e-5).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_zero_vectors_with_the_smallest_scale(pkg, dim):
    """A quantiser that clamps its scales at the smallest normal float writes
    2^-126 for a vector of zeros: O = 0, whatever the length."""
    p = R.make([1, 40, 1000], [1] * 3, 4, 1, dim, 16, fp8=True, seed=42)
    held = ~torch.isnan(p.v_scale)
    p.v_scale[held] = 2.0 ** -126
    p.v_cache.view(torch.uint8)[held.transpose(1, 2)] = 0
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    assert bool((o == 0).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("size", [-118, -122, -126, -131])
def test_attend_to_what_append_wrote_for_tiny_values(pkg, size):
    p = R.make([5, 300], [5, 5], 4, 2, 128, 16, fp8=True, seed=43)
    p.v_new.copy_((p.v_new.double() * 2.0 ** size).to(torch.bfloat16))
    table, lens = p.table, p.seqlens
    pkg.cache_append(p.k_new, p.v_new, *p.cache, **p.scales)
    o, lse = pkg.paged_forward(p.q, *p.cache, **p.scales)
    pkg.check()
    for b, (ro, rl, ra) in enumerate(R.attend(p, True)):
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 2.0 ** -134
        assert ((o[b].double() - ro).abs() <= bound).all()
