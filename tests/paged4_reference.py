"""Rotary positions and the 4-bit cache from their definitions, and problems to
run them on: torch, nothing of the library. Values of a cache are told as
doubles, so that paged_reference's attention runs on them as they are."""
import dataclasses
import math

import torch

import paged_reference as R

BLOCK = 16
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def angles(length, rot, base=10000.0, device="cuda"):
    """cosines and sines of positions, [length, rot]."""
    a = torch.arange(length, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


def rotated(x, table, at, interleaved=False, inverse=False, dtype=torch.float32):
    """Rows [T, H, D] turned by their positions ``at`` [T], in ``dtype`` (fp32: every product and sum rounded)."""
    rot = table.shape[1]
    x = x.to(dtype)
    c, s = table[at.long()].to(dtype)[:, None].chunk(2, -1)
    s = -s if inverse else s
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x1, x2 = x[..., first], x[..., second]
    y = x.clone()
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def power_at_least(amax, most):
    """The smallest power of two s >= 2^-126 with amax / s <= most (1 for amax = 0), as doubles."""
    amax = amax.double()
    s = torch.ones_like(amax)
    todo = amax > 0
    e = -126
    while bool(todo.any()):
        fits = todo & (amax <= most * 2.0 ** e)
        s[fits] = 2.0 ** e
        todo &= ~fits
        e += 1
    return s


def e2m1_codes(y):
    """Codes of fp32 quotients: the nearest magnitude, ties to the even code, beyond 6 the last one."""
    a = y.double().abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=y.device)
    for n, (lo, hi) in enumerate(zip(MAGNITUDES, MAGNITUDES[1:])):
        border = (lo + hi) / 2
        code += ((a >= border) if n % 2 else (a > border)).to(torch.uint8)
    return code + 8 * torch.signbit(y).to(torch.uint8)


def quantise(x):
    """(bytes [..., D / 2], block scales e4m3 [..., D / 16], scale [...]) of fp32 vectors."""
    x = x.float()
    fine = torch.where(torch.isfinite(x), x.abs(), 0.0)
    scale = power_at_least(fine.amax(-1), 2688.0)
    y = (x.double() / scale[..., None]).clamp(-2688, 2688).float().unflatten(-1, (-1, BLOCK))
    top = (fine.double() / scale[..., None]).float().unflatten(-1, (-1, BLOCK)).amax(-1)
    block = (top / 6.0).to(R.E4M3)
    size = block.float()[..., None]
    codes = torch.where(size == 0, 0, e2m1_codes(y / torch.where(size == 0, 1.0, size))).flatten(-2).to(torch.uint8)
    block = torch.where(torch.isnan(x).unflatten(-1, (-1, BLOCK)).any(-1), math.nan, block.float()).to(R.E4M3)
    return codes[..., 0::2] + 16 * codes[..., 1::2], block, scale.float()


def values(codes, block, scale):
    """Doubles [..., D] of bytes, block scales and scales."""
    line = torch.tensor(MAGNITUDES, dtype=torch.float64, device=codes.device)
    line = torch.cat([line, -line])
    x = torch.stack([line[(codes & 15).long()], line[(codes >> 4).long()]], -1).flatten(-2)
    x = x.unflatten(-1, (-1, BLOCK)) * block.double()[..., None]
    return x.flatten(-2) * scale.double()[..., None]


@dataclasses.dataclass
class Problem4:
    """A 4-bit cache (``args``: what the calls take) and the same as doubles (``p``, a paged_reference.Problem)."""
    p: R.Problem
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_block: torch.Tensor
    v_block: torch.Tensor

    @property
    def cache(self):
        return self.k_cache, self.v_cache, self.p.table, self.p.seqlens

    @property
    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale, k_block=self.k_block, v_block=self.v_block)

    def all(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.k_block, self.v_block

    def refresh(self):
        """The doubles again, after the cache has changed."""
        for n in "kv":
            codes, block, scale = (getattr(self, n + x) for x in ("_cache", "_block", "_scale"))
            setattr(self.p, n + "_cache", values(codes, block.transpose(1, 2), scale.transpose(1, 2)))


def make(lens_k, lens_q, heads_q, heads_kv, dim, page, *, packed=False, head_major=False, seed=0, device="cuda", spare=2,
         poison=True, high_pages=0):
    """Random problem; slots no sequence holds have NaN scales of both kinds (``poison``)."""
    p = R.make(lens_k, lens_q, heads_q, heads_kv, dim, page, packed=packed, head_major=head_major, seed=seed,
               device=device, spare=spare, poison=poison) if not high_pages else None
    if high_pages:   # numbers of pages past `high_pages`, without a cache of doubles that large
        p = R.make(lens_k, lens_q, heads_q, heads_kv, dim, page, packed=packed, seed=seed, device=device, spare=spare)
    parts = {}
    for n in "kv":
        x = getattr(p, n + "_cache").float()
        held = ~torch.isnan(x).any(-1)                                   # [pages, page, Hkv]
        codes, block, scale = quantise(torch.nan_to_num(x))
        # other values too: any code, block scales over their range, signs
        g = torch.Generator().manual_seed(seed + 77)
        odd = (torch.rand(held.shape, generator=g) < 0.25).to(device) & held
        codes[odd] = torch.randint(0, 256, codes.shape, generator=g).to(device).to(torch.uint8)[odd]
        if not poison:
            held = torch.ones_like(held)
        codes[~held] = 0xff
        block = torch.where(held[..., None], block.float(), math.nan).to(R.E4M3)
        scale = torch.where(held, scale, math.nan)
        if head_major:   # the codes of a head together, as the cache of R.make
            codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
        parts[n] = [codes.contiguous() if not head_major else codes, scale.transpose(1, 2).contiguous(),
                    block.transpose(1, 2).contiguous()]
    r = Problem4(p, parts["k"][0], parts["v"][0], parts["k"][1], parts["v"][1], parts["k"][2], parts["v"][2])
    r.refresh()
    return r


def append(q, table=None, positions=None, interleaved=False):
    """Writes the new rows into clones of a Problem4's cache, keys turned first; returns what all() gives."""
    p = q.p
    page = q.k_cache.shape[1]
    out = [x.clone() for x in q.all()]
    row = 0
    for b in range(len(p.lens_k)):
        n = p.lens_q[b]
        first = p.lens_k[b] - n
        for i, name in enumerate("kv"):
            rows = R.rows_of(p, getattr(p, name + "_new"), b).float()
            if n == 0:
                continue
            if name == "k" and table is not None:
                at = torch.arange(first, first + n, device=rows.device) if positions is None else \
                    positions.reshape(-1)[row:row + n]
                rows = rotated(rows, table, at, interleaved)
            codes, block, scale = quantise(rows)
            for j in range(n):
                pos = first + j
                at, slot = int(p.table[b, pos // page]), pos % page
                out[i][at, slot] = codes[j]
                out[2 + i][at, :, slot] = scale[j]
                out[4 + i][at, :, slot] = block[j]
        row += n
    return out


def same(got, want):
    """Bit for bit, but for the sign of an e4m3 NaN and the codes under one (whatever
    they are, their values are NaN). Both in the order of Problem4.all()."""
    got, want = list(got), list(want)
    for i in (0, 1):
        nan = torch.isnan(want[4 + i].float()).transpose(1, 2).repeat_interleave(BLOCK // 2, -1)   # [pages, page, Hkv, D / 2]
        got[i], want[i] = got[i].masked_fill(nan, 0), want[i].masked_fill(nan, 0)
    for g, w in zip(got, want):
        if g.dtype == R.E4M3:
            g, w = g.float(), w.float()
            assert torch.equal(torch.isnan(g), torch.isnan(w))
            g, w = g.nan_to_num(-1.0), w.nan_to_num(-1.0)
        assert torch.equal(R.bits(g), R.bits(w))
