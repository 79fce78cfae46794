"""The paged-cache operators from their definitions in 64 bits, one sequence
at a time with plain loops over tokens and heads, and problems to run them
on. Torch doubles on the device of the inputs; nothing of the library."""
import dataclasses
import math

import torch

E4M3 = torch.float8_e4m3fn


@dataclasses.dataclass
class Problem:
    """A cache, its tables and the new rows of one call."""
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: object
    v_scale: object
    table: torch.Tensor
    seqlens: torch.Tensor
    lens_k: list
    lens_q: list
    cu_q: object
    q: torch.Tensor
    k_new: torch.Tensor
    v_new: torch.Tensor

    @property
    def cache(self):
        return (self.k_cache, self.v_cache, self.table, self.seqlens)

    @property
    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)


def make(lens_k, lens_q, heads_q, heads_kv, dim, page, *, fp8=False, packed=False, head_major=False, seed=0,
         device="cuda", spare=2, poison=True, high_pages=0):
    """Random problem. Every slot no sequence holds is NaN (``poison``), table
    columns past a sequence's pages hold numbers outside the cache, page order
    is shuffled; ``high_pages`` unused pages come first."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens_k]
    pages = sum(used) + spare + high_pages
    order = (torch.randperm(sum(used) + spare, generator=g) + high_pages).tolist()
    width = max(used + [1]) + 1
    table = torch.full((len(lens_k), width), 1 << 30, dtype=torch.int32)
    for b, n in enumerate(used):
        for c in range(n):
            table[b, c] = order.pop()
    shape = (pages, heads_kv, page, dim) if head_major else (pages, page, heads_kv, dim)

    def randn(*s):
        return torch.randn(*s, generator=g)

    def cache():
        if high_pages:
            x = torch.empty(shape, dtype=E4M3 if fp8 else torch.bfloat16, device=device)
            x.view(torch.uint8 if fp8 else torch.int16).fill_(0x7f if fp8 else 0x7fff)
        else:
            x = torch.full(shape, math.nan, device=device).to(E4M3 if fp8 else torch.bfloat16)
        x = x.transpose(1, 2) if head_major else x
        sc = torch.full((pages, heads_kv, page), math.nan, device=device) if fp8 else None
        for b, n in enumerate(lens_k):
            for c in range(used[b]):
                m = min(page, n - c * page) if poison else page
                rows = randn(m, heads_kv, dim)
                at = int(table[b, c])
                if fp8:
                    x[at, :m] = (rows * 100).clamp(-448, 448).to(device).to(E4M3)
                    sc[at, :, :m] = torch.exp2(torch.randint(-9, -4, (heads_kv, m), generator=g).double()).float().to(device)
                else:
                    x[at, :m] = rows.to(device).to(torch.bfloat16)
        return x, sc

    k_cache, k_scale = cache()
    v_cache, v_scale = cache()
    cu = None
    if packed:
        cu = torch.tensor([sum(lens_q[:b]) for b in range(len(lens_q) + 1)], dtype=torch.int32, device=device)
        rows = (sum(lens_q),)
    else:
        assert len(set(lens_q)) <= 1
        rows = (len(lens_q), lens_q[0] if lens_q else 1)
    bf = lambda *s: randn(*s).to(torch.bfloat16).to(device)  # noqa: E731
    return Problem(k_cache, v_cache, k_scale, v_scale, table.to(device),
                   torch.tensor(lens_k, dtype=torch.int32, device=device), list(lens_k), list(lens_q), cu,
                   bf(*rows, heads_q, dim), bf(*rows, heads_kv, dim), bf(*rows, heads_kv, dim) * 2)


def rows_of(p, x, b):
    """New rows of sequence b, [Lq, H, D]."""
    if p.cu_q is None:
        return x[b]
    return x[sum(p.lens_q[:b]):sum(p.lens_q[:b + 1])]


def gather(p, b):
    """Cached K and V of sequence b as doubles, [Lk, Hkv, D]."""
    page = p.k_cache.shape[1]
    out = []
    for x, s in ((p.k_cache, p.k_scale), (p.v_cache, p.v_scale)):
        parts = []
        for c in range(-(-p.lens_k[b] // page)):
            m = min(page, p.lens_k[b] - c * page)
            at = int(p.table[b, c])
            rows = x[at, :m].double()
            if s is not None:
                rows = rows * s[at, :, :m].double().t()[..., None]
            parts.append(rows)
        out.append(torch.cat(parts) if parts else x.new_zeros((0,) + tuple(x.shape[2:]), dtype=torch.float64))
    return out


def attend(p, causal, scale=None):
    """Per sequence (O, LSE, sum of weight * |v|) as doubles: [Lq, Hq, D], [Hq, Lq], [Lq, Hq, D]."""
    heads_q, dim = p.q.shape[-2:]
    group = heads_q // p.k_cache.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    result = []
    for b in range(len(p.lens_k)):
        k, v = gather(p, b)
        q = rows_of(p, p.q, b).double()
        lq, lk = q.shape[0], k.shape[0]
        o = torch.zeros_like(q)
        absv = torch.zeros_like(q)
        lse = torch.full((heads_q, lq), -math.inf, dtype=torch.float64, device=q.device)
        last = torch.arange(lq, device=q.device)[:, None] + (lk - lq)
        sees = torch.arange(lk, device=q.device)[None] <= (last if causal else torch.full_like(last, lk))
        some = sees.any(1)
        for h in range(heads_q):
            s = torch.where(sees, scale * (q[:, h] @ k[:, h // group].t()), -math.inf)
            if not some.any():
                continue
            lse[h, some] = torch.logsumexp(s[some], 1)
            w = torch.zeros_like(s)
            w[some] = torch.exp(s[some] - lse[h, some][:, None])
            o[:, h] = w @ v[:, h // group]
            absv[:, h] = w @ v[:, h // group].abs()
        result.append((o, lse, absv))
    return result


def check_attend(p, o, lse, causal, scale=None):
    """Holds every element to the bound the roundings imply: O is rounded once
    to bf16 (2^-8 of it) and every weight once (2^-8 of sum w |v|); scores,
    exponentials and sums in fp32 add less than 2^-14 of that. LSE is fp32:
    the score's error, below 2^-24 * (2 + D / 16) * scale * sum |q k| < 2e-5 here,
    the exponential's 2^-22 and the logarithm's rounding."""
    for b, (ro, rl, ra) in enumerate(attend(p, causal, scale)):
        if ro.shape[0] == 0:
            continue
        if p.cu_q is None:
            go, gl = o[b], lse[b]
        else:
            at = slice(sum(p.lens_q[:b]), sum(p.lens_q[:b + 1]))
            go, gl = o[at], lse[:, at]
        bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -14) * ra + 1e-6
        worst = ((go.double() - ro).abs() / bound).max().item()
        assert worst <= 1.0, f"sequence {b}: O is {worst:.3f} of its bound off"
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(gl), empty) and bool((gl[empty] < 0).all())
        assert bool((go.double().permute(1, 0, 2)[empty] == 0).all())
        off = (gl.double() - rl)[~empty].abs()
        assert off.numel() == 0 or off.max().item() <= 5e-5, f"sequence {b}: LSE off by {off.max().item():.2e}"


def quantise(x):
    """(codes as e4m3, scale) of bf16 vectors [..., D], in doubles and from the definition."""
    y = x.double()
    fine = torch.where(torch.isfinite(y), y.abs(), 0.0).amax(-1)
    scale = torch.ones_like(fine)
    e = -126
    todo = fine > 0
    while bool(todo.any()):   # the smallest power of two that brings amax to 448 or below
        fits = todo & (fine <= 448.0 * 2.0 ** e)
        scale[fits] = 2.0 ** e
        todo &= ~fits
        e += 1
    z = (y / scale[..., None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)   # exact for e4m3's exponents
    z = torch.where(torch.isnan(y), math.nan, torch.round(z / step) * step)
    return z.float().to(E4M3), scale.float()


def append(p):
    """Writes the new rows into clones of the cache; returns (k, v, k_scale, v_scale)."""
    page = p.k_cache.shape[1]
    out = []
    for x, s, new in ((p.k_cache, p.k_scale, p.k_new), (p.v_cache, p.v_scale, p.v_new)):
        x = x.clone()
        s = None if s is None else s.clone()
        for b in range(len(p.lens_k)):
            rows = rows_of(p, new, b)
            if rows.shape[0] == 0:
                continue
            codes, scale = (rows, None) if s is None else quantise(rows)
            for i in range(rows.shape[0]):
                pos = p.lens_k[b] - p.lens_q[b] + i
                at, slot = int(p.table[b, pos // page]), pos % page
                x[at, slot] = codes[i]
                if s is not None:
                    s[at, :, slot] = scale[i]
        out.append((x, s))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def bits(t):
    """The tensor's bit patterns (NaN compares equal to itself)."""
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])
