"""Rotary positions and the paged cache in 4 bits, as cases that can be measured.

Four operators: ``rotary`` rotates the queries and keys of new tokens by their
positions, ``append`` writes new keys and values into the pages of a cache
with the rotation applied on the way (and rotates the queries), ``append_read``
quantises them into an e4m3 or a 4-bit (e2m1) cache and takes the sequences
back out, ``attend`` is the attention of each sequence's newest tokens over a
4-bit cache. ``step`` is a decoding step as it is used: append with rotation,
then attention. Every case runs either in its plain form (elementary torch
operations in fp32) or, with ``own`` set, through the framework's calls.

A 4-bit cache holds e2m1 codes, two to a byte (even depths in the low half),
an e4m3 scale for every 16 depths and an fp32 power of two for every (token,
head): a cached value is code * block scale * scale.

Lengths are a fixed function of the case (so that ``work`` knows them); values
and the order of the pages come from the seed.
"""
import math

import torch

own = False

E4M3_MAX, E2M1_MAX, BLOCK = 448.0, 6.0, 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the new tokens of 96 sequences rotated by their positions: a call where latency counts
        dict(name="rotary_step", op="rotary", batch=96, new=1, ragged_new=False, ctx=4096, heads_q=32, heads_kv=8,
             dim=128, page=16, kind="bf16", causal=True, rot=128, interleaved=False),
        # four prompts of 512 to 8192 tokens (packed); half of each head rotated, neighbouring values paired
        dict(name="rotary_prompts_partial", op="rotary", batch=4, new=8192, ragged_new=True, ctx=8192, heads_q=32,
             heads_kv=8, dim=128, page=16, kind="bf16", causal=True, rot=64, interleaved=True),
        # one decoding step's new tokens of 100 sequences, rotated and written
        dict(name="append_rotary_step", op="append", batch=100, new=1, ragged_new=False, ctx=2000, heads_q=32,
             heads_kv=8, dim=128, page=16, kind="bf16", causal=True, rot=128, interleaved=False),
        # the prompts of eight sequences of 512 to 8192 tokens (packed), rotated and written
        dict(name="append_rotary_prompts", op="append", batch=8, new=8192, ragged_new=True, ctx=8192, heads_q=32,
             heads_kv=8, dim=128, page=64, kind="bf16", causal=True, rot=128, interleaved=False),
        # a prompt chunk quantised to 4 bits, then every sequence read back for a contiguous prefill
        dict(name="append_read_e2m1", op="append_read", batch=6, new=1500, ragged_new=True, ctx=9000, heads_q=32,
             heads_kv=8, dim=128, page=32, kind="e2m1", causal=True, rot=0, interleaved=False),
        # the same at the small end: few heads, half the depth, odd lengths, part of the head rotated on the way
        dict(name="append_read_e2m1_d64", op="append_read", batch=3, new=37, ragged_new=True, ctx=331, heads_q=2,
             heads_kv=2, dim=64, page=16, kind="e2m1", causal=True, rot=32, interleaved=True),
        # one user's next token: the latency of a single short sequence
        dict(name="decode_one_e2m1", op="attend", batch=1, new=1, ragged_new=False, ctx=777, heads_q=32, heads_kv=8,
             dim=128, page=16, kind="e2m1", causal=True, rot=0, interleaved=False),
        # next tokens of 64 sequences of mixed lengths up to 8192: the ordinary serving step
        dict(name="decode_batch_e2m1", op="attend", batch=64, new=1, ragged_new=False, ctx=8192, heads_q=32,
             heads_kv=8, dim=128, page=64, kind="e2m1", causal=True, rot=0, interleaved=False),
        # next tokens of 16 long sequences: what 4 bits are for
        dict(name="decode_long_e2m1", op="attend", batch=16, new=1, ragged_new=False, ctx=32768, heads_q=32,
             heads_kv=8, dim=128, page=64, kind="e2m1", causal=True, rot=0, interleaved=False),
        # five drafted tokens per sequence, checked in one call; one query head per key head, depth 64
        dict(name="verify_d64_e2m1", op="attend", batch=24, new=5, ragged_new=False, ctx=4097, heads_q=16, heads_kv=16,
             dim=64, page=16, kind="e2m1", causal=True, rot=0, interleaved=False),
        # chunks of odd lengths of four sequences against what they have cached (packed queries): tensor-core work
        dict(name="chunk_ragged_e2m1", op="attend", batch=4, new=1023, ragged_new=True, ctx=12000, heads_q=32,
             heads_kv=8, dim=128, page=32, kind="e2m1", causal=True, rot=0, interleaved=False),
        # a whole step as it is used: the new token of each sequence rotated, written and attended with
        dict(name="step_rotary_e2m1", op="step", batch=32, new=1, ragged_new=False, ctx=4096, heads_q=32, heads_kv=8,
             dim=128, page=32, kind="e2m1", causal=True, rot=128, interleaved=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: any operator, odd sizes, few and many heads."""
    top = {n: max(work(c)[n] for c in listed()) for n in ("bytes", "flops")}
    while True:
        op = rng.choice(("rotary", "append", "append_read", "append_read", "attend", "attend", "attend", "attend", "step"))
        heads_kv = rng.choice((1, 2, 3, 4, 8, 16))
        group = rng.choice((1, 1, 2, 3, 4, 4, 5, 8, 16))
        ctx = _log(rng, 1, 32768)
        new = 1 if op in ("attend", "step") and rng.random() < 0.5 else _log(rng, 1, min(ctx, 2048))
        dim = rng.choice((64, 128, 128))
        rot = rng.choice((dim, dim, dim // 2, dim // 4)) if op in ("rotary", "append", "step") else rng.choice((0, dim, 16))
        kind = "e2m1"
        if op in ("rotary", "append"):
            kind = "bf16"
        elif op == "append_read" and rot and rng.random() < 0.4:
            kind = "e4m3"
        case = dict(op=op, batch=_log(rng, 1, 128), new=new, ragged_new=new > 1 and rng.random() < 0.5, ctx=ctx,
                    heads_q=heads_kv * group, heads_kv=heads_kv, dim=dim, page=rng.choice((16, 32, 64, 128)), kind=kind,
                    causal=rng.random() < 0.9, rot=0 if op == "attend" else rot,
                    interleaved=op != "attend" and rng.random() < 0.4)
        w = work(case)
        # the plain form holds every score and the gathered cache in fp32
        scores = case["batch"] * case["heads_q"] * new * ctx if op in ("attend", "step") else 0
        rows = case["batch"] * ctx * heads_kv * dim
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and scores <= 2.2e9 and rows <= 1.1e9:
            return case


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence: spread over their range, the last one at its upper end."""
    n = case["batch"]
    spread = [(0.37 + 0.6180339887 * (n - 1 - b)) % 1.0 if b < n - 1 else 1.0 for b in range(n)]
    new = [max(1, round(case["new"] * (1 + 15 * f) / 16)) if case["ragged_new"] else case["new"] for f in spread]
    low = max(1, case["ctx"] // 16)
    total = [max(q, round(low + (case["ctx"] - low) * f)) for q, f in zip(new, spread)]
    return new, total


def _row_bytes(case):
    """Bytes of one cached (token, head) vector."""
    dim = case["dim"]
    return {"bf16": 2 * dim, "e4m3": dim + 4, "e2m1": dim // 2 + dim // BLOCK + 4}[case["kind"]]


def work(case):
    new, total = _lengths(case)
    op, dim, hq, hkv = case["op"], case["dim"], case["heads_q"], case["heads_kv"]
    row, row16 = 2 * hkv * _row_bytes(case), 2 * hkv * 2 * dim   # one token's cached keys and values; the same as bf16
    n_new, n_all = sum(new), sum(total)
    pages = sum(-(-k // case["page"]) for k in total)
    nbytes = flops = 0
    if op in ("rotary", "append", "append_read", "step") and case["rot"]:
        seen = set()
        for q, k in zip(new, total):
            seen.update(range(k - q, k))
        nbytes += 4 * case["rot"] * len(seen)
        flops += 3 * n_new * case["rot"] * (hkv + (0 if op == "append_read" else hq))
    if op == "rotary":
        nbytes += n_new * (hq + hkv) * 4 * dim
    if op in ("append", "append_read", "step"):
        nbytes += n_new * (row16 + row) + 4 * len(new)
    if op in ("append", "step"):
        nbytes += n_new * hq * 4 * dim
    if op == "append_read":
        nbytes += n_all * (row16 + row) + 4 * pages
    if op in ("attend", "step"):
        nbytes += n_all * row + n_new * hq * (4 * dim + 4) + 4 * pages
        pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(new, total))
        flops += 4 * dim * hq * pairs
    return {"bytes": nbytes, "flops": flops}


def _empty_cache(case, pages):
    hkv, page, dim, dev = case["heads_kv"], case["page"], case["dim"], "cuda"
    if case["kind"] == "bf16":
        return torch.empty(pages, page, hkv, dim, dtype=torch.bfloat16, device=dev), None, None
    scale = torch.empty(pages, hkv, page, device=dev)
    if case["kind"] == "e4m3":
        return torch.empty(pages, page, hkv, dim, dtype=torch.float8_e4m3fn, device=dev), scale, None
    return (torch.empty(pages, page, hkv, dim // 2, dtype=torch.uint8, device=dev), scale,
            torch.empty(pages, hkv, page, dim // BLOCK, dtype=torch.float8_e4m3fn, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    new, total = _lengths(case)
    batch, page, hkv, dim, rot = case["batch"], case["page"], case["heads_kv"], case["dim"], case["rot"]
    used = [-(-k // page) for k in total]
    width = -(-case["ctx"] // page)
    pages = sum(used) + 3                                     # a few pages nobody holds
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([sum(used[:b]) for b in range(batch)], device=dev)
    col = torch.arange(width, device=dev)
    held = col[None] < torch.tensor(used, device=dev)[:, None]
    table = torch.where(held, order[(first[:, None] + col[None]).clamp(max=pages - 1)], 0).to(torch.int32)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def offsets(lengths):
        return torch.tensor([sum(lengths[:b]) for b in range(batch + 1)], dtype=torch.int32, device=dev)

    s = dict(case=case, table=table, seqlens=torch.tensor(total, dtype=torch.int32, device=dev), max_new=case["new"],
             total_k=sum(total), cu_k=offsets(total), cu_q=offsets(new) if case["ragged_new"] else None, angles=None)
    rows = (sum(new),) if case["ragged_new"] else (batch, case["new"])
    if case["op"] != "attend":
        s["k_new"], s["v_new"] = randn(*rows, hkv, dim), randn(*rows, hkv, dim) * 2
    if case["op"] != "append_read":
        s["q"] = randn(*rows, case["heads_q"], dim)
    if rot:
        # cosines and sines of every position: what a program makes once for its model
        turn = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        angle = torch.arange(case["ctx"], dtype=torch.float64, device=dev)[:, None] * turn
        s["angles"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["op"] == "rotary":
        return s
    # what the cache holds already: normally distributed values as its kind keeps them
    for name in ("k", "v"):
        cache, scale, block = _empty_cache(case, pages)
        step = max(1, (1 << 26) // (page * hkv * dim))
        for a in range(0, pages, step):
            x = randn(min(step, pages - a), page, hkv, dim)
            if case["kind"] == "bf16":
                cache[a:a + step] = x
                continue
            codes, sc, bl = _plain_quantise(x.float(), case["kind"])
            cache[a:a + step] = codes
            scale[a:a + step] = sc.transpose(1, 2)
            if block is not None:
                block[a:a + step] = bl.transpose(1, 2)
        s[name + "_cache"], s[name + "_scale"], s[name + "_block"] = cache, scale, block
    return s


# ------------------------------------------------------------------ plain forms
def _batch_of(s, x):
    """Packed rows [T, ...] as [B, new, ...] (short sequences padded), and which rows exist."""
    if s["cu_q"] is None:
        return x, None
    cu = s["cu_q"].long()
    i = torch.arange(s["max_new"], device=x.device)
    there = i[None] < (cu[1:] - cu[:-1])[:, None]
    return x[(cu[:-1, None] + i[None]).clamp(max=x.shape[0] - 1)], there


def _new_lengths(s, batch):
    if s["cu_q"] is None:
        return torch.full((batch,), s["max_new"], device=s["seqlens"].device)
    return (s["cu_q"][1:] - s["cu_q"][:-1]).long()


def _tokens(s):
    """Sequence and position of every new token, in the order of the rows."""
    batch = s["case"]["batch"]
    lengths = _new_lengths(s, batch)
    i = torch.arange(s["max_new"], device=lengths.device)
    at = s["seqlens"].long()[:, None] - lengths[:, None] + i[None]
    there = i[None] < lengths[:, None]
    b = torch.arange(batch, device=at.device)[:, None].expand_as(at)[there]
    return b, at[there]


def _plain_rotate(s, x, at):
    """Rows [T, H, D] in fp32, turned by their positions."""
    rot = s["case"]["rot"]
    if not rot:
        return x
    both = s["angles"][at]
    c, n = both[:, None, :rot // 2], both[:, None, rot // 2:]
    if s["case"]["interleaved"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([x1 * c - x2 * n, x2 * c + x1 * n], -1).flatten(-2)
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([x1 * c - x2 * n, x2 * c + x1 * n], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_quantise(x, kind):
    """fp32 vectors [..., D] as (codes, scale, block scales)."""
    most = E4M3_MAX if kind == "e4m3" else E4M3_MAX * E2M1_MAX          # 2^8 * 1.75, 2^11 * 1.3125
    border, drop = (0.875, 9) if kind == "e4m3" else (0.65625, 12)
    m, e = torch.frexp(x.abs().amax(-1))                               # amax = m 2^e, m in [1/2, 1)
    e = torch.where(m > border, e - drop + 1, e - drop).clamp(min=-126)  # smallest 2^e with amax / 2^e <= most
    scale = torch.where(m == 0, 1.0, torch.exp2(e.double())).float()
    x = (x / scale[..., None]).clamp(-most, most)
    if kind == "e4m3":
        return x.to(torch.float8_e4m3fn), scale, None
    parts = x.unflatten(-1, (-1, BLOCK))
    block = (parts.abs().amax(-1) / E2M1_MAX).to(torch.float8_e4m3fn)
    size = block.float()[..., None]
    y = torch.where(size == 0, 0.0, parts / torch.where(size == 0, 1.0, size)).flatten(-2)
    a = y.abs().clamp(max=E2M1_MAX)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) + 8 * torch.signbit(y)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale, block


def _plain_append(s):
    case = s["case"]
    b, at = _tokens(s)
    page, slot = s["table"][b, at // case["page"]].long(), at % case["page"]
    k = s["k_new"].reshape(-1, case["heads_kv"], case["dim"]).float()
    v = s["v_new"].reshape(-1, case["heads_kv"], case["dim"]).float()
    k = _plain_rotate(s, k, at)
    if case["kind"] == "bf16":
        s["k_cache"][page, slot] = k.to(torch.bfloat16)
        s["v_cache"][page, slot] = v.to(torch.bfloat16)
    else:
        (s["k_cache"][page, slot], s["k_scale"][page, :, slot], k_block) = _plain_quantise(k, case["kind"])
        (s["v_cache"][page, slot], s["v_scale"][page, :, slot], v_block) = _plain_quantise(v, case["kind"])
        if k_block is not None:
            s["k_block"][page, :, slot] = k_block
            s["v_block"][page, :, slot] = v_block


def _plain_rotated(s, name):
    _, at = _tokens(s)
    x = s[name]
    return _plain_rotate(s, x.reshape(-1, *x.shape[-2:]).float(), at).to(torch.bfloat16).view(x.shape)


def _gather(s, name, b, at):
    """Cached rows of sequences b at positions at, in fp32."""
    case = s["case"]
    page, slot = s["table"][b, at // case["page"]].long(), at % case["page"]
    x = s[name + "_cache"][page, slot]
    if case["kind"] == "bf16":
        return x.float()
    if case["kind"] == "e2m1":
        line = torch.tensor(E2M1, device=x.device)
        line = torch.cat([line, -line])
        pair = torch.stack([line.repeat(16), line.repeat_interleave(16)], -1)      # [256, 2]: what a byte holds
        x = pair[x.int()].flatten(-2).unflatten(-1, (-1, BLOCK))
        x = (x * s[name + "_block"][page, :, slot].float()[..., None]).flatten(-2)
    return x.float() * s[name + "_scale"][page, :, slot][..., None]


def _plain_read(s):
    cu = s["cu_k"].long()
    t = torch.arange(s["total_k"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return {"k": _gather(s, "k", b, t - cu[b]).to(torch.bfloat16), "v": _gather(s, "v", b, t - cu[b]).to(torch.bfloat16)}


def _plain_attend(s, rows):
    case = s["case"]
    batch, new, hq, hkv, dim = case["batch"], s["max_new"], case["heads_q"], case["heads_kv"], case["dim"]
    group = hq // hkv
    q, there = _batch_of(s, rows)
    at = torch.arange(case["ctx"], device=q.device)
    b = torch.arange(batch, device=q.device)[:, None].expand(batch, case["ctx"])
    held = at[None] < s["seqlens"][:, None]                                     # [B, ctx]
    pos = torch.where(held, at[None], 0)
    k = _gather(s, "k", b, pos).permute(0, 2, 3, 1)                             # [B, Hkv, D, ctx]
    v = torch.where(held[..., None, None], _gather(s, "v", b, pos), 0.0).permute(0, 2, 1, 3)
    r = q.float().reshape(batch, new, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * new, dim)
    x = torch.matmul(r, k) * dim ** -0.5                                        # [B, Hkv, group * new, ctx]
    sees = held[:, None, :]
    if case["causal"]:
        last = (s["seqlens"].long() - _new_lengths(s, batch))[:, None] + torch.arange(new, device=q.device)[None]
        sees = sees & (at[None, None] <= last[..., None])                       # [B, new, ctx]
    x = x.view(batch, hkv, group, new, -1).masked_fill_(~sees[:, None, None], -math.inf).view(batch, hkv, group * new, -1)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0].view(batch, hq, new)
    o = o.view(batch, hkv, group, new, dim).permute(0, 3, 1, 2, 4).reshape(batch, new, hq, dim).to(torch.bfloat16)
    if there is None:
        return {"o": o, "lse": lse}
    return {"o": o[there], "lse": lse.permute(0, 2, 1)[there].t().contiguous()}


def _plain(s):
    op = s["case"]["op"]
    if op == "rotary":
        return {"q": _plain_rotated(s, "q"), "k": _plain_rotated(s, "k_new")}
    if op == "attend":
        return _plain_attend(s, s["q"])
    _plain_append(s)
    if op == "append_read":
        return _plain_read(s)
    q = _plain_rotated(s, "q")
    if op == "append":
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    return dict(_plain_attend(s, q), q=q)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import attention_forward_sm100_gb300 as attn
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        q, k = attn.rotary(s["q"], s["k_new"], s["angles"], seqlens=s["seqlens"], cu_seqlens=s["cu_q"],
                           interleaved=case["interleaved"])
        return {"q": q, "k": k}
    held = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_block=s["k_block"], v_block=s["v_block"])
    q = s.get("q")
    if op != "attend":
        turn = dict(rotary_table=s["angles"], interleaved=case["interleaved"], q=q) if case["rot"] else {}
        q = attn.cache_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["seqlens"],
                              cu_seqlens_q=s["cu_q"], **held, **turn)
    if op == "append":
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    if op == "append_read":
        k, v = attn.cache_read(s["k_cache"], s["v_cache"], s["table"], s["cu_k"], total_k=s["total_k"], **held)
        return {"k": k, "v": v}
    o, lse = attn.paged_forward(q, s["k_cache"], s["v_cache"], s["table"], s["seqlens"], causal=case["causal"],
                                cu_seqlens_q=s["cu_q"], max_seqlen_q=s["max_new"] if s["cu_q"] is not None else None,
                                **held)
    return dict(o=o, lse=lse, q=q) if op == "step" else dict(o=o, lse=lse)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits
def _turned(case, angles, x, first):
    """Rows [L, H, D] of positions first, first + 1, ..., as doubles: each pair times the matrix of its angle."""
    rot = case["rot"]
    x = x.double()
    if not rot:
        return x
    half = rot // 2
    even, odd = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if case["interleaved"] else \
        (torch.arange(half), torch.arange(half, rot))
    z = torch.complex(x[..., even.to(x.device)], x[..., odd.to(x.device)])
    w = angles[first:first + x.shape[0]].double()
    z = z * torch.complex(w[:, :half], w[:, half:])[:, None]
    y = x.clone()
    y[..., even.to(x.device)], y[..., odd.to(x.device)] = z.real, z.imag
    return y


def _rounded_e4m3(y):
    """Doubles on the e4m3 grid (three mantissa bits, exponents from -6), nearest even, at most 448."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _kept(x, kind):
    """What a quantised cache makes of vectors [..., D], in doubles."""
    most = E4M3_MAX if kind == "e4m3" else E4M3_MAX * E2M1_MAX
    top = x.abs().amax(-1, keepdim=True)
    size = torch.exp2(torch.ceil(torch.log2(top / most)).clamp(min=-126))
    size = torch.where(top / size > most, size * 2, size)            # a log rounded down
    size = torch.where(top / (size / 2) <= most, size / 2, size)     # or up
    size = torch.where(top == 0, 1.0, size)
    if kind == "e4m3":
        return _rounded_e4m3(x / size) * size
    y = (x / size).unflatten(-1, (-1, BLOCK))
    block = _rounded_e4m3(y.abs().amax(-1, keepdim=True) / E2M1_MAX)
    y = torch.where(block == 0, 0.0, y / torch.where(block == 0, 1.0, block))
    # how many borders between neighbouring magnitudes lie below; ties go to the even code
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.int64)
    for n, (lo, hi) in enumerate(zip(E2M1, E2M1[1:])):
        code += (a >= (lo + hi) / 2) if n % 2 else (a > (lo + hi) / 2)
    values = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (torch.sign(y) * values[code] * block).flatten(-2) * size


def exact(case, seed):
    """Sequence by sequence from the definitions, in doubles; None where an output only holds copied values."""
    op, kind, hkv = case["op"], case["kind"], case["heads_kv"]
    s = prepare(case, seed)
    new, total = _lengths(case)
    table = s["table"].cpu().tolist()
    page, group = case["page"], case["heads_q"] // case["heads_kv"]
    angles, ragged = s["angles"], case["ragged_new"]
    out_k, out_v, out_o, out_l, out_q = [], [], [], [], []
    cache = s["k_cache"].double() if op == "append" else None
    row = 0
    for b in range(case["batch"]):
        q_len, k_len = new[b], total[b]
        at = slice(row, row + q_len)
        row += q_len
        first = k_len - q_len

        def rows(name):
            return s[name][at] if ragged else s[name][b]

        q = rows("q") if "q" in s else None
        if q is not None:
            q = _turned(case, angles, q, first)
            out_q.append(q)
        if op == "rotary":
            out_k.append(_turned(case, angles, rows("k_new"), first))
            continue
        ids = torch.tensor(table[b][:-(-k_len // page)], device=s["table"].device, dtype=torch.long)
        if op == "append":
            pos = torch.arange(first, k_len, device=ids.device)
            cache[ids[pos // page], pos % page] = _turned(case, angles, rows("k_new"), first)
            continue
        kv = {}
        for name in ("k", "v"):
            x = s[name + "_cache"][ids]
            if kind == "e2m1":
                values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=x.device)
                x = torch.stack([values[(x % 16).long()], values[(x // 16).long()]], -1).flatten(-2)
                x = x.unflatten(-1, (-1, BLOCK)) * s[name + "_block"][ids].double().transpose(1, 2)[..., None]
                x = x.flatten(-2)
            x = x.double() * s[name + "_scale"][ids].double().transpose(1, 2)[..., None]
            x = x.flatten(0, 1)[:k_len]                                               # [Lk, Hkv, D]
            if op in ("append_read", "step"):
                fresh = rows(name + "_new")
                fresh = _turned(case, angles, fresh, first) if name == "k" else fresh.double()
                x[first:] = _kept(fresh, kind)
            kv[name] = x
        if op == "append_read":
            out_k.append(kv["k"])
            out_v.append(kv["v"])
            continue
        if op == "step":
            q = q.to(torch.bfloat16).double()                                         # as it is handed on
        sees = torch.ones(q_len, k_len, dtype=torch.bool, device=q.device)
        if case["causal"]:
            sees = sees.tril(k_len - q_len)
        o, lse = torch.empty_like(q), torch.empty(case["heads_q"], q_len, device=q.device, dtype=torch.float64)
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            w = torch.einsum("qhd,kd->hqk", q[:, heads], kv["k"][:, h]) / math.sqrt(case["dim"])
            w = torch.where(sees, w, -math.inf)
            lse[heads] = torch.logsumexp(w, -1)
            o[:, heads] = torch.einsum("hqk,kd->qhd", torch.softmax(w, -1), kv["v"][:, h])
        out_o.append(o)
        out_l.append(lse)

    def joined(parts):
        return torch.cat(parts) if ragged else torch.stack(parts)

    if op == "rotary":
        return {"q": joined(out_q), "k": joined(out_k)}
    if op == "append":
        return {"q": joined(out_q), "k": cache, "v": None}
    if op == "append_read":
        return {"k": torch.cat(out_k), "v": torch.cat(out_v)}
    r = {"o": joined(out_o), "lse": torch.cat(out_l, 1) if ragged else torch.stack(out_l)}
    return dict(r, q=joined(out_q)) if op == "step" else r
