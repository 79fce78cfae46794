"""The paged key/value cache operators, as cases that can be measured.

Three operators: ``append`` writes the keys and values of new tokens into the
pages of a cache (as bf16, or rounded to e4m3 with one scale per token and
head), ``read`` takes sequences back out of the pages, ``attend`` is the
attention of each sequence's newest tokens over everything it has cached.
Every case runs either in its plain form (elementary torch operations in
fp32) or, with ``own`` set, through the framework's calls.

Lengths are a fixed function of the case (so that ``work`` knows them); values
and the order of the pages come from the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one decoding step's new tokens of 100 sequences: a write where latency counts
        dict(name="append_step_bf16", op="append", batch=100, new=1, ragged_new=False, ctx=2000, heads_q=8, heads_kv=8,
             dim=128, page=16, fp8=False, causal=True),
        # the prompts of eight sequences of 512 to 8192 tokens (packed), written to the cache as they are
        dict(name="append_prompts_bf16", op="append", batch=8, new=8192, ragged_new=True, ctx=8192, heads_q=32,
             heads_kv=8, dim=128, page=64, fp8=False, causal=True),
        # a prompt chunk quantised into the cache, then every sequence read back for a contiguous prefill
        dict(name="append_read_e4m3", op="append_read", batch=6, new=1500, ragged_new=True, ctx=9000, heads_q=32,
             heads_kv=8, dim=128, page=32, fp8=True, causal=True),
        # the same at the small end: few heads, half the depth, odd lengths
        dict(name="append_read_e4m3_d64", op="append_read", batch=3, new=37, ragged_new=True, ctx=331, heads_q=2,
             heads_kv=2, dim=64, page=16, fp8=True, causal=True),
        # cached sequences handed to a contiguous kernel: reading only
        dict(name="read_bf16", op="read", batch=8, new=1, ragged_new=False, ctx=8192, heads_q=32, heads_kv=8, dim=128,
             page=128, fp8=False, causal=True),
        # one user's next token: the latency of a single short sequence
        dict(name="decode_one_bf16", op="attend", batch=1, new=1, ragged_new=False, ctx=777, heads_q=32, heads_kv=8,
             dim=128, page=16, fp8=False, causal=True),
        # next tokens of 64 sequences of mixed lengths up to 8192: the ordinary serving step
        dict(name="decode_batch_bf16", op="attend", batch=64, new=1, ragged_new=False, ctx=8192, heads_q=32, heads_kv=8,
             dim=128, page=64, fp8=False, causal=True),
        # next tokens of 16 long sequences over an e4m3 cache
        dict(name="decode_long_e4m3", op="attend", batch=16, new=1, ragged_new=False, ctx=32768, heads_q=32, heads_kv=8,
             dim=128, page=64, fp8=True, causal=True),
        # five drafted tokens per sequence, checked in one call; one query head per key head, depth 64
        dict(name="verify_d64_bf16", op="attend", batch=24, new=5, ragged_new=False, ctx=4097, heads_q=16, heads_kv=16,
             dim=64, page=16, fp8=False, causal=True),
        # a chunk of a long prompt against what is cached already: tensor-core work
        dict(name="chunk_long_bf16", op="attend", batch=1, new=2048, ragged_new=False, ctx=32768, heads_q=32,
             heads_kv=8, dim=128, page=64, fp8=False, causal=True),
        # chunks of odd lengths of four sequences over an e4m3 cache (packed queries)
        dict(name="chunk_ragged_e4m3", op="attend", batch=4, new=1023, ragged_new=True, ctx=12000, heads_q=32,
             heads_kv=8, dim=128, page=32, fp8=True, causal=True),
        # a whole step as it is used: the new token of each sequence written, then its attention
        dict(name="step_bf16", op="step", batch=32, new=1, ragged_new=False, ctx=4096, heads_q=32, heads_kv=8, dim=128,
             page=32, fp8=False, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: any operator, odd sizes, few and many heads."""
    top = {n: max(work(c)[n] for c in listed()) for n in ("bytes", "flops")}
    while True:
        op = rng.choice(("append", "append_read", "read", "attend", "attend", "attend", "attend", "step"))
        heads_kv = rng.choice((1, 2, 3, 4, 8, 16))
        group = rng.choice((1, 1, 2, 3, 4, 4, 5, 8, 16))
        ctx = _log(rng, 1, 32768)
        new = 1 if op in ("attend", "step") and rng.random() < 0.5 else _log(rng, 1, min(ctx, 2048))
        case = dict(op=op, batch=_log(rng, 1, 128), new=new, ragged_new=new > 1 and rng.random() < 0.5, ctx=ctx,
                    heads_q=heads_kv * group, heads_kv=heads_kv, dim=rng.choice((64, 128, 128)),
                    page=rng.choice((16, 32, 64, 128)), fp8=op == "append_read" or (op in ("read", "attend") and rng.random() < 0.5),
                    causal=rng.random() < 0.9)
        w = work(case)
        # the plain form holds every score and the gathered cache in fp32
        scores = case["batch"] * case["heads_q"] * new * ctx if op in ("attend", "step") else 0
        rows = case["batch"] * ctx * heads_kv * case["dim"]
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


def work(case):
    new, total = _lengths(case)
    dim, hq, hkv = case["dim"], case["heads_q"], case["heads_kv"]
    row = 2 * hkv * ((dim + 4) if case["fp8"] else 2 * dim)   # one token's cached keys and values
    row16 = 2 * hkv * 2 * dim                                 # the same as bf16
    n_new, n_all = sum(new), sum(total)
    pages = sum(-(-k // case["page"]) for k in total)
    nbytes = flops = 0
    if case["op"] in ("append", "append_read", "step"):
        nbytes += n_new * (row16 + row)
    if case["op"] in ("read", "append_read"):
        nbytes += n_all * (row16 + row) + 4 * pages
    if case["op"] in ("attend", "step"):
        nbytes += n_all * row + n_new * hq * (4 * dim + 4) + 4 * pages
        pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(new, total))
        flops += 4 * dim * hq * pairs
    return {"bytes": nbytes, "flops": flops}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    new, total = _lengths(case)
    batch, page, hkv, dim = case["batch"], case["page"], case["heads_kv"], case["dim"]
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
             total_k=sum(total), cu_k=offsets(total), k_scale=None, v_scale=None,
             cu_q=offsets(new) if case["ragged_new"] else None)
    rows = (sum(new),) if case["ragged_new"] else (batch, case["new"])
    if case["op"] in ("append", "append_read", "step"):
        s["k_new"], s["v_new"] = randn(*rows, hkv, dim), randn(*rows, hkv, dim) * 2
    if case["op"] in ("attend", "step"):
        s["q"] = randn(*rows, case["heads_q"], dim)
    for name in ("k", "v"):
        x = randn(pages, page, hkv, dim)
        if case["fp8"]:
            # what a quantised cache holds: codes up to 448 and a power of two per token and head
            s[name + "_cache"] = (x * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            e = torch.randint(-8, -5, (pages, hkv, page), generator=g, device=dev)
            s[name + "_scale"] = torch.exp2(e.double()).float()
        else:
            s[name + "_cache"] = x
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
        return torch.full((batch,), s["max_new"], device=s["table"].device)
    return (s["cu_q"][1:] - s["cu_q"][:-1]).long()


def _plain_append(s):
    case, table = s["case"], s["table"]
    lengths = _new_lengths(s, case["batch"])
    i = torch.arange(s["max_new"], device=table.device)
    at = s["seqlens"].long()[:, None] - lengths[:, None] + i[None]          # position of every new token
    there = i[None] < lengths[:, None]
    b = torch.arange(case["batch"], device=table.device)[:, None].expand_as(at)[there]
    at = at[there]
    page, slot = table[b, at // case["page"]].long(), at % case["page"]
    for name in ("k", "v"):
        x = s[name + "_new"].reshape(-1, case["heads_kv"], case["dim"])
        if case["fp8"]:
            x = x.float()
            m, e = torch.frexp(x.abs().amax(-1))                               # amax = m 2^e, m in [1/2, 1)
            e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)            # smallest 2^e with amax / 2^e <= 448
            scale = torch.where(m == 0, 1.0, torch.exp2(e.double())).float()
            x = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s[name + "_scale"][page, :, slot] = scale
        s[name + "_cache"][page, slot] = x


def _gather(s, name, b, at):
    """Cached rows of sequences b at positions at, in fp32."""
    page, slot = s["table"][b, at // s["case"]["page"]].long(), at % s["case"]["page"]
    x = s[name + "_cache"][page, slot].float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][page, :, slot][..., None]
    return x


def _plain_read(s):
    cu = s["cu_k"].long()
    t = torch.arange(s["total_k"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return {n: _gather(s, n, b, t - cu[b]).to(torch.bfloat16) for n in ("k", "v")}


def _plain_attend(s):
    case = s["case"]
    batch, new, hq, hkv, dim = case["batch"], s["max_new"], case["heads_q"], case["heads_kv"], case["dim"]
    group = hq // hkv
    q, there = _batch_of(s, s["q"])
    at = torch.arange(case["ctx"], device=q.device)
    b = torch.arange(batch, device=q.device)[:, None].expand(batch, case["ctx"])
    held = at[None] < s["seqlens"][:, None]                                     # [B, ctx]
    pos = torch.where(held, at[None], 0)
    k = _gather(s, "k", b, pos).permute(0, 2, 3, 1)                             # [B, Hkv, D, ctx]
    v = torch.where(held[..., None, None], _gather(s, "v", b, pos), 0.0).permute(0, 2, 1, 3)
    rows = q.float().reshape(batch, new, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * new, dim)
    x = torch.matmul(rows, k) * dim ** -0.5                                     # [B, Hkv, group * new, ctx]
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
    if op in ("append", "append_read", "step"):
        _plain_append(s)
    if op == "append":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    if op in ("append_read", "read"):
        return _plain_read(s)
    r = _plain_attend(s)
    return dict(r, k=s["k_cache"], v=s["v_cache"]) if op == "step" else r


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import attention_forward_sm100_gb300 as attn
    op = s["case"]["op"]
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op in ("append", "append_read", "step"):
        attn.cache_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["seqlens"],
                          cu_seqlens_q=s["cu_q"], **scales)
    if op == "append":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    if op in ("append_read", "read"):
        k, v = attn.cache_read(s["k_cache"], s["v_cache"], s["table"], s["cu_k"], total_k=s["total_k"], **scales)
        return {"k": k, "v": v}
    o, lse = attn.paged_forward(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seqlens"],
                                causal=s["case"]["causal"], cu_seqlens_q=s["cu_q"],
                                max_seqlen_q=s["max_new"] if s["cu_q"] is not None else None, **scales)
    return dict(o=o, lse=lse, k=s["k_cache"], v=s["v_cache"]) if op == "step" else dict(o=o, lse=lse)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits
def _rounded_e4m3(y):
    """Doubles on the e4m3 grid (three mantissa bits, exponents from -6), nearest even, at most 448."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    """Sequence by sequence from the definitions, in doubles; None where an output only holds copied values."""
    op = case["op"]
    if op in ("append", "read") and not case["fp8"]:
        return None
    s = prepare(case, seed)
    new, total = _lengths(case)
    table = s["table"].cpu().tolist()
    page, group = case["page"], case["heads_q"] // case["heads_kv"]
    out_k, out_v, out_o, out_l = [], [], [], []
    row = 0
    for b in range(case["batch"]):
        q_len, k_len = new[b], total[b]
        ids = torch.tensor(table[b][:-(-k_len // page)], device=s["table"].device, dtype=torch.long)
        kv = {}
        for name in ("k", "v"):
            x = s[name + "_cache"][ids].double().flatten(0, 1)[:k_len]              # [Lk, Hkv, D]
            if case["fp8"]:
                x = x * s[name + "_scale"][ids].double().transpose(1, 2).flatten(0, 1)[:k_len, :, None]
            if op in ("append_read", "step"):
                fresh = s[name + "_new"]
                fresh = (fresh[row:row + q_len] if case["ragged_new"] else fresh[b]).double()
                if case["fp8"]:
                    top = fresh.abs().amax(-1, keepdim=True)
                    size = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-126))
                    size = torch.where(top / size > E4M3_MAX, size * 2, size)       # a log rounded down
                    size = torch.where(top / (size / 2) <= E4M3_MAX, size / 2, size)  # or up
                    fresh = _rounded_e4m3(fresh / size) * size
                x[k_len - q_len:] = fresh
            kv[name] = x
        if op in ("append_read", "read"):
            out_k.append(kv["k"])
            out_v.append(kv["v"])
            row += q_len
            continue
        q = (s["q"][row:row + q_len] if case["ragged_new"] else s["q"][b]).double()   # [Lq, Hq, D]
        row += q_len
        sees = torch.ones(q_len, k_len, dtype=torch.bool, device=q.device)
        if case["causal"]:
            sees = sees.tril(k_len - q_len)
        o, lse = torch.empty_like(q), torch.empty(case["heads_q"], q_len, device=q.device, dtype=torch.float64)
        for h in range(case["heads_q"]):
            w = (q[:, h] @ kv["k"][:, h // group].t()) / math.sqrt(case["dim"])
            w = torch.where(sees, w, -math.inf)
            lse[h] = torch.logsumexp(w, -1)
            o[:, h] = torch.softmax(w, -1) @ kv["v"][:, h // group]
        out_o.append(o)
        out_l.append(lse)
    if op in ("append_read", "read"):
        return {"k": torch.cat(out_k), "v": torch.cat(out_v)}
    packed = case["ragged_new"]
    r = {"o": torch.cat(out_o) if packed else torch.stack(out_o),
         "lse": torch.cat(out_l, 1) if packed else torch.stack(out_l)}
    return dict(r, k=None, v=None) if op == "step" else r
