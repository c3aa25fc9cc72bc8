"""The attention sublayer of a decoder layer that serves prompts and then continues them: attention
over packed prompts, writing a chunk's keys and values into a paged cache, and attention of a chunk
of new tokens (one token each, when decoding) over that cache.

Every case goes through run() in two forms: elementary torch operations in 32 bits, rounded once at
the end (own = False), and the library's operators (own = True).
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _lens(text):
    return [int(t) for t in text.split(",")]


def _text(lens):
    return ",".join(str(n) for n in lens)


def listed():
    return [
        # One short question to a small model: 17 tokens, nothing but latency.
        dict(name="prompt short", op="prompt", lens="17", heads=8, kv_heads=2, head_dim=64, dtype="bf16"),
        # A batch of prompts of very different lengths, one of a single token and one empty (a
        # request that was withdrawn), packed one after the other.
        dict(name="prompt ragged batch", op="prompt", lens="333,1,700,64,0,129,512,45,255,801,17,390,128,611",
             heads=32, kv_heads=8, head_dim=128, dtype="bf16"),
        # Narrow heads without grouping, in f16: four documents of odd lengths.
        dict(name="prompt narrow heads", op="prompt", lens="1999,2048,1501,777", heads=16, kv_heads=16,
             head_dim=64, dtype="f16"),
        # One long document: bound by the tensor cores.
        dict(name="prompt long", op="prompt", lens="16384", heads=16, kv_heads=4, head_dim=128, dtype="bf16"),
        # One user decoding early in a conversation: one token over 511 positions, small pages.
        dict(name="decode one", op="paged", q_lens="1", kv_lens="511", page=16, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # The batch that the benchmark decodes: 64 sequences, one token each, about 2048 positions.
        dict(name="decode batch", op="paged", q_lens=_text([1] * 64),
             kv_lens=_text([2048 - 29 * (i % 17) for i in range(64)]), page=64, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # Four conversations over very long caches: the cache's bytes and nothing else count.
        dict(name="decode long", op="paged", q_lens="1,1,1,1", kv_lens="131072,100003,131001,70001", page=64,
             heads=64, kv_heads=8, head_dim=128, dtype="bf16"),
        # Checking a draft of five tokens for sixteen sequences at once, f16, pages of 48 slots.
        dict(name="verify draft", op="paged", q_lens=_text([5] * 16),
             kv_lens=_text([3000 + 111 * i for i in range(16)]), page=48, heads=32, kv_heads=4, head_dim=128,
             dtype="f16"),
        # A server that mixes a chunk of a long prompt with requests that decode.
        dict(name="chunk mixed", op="paged", q_lens="1024,1,1,300,1,1,1,1",
             kv_lens="9000,4100,700,300,2222,1,6001,3333", page=32, heads=32, kv_heads=8, head_dim=128,
             dtype="bf16"),
        # The new keys and values of the decoding batch.
        dict(name="append batch", op="append", q_lens=_text([1] * 64),
             kv_lens=_text([2048 - 29 * (i % 17) for i in range(64)]), page=64, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # The keys and values of two long chunks.
        dict(name="append chunks", op="append", q_lens="8192,5003", kv_lens="16384,5003", page=16, heads=32,
             kv_heads=8, head_dim=128, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    case = dict(op=rng.choice(["prompt", "prompt", "paged", "paged", "paged", "append"]),
                heads=kv_heads * group, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128, 80]),
                dtype=rng.choice(["bf16", "bf16", "f16"]))
    if case["op"] == "prompt":
        longest = _log_int(rng, 1, 12000)
        lens = [longest] + [_log_int(rng, 1, longest) for _ in range(_log_int(rng, 1, 24) - 1)]
        # the plain form holds a score for every pair of a padded batch: at most 4 G of them
        while len(lens) * longest ** 2 * case["heads"] > 4 << 30 and len(lens) > 1:
            lens.pop()
        while longest ** 2 * case["heads"] > 4 << 30:
            longest = longest * 3 // 4
            lens[0] = longest
        rng.shuffle(lens)
        return dict(case, lens=_text(lens))
    n = _log_int(rng, 1, 64)
    chunk = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1500)
    longest = _log_int(rng, max(chunk, 16), 120000)
    while n > 1 and (n * longest * kv_heads * case["head_dim"] > 400 << 20 or n * chunk * longest * case["heads"] > 1 << 30):
        n -= 1
    while chunk > 1 and chunk * longest * case["heads"] > 1 << 30:
        chunk = chunk * 3 // 4
    q = [chunk] + [rng.randint(1, chunk) for _ in range(n - 1)]
    kv = [longest] + [max(q[i], _log_int(rng, 1, longest)) for i in range(1, n)]
    return dict(case, q_lens=_text(q), kv_lens=_text(kv), page=rng.choice([16, 32, 48, 64, 128]))


def _pages(case):
    return [-(-n // case["page"]) for n in _lens(case["kv_lens"])]


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "prompt":
        lens = _lens(case["lens"])
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * h + 2 * hk) * d * 2, "flops": 4 * d * h * pairs}
    q, kv = _lens(case["q_lens"]), _lens(case["kv_lens"])
    if case["op"] == "append":  # every new key and value is read once and written once
        return {"bytes": sum(q) * hk * d * 2 * 2 * 2, "flops": 0}
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, kv))
    return {"bytes": (sum(q) * 2 * h + sum(kv) * 2 * hk) * d * 2, "flops": 4 * d * h * pairs}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    lens = _lens(case["lens"] if case["op"] == "prompt" else case["q_lens"])
    total = sum(lens)
    # what a layer's projection leaves: queries, keys and values of a token beside each other
    qkv = torch.randn((total, h + 2 * hk, d), generator=g, device="cuda")
    qkv[:, :h] *= 1.5
    qkv = qkv.to(dtype)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s = dict(case=dict(case), q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:], max_q=max(lens),
             cu=torch.tensor(starts, dtype=torch.int32, device="cuda"),
             out=torch.empty((total, h, d), dtype=dtype, device="cuda"))
    if case["op"] != "prompt":
        need = _pages(case)
        width = max(need)
        order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((len(need), width), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):  # a sequence's pages lie anywhere in the cache
            table[i, :n] = order[at:at + n]
            at += n
        shape = (order.numel(), case["page"], hk, d)
        s["k_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        s["v_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
        s["table"] = table
        s["kv_len"] = torch.tensor(_lens(case["kv_lens"]), dtype=torch.int32, device="cuda")
        s["max_kv"] = max(_lens(case["kv_lens"]))
    return s


def _rows(s):
    """For each packed token, its sequence and its place in it."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, t - cu[b]


def _padded(x, b, i, n, width):
    y = torch.zeros((n, width) + x.shape[1:], dtype=torch.float32, device=x.device)
    y[b, i] = x.float()
    return y


def _attend(q, k, v, ok, scale):
    """q [B, T, H, D], k and v [B, S, Hk, D] in 32 bits, ok [B, T, S]: which keys a query sees."""
    B, T, H, D = q.shape
    hk = k.shape[2]
    q = q.reshape(B, T, hk, H // hk, D).permute(0, 2, 3, 1, 4).reshape(B, hk, H // hk * T, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, H, T, -1)
    p.mul_(scale).masked_fill_(~ok[:, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hk, H // hk * T, -1), v.permute(0, 2, 1, 3)).view(B, H, T, D)
    return (o / torch.where(total == 0, torch.ones_like(total), total)).transpose(1, 2)


def _plain(s):
    case = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    b, i = _rows(s)
    if case["op"] == "append":
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        at = s["kv_len"].long()[b] - n[b] + i
        page = s["table"][b, at // case["page"]].long()
        s["k_cache"][page, at % case["page"]] = k
        s["v_cache"][page, at % case["page"]] = v
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    n = s["cu"].numel() - 1
    qp = _padded(q, b, i, n, s["max_q"])
    t = torch.arange(s["max_q"], device=q.device)
    if case["op"] == "prompt":
        kp, vp = _padded(k, b, i, n, s["max_q"]), _padded(v, b, i, n, s["max_q"])
        ok = (t[None, :] <= t[:, None]).expand(n, -1, -1)
    else:
        kp = s["k_cache"][s["table"].long()].flatten(1, 2)[:, :s["max_kv"]].float()
        vp = s["v_cache"][s["table"].long()].flatten(1, 2)[:, :s["max_kv"]].float()
        last = s["kv_len"] - (s["cu"][1:] - s["cu"][:-1])
        ok = torch.arange(s["max_kv"], device=q.device)[None, None] <= (last[:, None] + t[None, :])[:, :, None]
    o = _attend(qp, kp, vp, ok, 1.0 / math.sqrt(case["head_dim"]))
    return {"out": o[b, i].to(q.dtype)}


def run(state):
    if not own:
        return _plain(state)
    import deepseek_v4_engram_gb300 as eg
    case = state["case"]
    if "desc" not in state:  # the plan and the scratch that a program keeps for a layer
        state["desc"] = eg.make_attn_desc(case["heads"], case["kv_heads"], case["head_dim"], state["q"].dtype)
        state["workspace"] = torch.empty(eg.engram_attn_workspace_size(state["desc"]), dtype=torch.uint8, device="cuda")
    desc, q, k, v, cu = state["desc"], state["q"], state["k"], state["v"], state["cu"]
    if case["op"] == "prompt":
        eg.engram_attn_prompt(desc, q, k, v, cu, state["out"], workspace=state["workspace"])
        return {"out": state["out"]}
    paged = (cu, state["kv_len"], state["table"], state["k_cache"], state["v_cache"])
    if case["op"] == "append":
        eg.engram_kv_append(desc, k, v, *paged)
        return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    eg.engram_attn_paged(desc, q, *paged, state["out"], state["max_q"], workspace=state["workspace"])
    return {"out": state["out"]}


def exact(case, seed):
    """Sequence by sequence and head by head in 64 bits; keys are fetched position by position
    through the page table, and the softmax goes through the logarithm of its sum."""
    s = prepare(case, seed)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    lens = _lens(case["lens"] if case["op"] == "prompt" else case["q_lens"])
    kv_lens = lens if case["op"] == "prompt" else _lens(case["kv_lens"])
    if 4 * d * h * sum(n * m for n, m in zip(lens, kv_lens)) > 6e12:
        return None
    out = torch.zeros((sum(lens), h, d), dtype=torch.float64, device="cuda")
    row = 0
    for j, (n, m) in enumerate(zip(lens, kv_lens)):
        if case["op"] != "prompt":
            pos = torch.arange(m, device="cuda")
            page, slot = s["table"][j].long()[torch.div(pos, case["page"], rounding_mode="floor")], pos % case["page"]
        if case["op"] == "append":
            s["k_cache"].index_put_((page[m - n:], slot[m - n:]), s["k"][row:row + n])
            s["v_cache"].index_put_((page[m - n:], slot[m - n:]), s["v"][row:row + n])
            row += n
            continue
        for c in range(hk):
            if case["op"] == "prompt":
                k, v = s["k"][row:row + n, c].double(), s["v"][row:row + n, c].double()
            else:
                k, v = s["k_cache"][page, slot, c].double(), s["v_cache"][page, slot, c].double()
            for head in range(c * (h // hk), (c + 1) * (h // hk)):
                for r in range(0, n, 2048):
                    e = min(n, r + 2048)
                    seen = m - n + e  # the last of these queries sees this many keys
                    z = s["q"][row + r:row + e, head].double() @ k[:seen].T / d ** 0.5
                    z.add_(torch.full_like(z, -math.inf).triu_(m - n + r + 1))
                    out[row + r:row + e, head] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v[:seen]
        row += n
    if case["op"] == "append":
        return {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    return {"out": out}
