"""A paged key-value cache in eight bits beside the attention sublayer: quantising a chunk's keys and
values as they are written, reading positions back, and attention of new tokens (one each, when
decoding) over the quantised pages.

A row (the head_dim values of one position and key-value head) is held as e4m3 codes with one power of
two, an e8m0 byte, beside them: value = code * 2^(byte - 127).

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


BATCH = [2048 - 29 * (i % 17) for i in range(64)]


def listed():
    return [
        # The new token of one conversation: nothing but latency.
        dict(name="append one", op="append", q_lens="1", kv_lens="512", page=16, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # The new keys and values of the batch that the benchmark decodes.
        dict(name="append batch", op="append", q_lens=_text([1] * 64), kv_lens=_text(BATCH), page=64,
             heads=32, kv_heads=8, head_dim=128, dtype="bf16"),
        # The keys and values of two long chunks, one behind 8192 positions that are there.
        dict(name="append chunks", op="append", q_lens="8192,5003", kv_lens="16384,5003", page=16, heads=32,
             kv_heads=8, head_dim=128, dtype="f16"),
        # A short prefix that goes to another conversation, narrow heads.
        dict(name="read prefix", op="read", q_lens="777", kv_lens="777", page=16, heads=8, kv_heads=2,
             head_dim=64, dtype="f16"),
        # Whole caches leave the pages, for a layer that computes on them in 16 bits.
        dict(name="read caches", op="read", q_lens="20011,0,1,9000,16384,3333", kv_lens="20011,7,900,9000,16384,5000",
             page=64, heads=32, kv_heads=8, head_dim=128, dtype="bf16"),
        # One user decoding early in a conversation: one token over 511 positions, small pages.
        dict(name="decode one", op="attend", q_lens="1", kv_lens="511", page=16, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # The decoding batch: 64 sequences, one token each, about 2048 positions.
        dict(name="decode batch", op="attend", q_lens=_text([1] * 64), kv_lens=_text(BATCH), page=64, heads=32,
             kv_heads=8, head_dim=128, dtype="bf16"),
        # Conversations over very long caches: the cache's bytes and nothing else count.
        dict(name="decode long", op="attend", q_lens="1,1,1,1", kv_lens="131072,100003,131001,70001", page=64,
             heads=64, kv_heads=8, head_dim=128, dtype="bf16"),
        # Narrow heads without grouping, f16, caches of very different lengths.
        dict(name="decode narrow", op="attend", q_lens=_text([1] * 24),
             kv_lens=_text([100 + 611 * (i % 11) + 37 * i for i in range(24)]), page=32, heads=16, kv_heads=16,
             head_dim=64, dtype="f16"),
        # Checking a draft of five tokens for sixteen sequences at once, f16, pages of 48 slots.
        dict(name="verify draft", op="attend", q_lens=_text([5] * 16),
             kv_lens=_text([3000 + 111 * i for i in range(16)]), page=48, heads=32, kv_heads=4, head_dim=128,
             dtype="f16"),
        # A server that mixes a chunk of a long prompt with requests that decode.
        dict(name="chunk mixed", op="attend", q_lens="1024,1,1,300,1,1,1,1",
             kv_lens="9000,4100,700,300,2222,1,6001,3333", page=32, heads=32, kv_heads=8, head_dim=128,
             dtype="bf16"),
        # The last chunk of a long document.
        dict(name="chunk long", op="attend", q_lens="2047", kv_lens="30000", page=64, heads=16, kv_heads=4,
             head_dim=128, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    case = dict(op=rng.choice(["append", "read", "attend", "attend", "attend"]),
                heads=kv_heads * group, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128, 80]),
                dtype=rng.choice(["bf16", "bf16", "f16"]), page=rng.choice([16, 32, 48, 64, 128]))
    n = _log_int(rng, 1, 64)
    if case["op"] != "attend":   # any part of the caches is written or read
        longest = _log_int(rng, 1, 16000)
        kv = [longest] + [_log_int(rng, 1, longest) for _ in range(n - 1)]
        while sum(kv) * kv_heads * case["head_dim"] > 48 << 20 and len(kv) > 1:
            kv.pop()
        q = [m if rng.random() < 0.3 else _log_int(rng, 1, m) for m in kv]
        return dict(case, q_lens=_text(q), kv_lens=_text(kv))
    chunk = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1500)
    longest = _log_int(rng, max(chunk, 16), 120000)
    while n > 1 and (n * longest * kv_heads * case["head_dim"] > 400 << 20 or n * chunk * longest * case["heads"] > 1 << 30):
        n -= 1
    while chunk > 1 and chunk * longest * case["heads"] > 1 << 30:
        chunk = chunk * 3 // 4
    q = [chunk] + [rng.randint(1, chunk) for _ in range(n - 1)]
    kv = [longest] + [max(q[i], _log_int(rng, 1, longest)) for i in range(1, n)]
    return dict(case, q_lens=_text(q), kv_lens=_text(kv))


def _pages(case):
    return [-(-n // case["page"]) for n in _lens(case["kv_lens"])]


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    q, kv = _lens(case["q_lens"]), _lens(case["kv_lens"])
    row = d + 1   # the codes and the scale of one key or value
    if case["op"] != "attend":   # 16-bit rows become codes, or codes 16-bit rows
        return {"bytes": sum(q) * hk * 2 * (2 * d + row), "flops": 0}
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, kv))
    return {"bytes": sum(q) * 2 * h * d * 2 + sum(kv) * 2 * hk * row, "flops": 4 * d * h * pairs}


# ---- the format, in elementary operations on 32 bits

def _power(e):
    """2^e in 32 bits, from its bits: -126 <= e <= 127."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x):
    """Codes and scales of the rows x [..., D]: the scale is the smallest power of two, from 2^-100 on,
    that leaves every value within 448, the largest code; 1 for a row of zeros."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)                       # 448 = 0.875 * 2^9
    e = torch.where(top == 0, torch.zeros_like(e), (e - 9 + (m > 0.875).int()).clamp_min(-100))
    codes = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * _power(scales.int() - 127)[..., None]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    h, hk, d, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    lens = _lens(case["q_lens"])
    total = sum(lens)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    # what a layer's projection leaves: queries, keys and values of a token beside each other, whose
    # sizes differ from token to token
    qkv = torch.randn((total, h + 2 * hk, d), generator=g, device="cuda")
    qkv[:, :h] *= 1.5
    qkv[:, h:] *= torch.exp2(torch.randn((total, 2 * hk, 1), generator=g, device="cuda"))
    qkv = qkv.to(dtype)
    need = _pages(case)
    order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):   # a sequence's pages lie anywhere in the cache
        table[i, :n] = order[at:at + n]
        at += n
    s = dict(case=dict(case), q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:], max_q=max(lens), table=table,
             cu=torch.tensor(starts, dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(_lens(case["kv_lens"]), dtype=torch.int32, device="cuda"),
             max_kv=max(_lens(case["kv_lens"])))
    pages = order.numel()
    step = max(1, (32 << 20) // (page * hk * d))
    for name in ("k", "v"):   # codes [pages, page, heads, D], scales [pages, heads, page]
        codes = torch.empty((pages, page, hk, d), dtype=torch.uint8, device="cuda")
        scales = torch.empty((pages, hk, page), dtype=torch.uint8, device="cuda")
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = torch.randn((n, page, hk, d), generator=g, device="cuda")
            x *= torch.exp2(torch.randn((n, page, hk, 1), generator=g, device="cuda"))
            c, e = _quantise(x.to(dtype))
            codes[i:i + n] = c
            scales[i:i + n] = e.transpose(1, 2)
        s[name + "_cache"], s[name + "_scale"] = codes, scales
        s[name + "_codes"] = codes.view(torch.float8_e4m3fn)   # the same bytes, as what they stand for
    if case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty((total, hk, d), dtype=dtype, device="cuda") for _ in range(2))
    elif case["op"] == "attend":
        s["out"] = torch.empty((total, h, d), dtype=dtype, device="cuda")
    return s


def _rows(s):
    """For each packed token, its sequence, its place in it, and its position in the cache."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    n = cu[1:] - cu[:-1]
    return b, t - cu[b], s["kv_len"].long()[b] - n[b] + t - cu[b]


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


def _outputs(s):
    op = s["case"]["op"]
    if op == "append":
        return {"k": s["k_codes"], "v": s["v_codes"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return {"k": s["k_out"], "v": s["v_out"]} if op == "read" else {"out": s["out"]}


def _plain(s):
    case = s["case"]
    b, i, at = _rows(s)
    if case["op"] != "attend":
        page, slot = s["table"][b, at // case["page"]].long(), at % case["page"]
        if case["op"] == "append":
            s["k_cache"][page, slot], s["k_scale"][page, :, slot] = _quantise(s["k"])
            s["v_cache"][page, slot], s["v_scale"][page, :, slot] = _quantise(s["v"])
        else:
            s["k_out"].copy_(_values(s["k_cache"][page, slot], s["k_scale"][page, :, slot]))
            s["v_out"].copy_(_values(s["v_cache"][page, slot], s["v_scale"][page, :, slot]))
        return _outputs(s)
    q = s["q"]
    n = s["cu"].numel() - 1
    qp = torch.zeros((n, s["max_q"]) + q.shape[1:], dtype=torch.float32, device=q.device)
    qp[b, i] = q.float()
    table = s["table"].long()
    kp = _values(s["k_cache"][table], s["k_scale"][table].transpose(2, 3)).flatten(1, 2)[:, :s["max_kv"]]
    vp = _values(s["v_cache"][table], s["v_scale"][table].transpose(2, 3)).flatten(1, 2)[:, :s["max_kv"]]
    last = s["kv_len"] - (s["cu"][1:] - s["cu"][:-1])
    t = torch.arange(s["max_q"], device=q.device)
    ok = torch.arange(s["max_kv"], device=q.device)[None, None] <= (last[:, None] + t[None, :])[:, :, None]
    o = _attend(qp, kp, vp, ok, 1.0 / math.sqrt(case["head_dim"]))
    s["out"].copy_(o[b, i])
    return _outputs(s)


def run(state):
    if not own:
        return _plain(state)
    import deepseek_v4_engram_gb300 as eg
    case = state["case"]
    if "desc" not in state:   # the plan and the scratch that a program keeps for a layer
        state["desc"] = eg.make_attn_desc(case["heads"], case["kv_heads"], case["head_dim"], state["q"].dtype)
        state["workspace"] = torch.empty(eg.engram_attn_workspace_size(state["desc"]), dtype=torch.uint8, device="cuda")
    desc = state["desc"]
    paged = (state["cu"], state["kv_len"], state["table"], state["k_cache"], state["v_cache"], state["k_scale"],
             state["v_scale"])
    if case["op"] == "append":
        eg.engram_kv_append_fp8(desc, state["k"], state["v"], *paged)
    elif case["op"] == "read":
        eg.engram_kv_read_fp8(desc, *paged, state["k_out"], state["v_out"])
    else:
        eg.engram_attn_paged_fp8(desc, state["q"], *paged, state["out"], state["max_q"], workspace=state["workspace"])
    return _outputs(state)


# ---- the same from the definition, in 64 bits

def _code_values():
    """The 256 values of e4m3, from its fields: sign, four bits of exponent, three of fraction."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        a = math.nan if c & 127 == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-a if c & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _scale_values():
    return torch.tensor([2.0 ** (c - 127) for c in range(255)] + [math.nan], dtype=torch.float64, device="cuda")


def _exact_quantise(x):
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.full_like(top, 2.0 ** -100)
    for e in range(-100, 121):   # the first power of two for which no value exceeds the largest code
        scale = torch.where(top > 448 * scale, torch.full_like(scale, 2.0 ** (e + 1)), scale)
    scale = torch.where(top == 0, torch.ones_like(scale), scale)
    y = x / scale
    # spacing of the codes around y: an eighth of its power of two, at least 2^-9
    power = (y.abs().clamp_min(2.0 ** -6).view(torch.int64) & (0x7FF << 52)).view(torch.float64)
    quantum = power / 8
    return torch.round(y / quantum) * quantum, scale.squeeze(-1)


def exact(case, seed):
    """Position by position through the page table, head by head; the softmax goes through the
    logarithm of its sum. None in the place of the scales, which are whole numbers."""
    s = prepare(case, seed)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    lens, kv_lens = _lens(case["q_lens"]), _lens(case["kv_lens"])
    value, scale = _code_values(), _scale_values()
    if case["op"] == "attend" and 4 * d * h * sum(n * m for n, m in zip(lens, kv_lens)) > 6e12:
        return None
    found = {n: value[s[n + "_cache"].long()] for n in ("k", "v")} if case["op"] == "append" else {
        n: torch.zeros((sum(lens), hk, d), dtype=torch.float64, device="cuda") for n in ("k", "v")}
    out = torch.zeros((sum(lens), h, d), dtype=torch.float64, device="cuda")
    row = 0
    for j, (n, m) in enumerate(zip(lens, kv_lens)):
        pos = torch.arange(m, device="cuda")
        page, slot = s["table"][j].long()[torch.div(pos, case["page"], rounding_mode="floor")], pos % case["page"]
        if case["op"] == "append":
            for name in ("k", "v"):
                found[name][page[m - n:], slot[m - n:]] = _exact_quantise(s[name][row:row + n])[0]
            row += n
            continue
        for c in range(hk):
            k, v = (value[s[x + "_cache"][page, slot, c].long()] *
                    scale[s[x + "_scale"][page, c, slot].long()][:, None] for x in ("k", "v"))
            if case["op"] == "read":
                found["k"][row:row + n, c], found["v"][row:row + n, c] = k[m - n:], v[m - n:]
                continue
            for head in range(c * (h // hk), (c + 1) * (h // hk)):
                for r in range(0, n, 2048):
                    e = min(n, r + 2048)
                    seen = m - n + e   # the last of these queries sees this many keys
                    z = s["q"][row + r:row + e, head].double() @ k[:seen].T / d ** 0.5
                    z.add_(torch.full_like(z, -math.inf).triu_(m - n + r + 1))
                    out[row + r:row + e, head] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ v[:seen]
        row += n
    if case["op"] == "attend":
        return {"out": out}
    return dict(found, k_scale=None, v_scale=None) if case["op"] == "append" else found
