"""The cases on which the attention path of a decode or verify step is measured.

Four operators, from request lengths to attention outputs over a paged cache that holds
keys and values in 4 bits:

* pages      block table, slots and positions of a step's new tokens from request lengths
* norm_rope  RMS norm of every query and key head and the position rotation
* append     the same, then keys and values quantized into the cache
* attention  attention of the new tokens over the cache

``run`` computes each either in its plain form (elementary torch operations in fp32) or,
with ``own``, through the library's calls.

The cache is a pool of pages of ``page`` tokens.  A page holds, per key/value head, page/16
records of 16 tokens; a record of 18 * dim bytes holds the keys' codes, the keys' scales,
the values' codes and the values' scales (G = dim / 32 blocks of 32 per token and head, in
G / I sets of I = min(G, 4); block g is g % I of set g / I):

    key codes    [set][16 tokens][4 c][I] uint32: nibble j of a word is dim 32 g + 8 c + j
    scales       [8 token pairs][G g][2 tokens] fp16
    value codes  [set][2 halves][8 r][4 pairs of the half][I][2 tokens] uint16: nibble j is
                 dim 32 g + 4 r + j

A value is (nibble - 8) * scale.
"""
from __future__ import annotations

import math
import random

import torch

own = False

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
BASE, EPS = 1.0e6, 1.0e-6


# ------------------------------------------------------------------------------------ cases

# Heads: the 2560 -> 10240 projection is 48 query, 16 key and 16 value heads of 128 (its
# output projection is 6144 -> 2560); the others are generic grouped-query layouts.
def listed():
    H = {"heads": 48, "kv_heads": 16, "dim": 128}
    G4 = {"heads": 32, "kv_heads": 8, "dim": 128}
    G8 = {"heads": 64, "kv_heads": 8, "dim": 128}
    return [
        # a decode step of a small batch: one new token each, most without a new page
        {"name": "pages decode", "op": "pages", "n_req": 48, "longest": 30000, "spread": "ragged", "new": 1, "page": 64, "lens": 1},
        # prompts enter: every token of 40 requests gets its slot
        {"name": "pages prompts", "op": "pages", "n_req": 40, "longest": 0, "spread": "ragged", "new": 16001, "page": 16, "lens": 2},
        # one verify step of one sequence: 4 tokens, the framework's largest
        {"name": "norm_rope verify", "op": "norm_rope", **H, "tokens": 4, "rot": 128, "act": "f32", "interleaved": False, "unit": False},
        # a prompt chunk in bf16, part of each head rotated
        {"name": "norm_rope chunk", "op": "norm_rope", **G8, "tokens": 8191, "rot": 64, "act": "bf16", "interleaved": False, "unit": True},
        # the same verify step, with its keys and values stored
        {"name": "append verify", "op": "append", **H, "tokens": 4, "rot": 128, "act": "f32", "interleaved": False, "unit": False, "page": 64},
        # a prompt chunk stored
        {"name": "append chunk", "op": "append", **G4, "tokens": 4100, "rot": 128, "act": "f32", "interleaved": True, "unit": False, "page": 32},
        # decode of one sequence, short context: latency
        {"name": "attend short", "op": "attention", **H, "n_req": 1, "longest": 777, "spread": "even", "new": 1, "page": 64, "window": 0, "tree": False, "act": "f32", "lens": 3},
        # verify of 4 tokens of one sequence at 32 k
        {"name": "attend verify", "op": "attention", **H, "n_req": 1, "longest": 32771, "spread": "even", "new": 4, "page": 64, "window": 0, "tree": False, "act": "f32", "lens": 4},
        # decode of one sequence with a long cache
        {"name": "attend long", "op": "attention", **G4, "n_req": 1, "longest": 262100, "spread": "even", "new": 1, "page": 64, "window": 0, "tree": False, "act": "f32", "lens": 5},
        # a tree of drafts for 12 sequences, heads of 256, in a sliding window
        {"name": "attend tree window", "op": "attention", "heads": 24, "kv_heads": 4, "dim": 256, "n_req": 12, "longest": 20000, "spread": "ragged", "new": 4, "page": 16, "window": 8192, "tree": True, "act": "f32", "lens": 6},
        # a served batch in bf16, ragged
        {"name": "attend batch", "op": "attention", **G8, "n_req": 64, "longest": 16384, "spread": "ragged", "new": 1, "page": 64, "window": 0, "tree": False, "act": "bf16", "lens": 7},
        # the largest: a served batch with fp32 activations
        {"name": "attend large batch", "op": "attention", **G4, "n_req": 96, "longest": 20000, "spread": "ragged", "new": 1, "page": 32, "window": 0, "tree": False, "act": "f32", "lens": 8},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["pages", "norm_rope", "append", "attention", "attention", "attention"])
    kv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8])
    dim = rng.choice([64, 128, 128, 256])
    page, act = rng.choice([16, 32, 48, 64, 128]), rng.choice(["f32", "f32", "bf16"])
    lens = rng.randrange(1 << 30)
    if op == "pages":
        if rng.random() < 0.5:
            return {"op": op, "n_req": log_int(rng, 1, 1024), "longest": log_int(rng, 1, 100000), "spread": "ragged", "new": rng.randint(1, 4), "page": page, "lens": lens}
        n = log_int(rng, 1, 64)
        return {"op": op, "n_req": n, "longest": rng.choice([0, 999]), "spread": "ragged", "new": log_int(rng, 2, 400000 // n), "page": page, "lens": lens}
    if op in ("norm_rope", "append"):
        most = max(1, 6144 * 64 * 128 // ((group + 2) * kv * dim))
        c = {"op": op, "heads": kv * group, "kv_heads": kv, "dim": dim, "tokens": log_int(rng, 1, min(8192, most)),
             "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "act": act, "interleaved": rng.random() < 0.3, "unit": rng.random() < 0.3}
        return {**c, "page": page} if op == "append" else c
    keys = log_int(rng, 1, max(2, 250_000_000 // (kv * dim)))       # cached tokens of all requests
    n = min(keys, log_int(rng, 1, 128))
    longest = max(1, min(keys // n, 4_000_000_000 // (n * kv * dim * 4)))
    return {"op": op, "heads": kv * group, "kv_heads": kv, "dim": dim, "n_req": n, "longest": longest,
            "spread": rng.choice(["even", "ragged"]), "new": rng.choice([1, 1, 2, 3, 4]), "page": page,
            "window": rng.choice([0, 0, 0, log_int(rng, 1, 8192)]), "tree": rng.random() < 0.25, "act": act, "lens": lens}


def lengths(case):
    """(tokens held before the step, new tokens) of every request: fixed by the case alone."""
    rng = random.Random(case["lens"])
    n, longest, new = case["n_req"], case["longest"], case["new"]
    if case["spread"] == "even":
        return [longest] * n, [new] * n
    held = [0 if longest == 0 or rng.random() < 0.05 else log_int(rng, max(1, longest // 16), longest) for _ in range(n)]
    held[rng.randrange(n)] = longest
    fresh = [new if new <= 4 else log_int(rng, max(1, new // 8), new) for _ in range(n)]
    return held, fresh


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------ inputs

def quantize(x):
    """Codes 0..15 and scales (fp32) of the blocks of 32 along the last axis of ``x``."""
    b = x.float().unflatten(-1, (-1, 32))
    at = b.abs().argmax(-1, keepdim=True)                              # the first of the largest
    m = b.gather(-1, at)
    d = m / -8
    t = b / torch.where(m == 0, torch.ones_like(d), d)
    a = t.abs()
    f = a.floor()
    t = torch.where(m == 0, torch.zeros_like(t), (f + ((a - f) >= 0.5)) * t.sign())
    return (t + 8).clamp(0, 15).to(torch.uint8).flatten(-2), d.bfloat16().to(torch.float16).squeeze(-1)


def key_bytes(codes):
    """[..., D] codes -> [..., set, 4 c, I, 4] bytes: a token's words."""
    D = codes.shape[-1]
    w = codes.unflatten(-1, (-1, min(D // 32, 4), 4, 8)).transpose(-3, -2)      # [..., set, c, i, j]
    return w[..., 0::2] | (w[..., 1::2] << 4)


def value_bytes(codes):
    """[..., D] codes -> [..., set, 8 r, I, 2] bytes: a token's halfwords."""
    D = codes.shape[-1]
    w = codes.unflatten(-1, (-1, min(D // 32, 4), 8, 4)).transpose(-3, -2)      # [..., set, r, i, j]
    return w[..., 0::2] | (w[..., 1::2] << 4)


def records(k, v):
    """Keys and values [n, 16, D] (fp32) -> their records, [n, 18 * D] bytes."""
    n, _, D = k.shape
    G = D // 32

    def scales(d):                                                      # [n, 16, G] -> pairs
        return d.view(n, 8, 2, G).transpose(2, 3).contiguous().view(torch.uint8).view(n, -1)

    kc, kd = quantize(k)
    vc, vd = quantize(v)
    kb = key_bytes(kc).transpose(1, 2)                                 # [n, set, 16, c, i, 4]
    vb = value_bytes(vc).unflatten(1, (2, 4, 2)).permute(0, 4, 1, 5, 2, 6, 3, 7)
    return torch.cat([kb.reshape(n, -1), scales(kd), vb.reshape(n, -1), scales(vd)], 1)


def rotations(n_pos, rot, dev):
    """cos | sin of position * BASE^(-2i / rot), fp32 [n_pos, rot]."""
    f = BASE ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if case["op"] == "pages":
        held, fresh = lengths(case)
        P, n = case["page"], case["n_req"]
        width = max(ceil_div(h + f, P) for h, f in zip(held, fresh)) + 3
        total = sum(ceil_div(h + f, P) for h, f in zip(held, fresh))
        pages = torch.randperm(total + 17, generator=g, device=dev).int()
        counts = ints([ceil_div(h, P) for h in held]).long()
        col = torch.arange(width, device=dev)
        has = col < counts[:, None]
        s["table"] = torch.full((n, width), -1, dtype=torch.int32, device=dev)
        used = int(counts.sum())
        s["table"][has] = pages[:used]
        s["free_pages"] = pages[used:].contiguous()
        s["held"], s["fresh"] = ints(held), ints(fresh)
        s["n_tok"] = sum(fresh)
        s["seq_len"], s["cu_new"] = ints([0] * n), ints([0] * (n + 1))
        s["slots"] = torch.zeros(s["n_tok"], dtype=torch.int64, device=dev)
        s["positions"] = torch.zeros(s["n_tok"], dtype=torch.int32, device=dev)
        s["free_end"] = ints([0])
        return s

    act = ACT[case["act"]]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("norm_rope", "append"):
        n = case["tokens"]
        # one row per token as the projection writes it: query, key and value heads
        qkv = (normal(n, Hq + 2 * Hk, D) * (0.5 + torch.rand(n, Hq + 2 * Hk, 1, generator=g, device=dev))).to(act)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        w = [normal(D) * 0.2 + (0.0 if case["unit"] else 1.0) for _ in range(2)]
        s["q_weight"], s["k_weight"] = w
        first = int(torch.randint(0, 4000, (1,), generator=g, device=dev))
        s["positions"] = (torch.arange(n, device=dev) + first).int()
        s["cos_sin"] = rotations(first + n, case["rot"], dev)
        s["q_out"] = torch.zeros(n, Hq, D, dtype=act, device=dev)
        s["k_out"] = torch.zeros(n, Hk, D, dtype=act, device=dev)
        if case["op"] == "append":
            P = case["page"]
            s["v_out"] = torch.zeros(n, Hk, D, dtype=act, device=dev)
            pages = ceil_div(P - 1 + n, P)
            ids = torch.randperm(pages + 5, generator=g, device=dev)
            at = torch.arange(n, device=dev) + first % P
            s["slots"] = ids[at // P] * P + at % P
            s["n_pages"] = pages + 5
            s["pool"] = torch.zeros(s["n_pages"] * Hk * (P // 16) * 18 * D, dtype=torch.uint8, device=dev)
    else:
        held, fresh = lengths(case)
        P, n = case["page"], case["n_req"]
        per = P // 16
        counts = [ceil_div(h + f, P) for h, f in zip(held, fresh)]
        s["n_pages"] = sum(counts) + 3
        s["pool"] = torch.empty(s["n_pages"] * Hk * per * 18 * D, dtype=torch.uint8, device=dev)
        rows = s["pool"].view(-1, 18 * D)
        step = max(1, (1 << 24) // (16 * D))
        for r0 in range(0, rows.shape[0], step):
            m = min(step, rows.shape[0] - r0)
            rows[r0:r0 + m] = records(normal(m, 16, D), normal(m, 16, D) * 0.7)
        ids = torch.randperm(s["n_pages"], generator=g, device=dev).int()
        c = ints(counts).long()
        s["table"] = torch.full((n, max(counts)), -1, dtype=torch.int32, device=dev)
        s["table"][torch.arange(max(counts), device=dev) < c[:, None]] = ids[:sum(counts)]
        s["seq_len"] = ints([h + f for h, f in zip(held, fresh)])
        s["cu_new"] = ints([sum(fresh[:i]) for i in range(n + 1)])
        s["n_tok"], s["max_new"] = sum(fresh), max(fresh)
        s["q"] = (normal(s["n_tok"], Hq, D) * 1.3).to(act)
        s["scale"] = D ** -0.5
        s["tree"] = None
        if case["tree"]:     # token j descends from itself and a random part of the ones before
            j = ints([i for f in fresh for i in range(f)])
            bits = torch.randint(0, 16, (s["n_tok"],), generator=g, device=dev).int()
            s["tree"] = (bits & ((1 << j) - 1)) | (1 << j)
        s["out"] = torch.zeros(s["n_tok"], Hq, D, dtype=act, device=dev)
        s["lse"] = torch.zeros(s["n_tok"], Hq, device=dev)
    if own:   # the handle and the workspace that a serving program makes once
        import block_quantized_token_format_gb300 as qg
        if case["op"] in ("append", "attention"):
            s["cache"] = qg.qg_cache(s["pool"], s["n_pages"], case["page"], Hk, D)
        if case["op"] == "attention":
            s["workspace"] = torch.zeros(qg.qg_attention_workspace_bytes(Hq, Hk, D), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return (run_own if own else PLAIN[state["case"]["op"]])(state)


def run_own(s):
    import block_quantized_token_format_gb300 as qg
    c = s["case"]
    if c["op"] == "pages":
        qg.qg_cache_pages(s["held"], s["fresh"], s["free_pages"], s["table"], s["seq_len"], s["cu_new"], s["slots"],
                          s["positions"], c["page"], free_end=s["free_end"])
        return {k: s[k] for k in ("table", "seq_len", "cu_new", "slots", "positions", "free_end")}
    if c["op"] == "norm_rope":
        qg.qg_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["cos_sin"], q_weight=s["q_weight"],
                           k_weight=s["k_weight"], eps=EPS, unit_offset=c["unit"], interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        qg.qg_cache_append(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], q_out=s["q_out"], positions=s["positions"],
                           cos_sin=s["cos_sin"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                           unit_offset=c["unit"], interleaved=c["interleaved"], k_back=s["k_out"], v_back=s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "cache": s["pool"]}
    qg.qg_attention(s["cache"], s["q"], s["table"], s["seq_len"], s["cu_new"], s["out"], s["workspace"], scale=s["scale"],
                    max_new=s["max_new"], window=c["window"], span_mask=s["tree"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def plain_pages(s):
    P, held, fresh = s["case"]["page"], s["held"].long(), s["fresh"].long()
    free, table, n, n_tok = s["free_pages"].long(), s["table"], s["case"]["n_req"], s["n_tok"]
    cu = torch.cat([torch.zeros_like(fresh[:1]), fresh.cumsum(0)])
    have = (held + P - 1) // P
    need = (held + fresh + P - 1) // P - have
    off = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)
    dealt = (col >= have[:, None]) & (col < (have + need)[:, None])
    index = (off - have)[:, None] + col
    table.copy_(torch.where(dealt, free[index.clamp(0, free.numel() - 1)], table.long()))
    req = torch.repeat_interleave(torch.arange(n, device=table.device), fresh, output_size=n_tok)
    pos = held[req] + torch.arange(n_tok, device=table.device) - cu[req]
    s["slots"].copy_(table[req, pos // P].long() * P + pos % P)
    s["positions"].copy_(pos)
    s["seq_len"].copy_(held + fresh)
    s["cu_new"].copy_(cu)
    s["free_end"].copy_(need.sum()[None])
    return {k: s[k] for k in ("table", "seq_len", "cu_new", "slots", "positions", "free_end")}


def halved(x):
    return x[..., 0::2] + x[..., 1::2]


def plain_norm_rope(x, weight, s):
    """The norm and rotation of heads x [n, H, D] in fp32; squares are summed pair by pair."""
    c = s["case"]
    x = x.float()
    D, R = c["dim"], c["rot"]
    ss = halved(halved(halved(halved(halved(halved(x * x))))))
    ss = halved(ss) if D > 64 else ss
    ss = halved(ss) if D > 128 else ss
    r = 1.0 / torch.sqrt(ss * (1.0 / D) + EPS)
    y = (x * r) * (weight + 1.0 if c["unit"] else weight)
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :R // 2], cs[..., R // 2:]
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if c["interleaved"] else (y[..., :R // 2], y[..., R // 2:R])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., R:]], -1)


def plain_norm_rope_op(s):
    act = ACT[s["case"]["act"]]
    return {"q": plain_norm_rope(s["q"], s["q_weight"], s).to(act), "k": plain_norm_rope(s["k"], s["k_weight"], s).to(act)}


def plain_append(s):
    c = s["case"]
    act, Hk, D, P = ACT[c["act"]], c["kv_heads"], c["dim"], c["page"]
    G, I = D // 32, min(D // 32, 4)
    q, k, v = plain_norm_rope(s["q"], s["q_weight"], s), plain_norm_rope(s["k"], s["k_weight"], s), s["v"].float()
    kc, kd = quantize(k)
    vc, vd = quantize(v)
    page, rec, t = s["slots"] // P, s["slots"] % P // 16, s["slots"] % 16
    pool = s["pool"].view(-1, Hk, P // 16, 18 * D)

    def part(at, width, *shape):
        return pool[..., at:at + width].unflatten(-1, shape)

    part(0, 8 * D, G // I, 16, 4, I, 4)[page, :, rec, :, t] = key_bytes(kc)
    part(9 * D, 8 * D, G // I, 2, 8, 4, I, 2, 2)[page, :, rec, :, t // 8, :, t // 2 % 4, :, t % 2] = value_bytes(vc)
    for at, d in ((8 * D, kd), (17 * D, vd)):
        part(at, D, 8, G, 2, 2)[page, :, rec, t // 2, :, t % 2] = d.contiguous().view(torch.uint8).view(-1, Hk, G, 2)

    def back(codes, d):
        return ((codes.float() - 8).unflatten(-1, (G, 32)) * d.float()[..., None]).flatten(-2).to(act)

    return {"q": q.to(act), "k": back(kc, kd), "v": back(vc, vd), "cache": s["pool"]}


def nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def plain_cache(s):
    """Keys and values of every request, fp32 [n_req, kv_heads, padded length, D]."""
    c = s["case"]
    Hk, D, P = c["kv_heads"], c["dim"], c["page"]
    G, I = D // 32, min(D // 32, 4)
    rec = s["pool"].view(-1, Hk, P // 16, 18 * D)[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)

    def scales(at):
        d = rec[..., at:at + D].contiguous().view(torch.float16).float()
        return d.unflatten(-1, (8, G, 2)).transpose(-1, -2).reshape(*d.shape[:2], -1, G, 1)

    # [n, head, record, set, 16, c, i, 8] and [n, head, record, set, half, r, pair, i, 2, 4] -> [n, head, token, G, 32]
    k = nibbles(rec[..., :8 * D].unflatten(-1, (G // I, 16, 4, I, 4))).permute(0, 1, 2, 4, 3, 6, 5, 7)
    v = nibbles(rec[..., 9 * D:17 * D].unflatten(-1, (G // I, 2, 8, 4, I, 2, 2))).permute(0, 1, 2, 4, 6, 8, 3, 7, 5, 9)
    k, v = (x.reshape(*x.shape[:2], -1, G, 32) for x in (k, v))
    k = ((k.float() - 8) * scales(8 * D)).flatten(-2)
    v = ((v.float() - 8) * scales(17 * D)).flatten(-2)
    return k, v


def plain_attention(s):
    c = s["case"]
    Hq, Hk, D, n = c["heads"], c["kv_heads"], c["dim"], c["n_req"]
    new, dev = s["max_new"], s["q"].device
    k, v = plain_cache(s)
    cu, seq = s["cu_new"].long(), s["seq_len"].long()
    fresh = cu[1:] - cu[:-1]
    j = torch.arange(new, device=dev)
    real = j < fresh[:, None]
    tok = (cu[:-1, None] + j).clamp(max=s["n_tok"] - 1)                  # [n, new]
    q = s["q"][tok].float().view(n, new, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    key = torch.arange(k.shape[2], device=dev)
    begin = seq - fresh
    pos = begin[:, None] + j
    sees = key <= pos[..., None]                                          # [n, new, keys]
    if c["window"]:
        sees &= key > (pos - c["window"])[..., None]
    if s["tree"] is not None:
        at = key - begin[:, None]
        bit = (s["tree"].long()[tok][..., None] >> at.clamp(0, 62)[:, None]) & 1
        sees &= (at < 0)[:, None] | (bit == 1)
    sees = sees[:, None, :, None].expand(n, 1, new, Hq // Hk, -1).flatten(2, 3)
    score = score.masked_fill(~sees, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + torch.log(total)

    def rows(x):
        return x.unflatten(2, (new, Hq // Hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)[real]

    return {"out": rows(out).to(ACT[c["act"]]), "lse": rows(lse).squeeze(-1)}


PLAIN = {"pages": plain_pages, "norm_rope": plain_norm_rope_op, "append": plain_append, "attention": plain_attention}


# ------------------------------------------------------------------------------------ what it takes

def visible(case):
    """Keys that a request's new tokens see, of all requests."""
    held, fresh = lengths(case)
    w = case["window"]
    return sum(h + f - (max(0, h + 1 - w) if w else 0) for h, f in zip(held, fresh))


def work(case):
    if case["op"] == "pages":
        held, fresh = lengths(case)
        P, n_tok = case["page"], sum(fresh)
        new_pages = sum(ceil_div(h + f, P) - ceil_div(h, P) for h, f in zip(held, fresh))
        return {"bytes": 16 * case["n_req"] + 12 * n_tok + 8 * new_pages, "flops": 0}
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    size = 4 if case["act"] == "f32" else 2
    if case["op"] == "norm_rope":
        n = case["tokens"]
        return {"bytes": n * (2 * (Hq + Hk) * D * size + 4 * case["rot"]), "flops": 7 * n * (Hq + Hk) * D}
    if case["op"] == "append":
        n = case["tokens"]
        return {"bytes": n * (2 * (Hq + 2 * Hk) * D * size + 18 * Hk * D // 16 + 4 * case["rot"] + 8), "flops": n * (7 * Hq + 17 * Hk) * D}
    _, fresh = lengths(case)
    keys, n_tok = visible(case), sum(fresh)
    return {"bytes": keys * Hk * D * 18 // 16 + n_tok * Hq * (2 * D * size + 4), "flops": 4 * case["new"] * keys * Hq * D}


# ------------------------------------------------------------------------------------ in 64 bits

def exact_heads(x, weight, s):
    c, D, R = s["case"], s["case"]["dim"], s["case"]["rot"]
    x = x.double()
    y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * (weight.double() + (1 if c["unit"] else 0))
    cs = s["cos_sin"].double()[s["positions"].long()]
    z = torch.complex(cs[:, :R // 2], cs[:, R // 2:])[:, None]
    first = torch.arange(0, R, 2) if c["interleaved"] else torch.arange(R // 2)
    second = first + (1 if c["interleaved"] else R // 2)
    t = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = t.real.clone(), t.imag.clone()
    return y


def exact_blocks(x):
    """What the cache holds for x, by the definition of a block."""
    b = x.reshape(-1, 32)
    lo, hi = b.min(1).values, b.max(1).values
    m = torch.where(-lo > hi, lo, hi)
    tie = -lo == hi
    m = torch.where(tie & (b.argmin(1) < b.argmax(1)), lo, m)
    d = -m / 8
    t = torch.where(d[:, None] == 0, torch.zeros_like(b), b / d[:, None])
    t = torch.clamp(torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)), -8, 7)
    return (t * d.bfloat16().half().double()[:, None]).view_as(x)


def exact_attention(s):
    """Request by request, each nibble fetched from its own place in the pool."""
    c = s["case"]
    Hq, Hk, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    G, I, dev, pool = D // 32, min(D // 32, 4), s["q"].device, s["pool"]
    half = pool.view(torch.float16)
    dim = torch.arange(D, device=dev)
    g, rest = dim // 32, dim % 32
    shift = dim % 2 * 4
    k_byte = (g // I * 64 + rest // 8) * I * 4 + g % I * 4 + rest % 8 // 2
    v_byte = (g // I * 64 + rest // 4 * 4) * I * 4 + g % I * 4 + rest % 4 // 2
    outs, lses = [], []
    seq, cu = s["seq_len"].tolist(), s["cu_new"].tolist()
    for r in range(c["n_req"]):
        L, n = seq[r], cu[r + 1] - cu[r]
        first = max(0, L - n - c["window"] + 1) if c["window"] else 0
        t = torch.arange(first, L, device=dev)
        page = s["table"][r].long()[t // P]
        head = torch.arange(Hk, device=dev)[:, None]
        rec = (((page * Hk + head) * (P // 16) + t % P // 16) * 18 * D)[..., None]      # [Hk, keys, 1]
        u = (t % 16)[:, None]
        k = ((pool[rec + u * 16 * I + k_byte] >> shift) & 15).double() - 8
        v = ((pool[rec + 9 * D + (u // 8 * 32 + u // 2 % 4) * I * 4 + u % 2 * 2 + v_byte] >> shift) & 15).double() - 8
        sc = (u // 2) * G * 2 + g * 2 + u % 2
        k *= half[(rec + 8 * D) // 2 + sc].double()
        v *= half[(rec + 17 * D) // 2 + sc].double()
        q = s["q"][cu[r]:cu[r + 1]].double().view(n, Hk, Hq // Hk, D).permute(1, 0, 2, 3).reshape(Hk, -1, D)
        score = torch.bmm(q, k.transpose(1, 2)) * s["scale"]
        pos = L - n + torch.arange(n, device=dev)[:, None]
        hide = t > pos
        if c["window"]:
            hide |= t <= pos - c["window"]
        if s["tree"] is not None:
            bits = s["tree"][cu[r]:cu[r + 1]].long()[:, None]
            hide |= (t >= L - n) & ((bits >> (t - (L - n)).clamp(min=0)) % 2 == 0)
        score.view(Hk, n, Hq // Hk, -1).masked_fill_(hide[None, :, None], -math.inf)
        outs.append(torch.bmm(score.softmax(-1), v).view(Hk, n, Hq // Hk, D).permute(1, 0, 2, 3).reshape(n, Hq, D))
        lses.append(score.logsumexp(-1).view(Hk, n, Hq // Hk).permute(1, 0, 2).reshape(n, Hq))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "attention":
        return exact_attention(s)
    q, k = exact_heads(s["q"], s["q_weight"], s), exact_heads(s["k"], s["k_weight"], s)
    if case["op"] == "norm_rope":
        return {"q": q, "k": k}
    return {"q": q, "k": exact_blocks(k), "v": exact_blocks(s["v"].double()), "cache": None}
