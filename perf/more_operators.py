"""The cases on which the pass of whole prompts through a layer is measured.

Three operators, for prompts of many tokens next to the mat-vecs and the paged cache that serve
a few tokens a step:

* gemm       y = f(W x + bias) + residual for block-quantized W and many tokens
* experts    the same product grouped by expert: ragged numbers of rows per expert
* attention  causal attention of packed prompts of different lengths, grouped heads

``run`` computes each either in its plain form (elementary torch operations in fp32) or, with
``own``, through the library's calls.

Weights are in the library's device layout.  A row is a run of steps; a step is 512 bytes of
codes and then the scales of those codes, the last one shorter and padded to 16 bytes:

    q8_0         codes q + 128;  fp16 d per 32;            w = q d
    q4_0         nibbles;        fp16 d per 32;            w = (q - 8) d
    affine4_g64  nibbles;        fp16 s, fp16 b per 64;    w = q s + b
    q5_0         low nibbles;    uint32 fifth bits, fp16 d per 32 (6 bytes), the fifth bit of
                 element e at bit 8 (e % 8 / 2) + 2 (e / 8) + e % 2;    w = (q - 16) d
    bf16         bf16
"""
from __future__ import annotations

import math
import random

import torch

own = False

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = {"q8_0": 32, "q4_0": 32, "affine4_g64": 64, "q5_0": 32, "bf16": 256}
CODES = {"q8_0": 1.0, "q4_0": 0.5, "affine4_g64": 0.5, "q5_0": 0.5, "bf16": 2.0}           # bytes of a weight
SCALES = {"q8_0": 2, "q4_0": 2, "affine4_g64": 4, "q5_0": 6, "bf16": 0}                    # bytes of a block


# ------------------------------------------------------------------------------------ cases

def listed():
    H = {"heads": 48, "kv_heads": 16, "dim": 128}
    G4 = {"heads": 32, "kv_heads": 8, "dim": 128}
    E = {"n_experts": 512, "topk": 10, "fmt": "q8_0", "routing": 1}
    return [
        # a handful of requests' new tokens through the output projection: latency
        {"name": "gemm few", "op": "gemm", "fmt": "q8_0", "n_out": 2560, "n_in": 6144, "ntok": 17, "act": "f32", "f": "none", "bias": False, "residual": True},
        # a served batch of decode steps through a projection with bias and activation
        {"name": "gemm batch", "op": "gemm", "fmt": "q4_0", "n_out": 8192, "n_in": 2560, "ntok": 129, "act": "bf16", "f": "gelu", "bias": True, "residual": False},
        # a prompt in fp32 through the gate and up projections
        {"name": "gemm gate up fp32", "op": "gemm", "fmt": "q8_0", "n_out": 12288, "n_in": 2560, "ntok": 2047, "act": "f32", "f": "swiglu", "bias": False, "residual": False},
        # the largest: a long prompt's query, key and value heads
        {"name": "gemm prompt", "op": "gemm", "fmt": "q8_0", "n_out": 10240, "n_in": 2560, "ntok": 8191, "act": "bf16", "f": "none", "bias": False, "residual": False},
        # routed experts, a short prompt: about one row an expert
        {"name": "experts few", "op": "experts", **E, "n_out": 1280, "n_in": 2560, "ntok": 61, "act": "bf16", "f": "swiglu", "gather": True},
        # routed experts, a prompt: about 40 rows an expert
        {"name": "experts gate up", "op": "experts", **E, "n_out": 1280, "n_in": 2560, "ntok": 2048, "act": "bf16", "f": "swiglu", "gather": True},
        # the down projection of a shorter one in fp32, rows by slot
        {"name": "experts down fp32", "op": "experts", **E, "n_out": 2560, "n_in": 640, "ntok": 700, "act": "f32", "f": "none", "gather": False},
        # a short question: latency
        {"name": "attend question", "op": "attention", **H, "n_seq": 1, "longest": 77, "act": "f32", "window": 0, "lens": 1},
        # many prompts of different lengths in one call
        {"name": "attend packed", "op": "attention", **G4, "n_seq": 60, "longest": 1500, "act": "bf16", "window": 0, "lens": 2},
        # heads of 256 with a sliding window
        {"name": "attend window", "op": "attention", "heads": 24, "kv_heads": 4, "dim": 256, "n_seq": 5, "longest": 5000, "act": "bf16", "window": 1024, "lens": 3},
        # a prompt with fp32 activations
        {"name": "attend fp32", "op": "attention", **G4, "n_seq": 2, "longest": 3500, "act": "f32", "window": 0, "lens": 4},
        # one long prompt
        {"name": "attend prompt", "op": "attention", **H, "n_seq": 1, "longest": 8191, "act": "bf16", "window": 0, "lens": 5},
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "experts", "experts", "attention", "attention", "attention"])
    fmt, act = rng.choice(list(BLOCK)), rng.choice(["f32", "bf16", "bf16"])
    f = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "swiglu"])
    unit = 64 if fmt == "affine4_g64" else 32
    if op == "gemm":
        n_in, n_out = unit * log_int(rng, 1, 8192 // unit), log_int(rng, 1, 16384)
        ntok = log_int(rng, 1, max(1, min(8191, 8191 * 10240 * 2560 // (n_in * n_out))))
        return {"op": op, "fmt": fmt, "n_out": n_out + n_out % 2 if f == "swiglu" else n_out, "n_in": n_in, "ntok": ntok, "act": act, "f": f,
                "bias": rng.random() < 0.4, "residual": rng.random() < 0.4}
    if op == "experts":
        n = log_int(rng, 1, 512)
        n_in = unit * log_int(rng, 1, 4096 // unit)
        n_out = 2 * log_int(rng, 1, max(1, min(2048, 512 * 1280 * 2560 // (n * n_in * 2))))
        topk = rng.randint(1, min(n, 10))
        return {"op": op, "n_experts": n, "topk": topk, "fmt": fmt, "routing": rng.randrange(1 << 30), "n_out": n_out, "n_in": n_in,
                "ntok": log_int(rng, 1, 2048), "act": act, "f": f, "gather": rng.random() < 0.6}
    kv, group, dim = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([64, 128, 128, 256])
    longest = log_int(rng, 1, min(8191, int(math.sqrt(48 * 8191 * 8191 * 128 / (kv * group * dim)))))
    n_seq = log_int(rng, 1, max(1, min(128, 48 * 8191 * 8191 * 128 // (kv * group * dim * longest * longest))))
    n_seq = max(1, min(n_seq, 100_000_000 // (longest * (group + 2) * kv * dim)))
    return {"op": op, "heads": kv * group, "kv_heads": kv, "dim": dim, "n_seq": n_seq, "longest": longest, "act": act,
            "window": rng.choice([0, 0, log_int(rng, 1, 4096)]), "lens": rng.randrange(1 << 30)}


def lengths(case):
    """Tokens of every prompt: fixed by the case alone, the longest among them."""
    rng = random.Random(case["lens"])
    n, longest = case["n_seq"], case["longest"]
    got = [log_int(rng, max(1, longest // 16), longest) for _ in range(n)]
    got[rng.randrange(n)] = longest
    return got


def routing(case):
    """Rows of every expert: fixed by the case alone.  An expert's popularity is drawn, a token picks topk."""
    rng = random.Random(case["routing"])
    n = case["n_experts"]
    weight = [math.exp(rng.gauss(0.0, 0.5)) for _ in range(n)]
    counts = [0] * n
    for _ in range(case["ntok"]):
        keys = sorted(range(n), key=lambda e: rng.expovariate(weight[e]))[:case["topk"]]
        for e in keys:
            counts[e] += 1
    return counts


# ------------------------------------------------------------------------------------ inputs

def quantize(fmt, w):
    """Codes (bytes) and scales (bytes) of the rows of ``w`` [n, n_in], fp32."""
    n = w.shape[0]
    if fmt == "bf16":
        return w.bfloat16().view(torch.uint8).view(n, -1), w.new_zeros(n, 0, dtype=torch.uint8)
    b = w.unflatten(1, (-1, BLOCK[fmt]))
    if fmt == "affine4_g64":
        lo = b.amin(-1, keepdim=True).half().float()
        s = ((b.amax(-1, keepdim=True) - b.amin(-1, keepdim=True)) / 15).half().float()
        q = ((b - lo) / s.clamp(min=1e-30)).round().clamp(0, 15)
        scales = torch.cat([s, lo], -1).half().view(torch.uint8)
    else:
        steps = {"q8_0": 127, "q4_0": 8, "q5_0": 16}[fmt]
        m = b.gather(-1, b.abs().argmax(-1, keepdim=True))
        d = m.abs() / 127 if fmt == "q8_0" else m / -steps
        q = (b / torch.where(d == 0, torch.ones_like(d), d)).round()
        q = q.clamp(-127, 127) + 128 if fmt == "q8_0" else (q + steps).clamp(0, 2 * steps - 1)
        scales = d.half().view(torch.uint8)
    q = q.to(torch.uint8)
    if fmt == "q8_0":
        return q.flatten(1), scales.flatten(1)
    if fmt == "q5_0":
        e = torch.arange(32, device=w.device)
        bit = ((q >> 4).long() << (8 * (e % 8 // 2) + 2 * (e // 8) + e % 2)).sum(-1, keepdim=True)
        fifth = torch.cat([(bit >> s) & 255 for s in (0, 8, 16, 24)], -1).to(torch.uint8)
        scales = torch.cat([fifth, scales], -1)
        q = q & 15
    q = q.flatten(1)
    return q[:, 0::2] | (q[:, 1::2] << 4), scales.flatten(1)


def layout(fmt, codes, scales):
    """Rows of steps, [n, row bytes]."""
    n, C = codes.shape
    per = int(512 / CODES[fmt]) // BLOCK[fmt] * SCALES[fmt]
    full = C // 512
    parts = []
    if full:
        parts.append(torch.cat([codes[:, :full * 512].reshape(n, full, 512), scales[:, :full * per].reshape(n, full, per)], 2).flatten(1))
    if C % 512:
        last = torch.cat([codes[:, full * 512:], scales[:, full * per:]], 1)
        parts.append(torch.nn.functional.pad(last, (0, -last.shape[1] % 16)))
    return torch.cat(parts, 1)


def weights(fmt, n_out, n_in, g, dev):
    """The packed bytes of n_out rows drawn from N(0, 0.02)."""
    rows = []
    step = max(1, (1 << 27) // n_in)
    for r in range(0, n_out, step):
        w = torch.randn(min(step, n_out - r), n_in, generator=g, device=dev) * 0.02
        rows.append(layout(fmt, *quantize(fmt, w)))
    return torch.cat(rows)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    act = ACT[case["act"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def tokens(n, width):
        return (normal(n, width) * (0.5 + torch.rand(n, 1, generator=g, device=dev))).to(act)

    if case["op"] == "attention":
        Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        lens = lengths(case)
        n = sum(lens)
        # one row per token as the projection writes it: query, key and value heads
        qkv = normal(n, Hq + 2 * Hk, D).to(act)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["cu_seq"] = ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["longest"], s["scale"] = max(lens), D ** -0.5
        s["out"] = torch.zeros(n, Hq, D, dtype=act, device=dev)
        s["lse"] = torch.zeros(n, Hq, device=dev)
    else:
        n_out, n_in, n_slots = case["n_out"], case["n_in"], case["ntok"]
        if case["op"] == "experts":
            counts = routing(case)
            n_slots = sum(counts)
            s["offsets"] = ints([sum(counts[:i]) for i in range(len(counts) + 1)])
            s["most"] = max(counts)
            s["rows"] = None
            n_x = n_slots
            if case["gather"]:       # any token may stand in any expert's rows
                n_x = case["ntok"]
                s["rows"] = torch.randint(0, n_x, (n_slots,), generator=g, device=dev).int()
            s["x"] = tokens(n_x, n_in)
            s["W"] = weights(case["fmt"], n_out * case["n_experts"], n_in, g, dev)
        else:
            s["x"] = tokens(n_slots, n_in)
            s["W"] = weights(case["fmt"], n_out, n_in, g, dev)
            s["bias"] = normal(n_out) * 0.5 if case["bias"] else None
        width = n_out // 2 if case["f"] == "swiglu" else n_out
        if case["op"] == "gemm":
            s["residual"] = normal(n_slots, width).to(act) if case["residual"] else None
        s["y"] = torch.zeros(n_slots, width, dtype=act, device=dev)
    if own:   # the workspace that a serving program makes once
        import block_quantized_token_format_gb300 as qg
        if case["op"] == "attention":
            size = qg.qg_prompt_attention_workspace_bytes(case["act"], n, Hq, Hk, D)
        else:
            size = qg.qgemm_workspace_bytes(case["fmt"], case["act"], n_out, n_in, n_slots, case.get("n_experts", 1))
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return (run_own if own else PLAIN[state["case"]["op"]])(state)


def run_own(s):
    import block_quantized_token_format_gb300 as qg
    c = s["case"]
    if c["op"] == "gemm":
        qg.qgemm(c["fmt"], s["W"], c["n_out"], c["n_in"], s["x"], s["y"], s["workspace"], bias=s["bias"], activation=c["f"], residual=s["residual"])
        return s["y"]
    if c["op"] == "experts":
        qg.qgemm_experts(c["fmt"], s["W"], c["n_experts"], c["n_out"], c["n_in"], s["x"], s["offsets"], s["y"], s["workspace"], rows=s["rows"],
                         activation=c["f"])
        return s["y"]
    qg.qg_prompt_attention(s["q"], s["k"], s["v"], s["cu_seq"], s["out"], s["workspace"], scale=s["scale"], longest=s["longest"], window=c["window"],
                           lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def blocks(fmt, W, n_in):
    """Codes [rows, blocks, bytes] and scales [rows, blocks, bytes] of packed rows."""
    n = W.shape[0]
    C = int(n_in * CODES[fmt])
    per = int(512 / CODES[fmt]) // BLOCK[fmt] * SCALES[fmt]
    full = C // 512
    steps, last = W[:, :full * (512 + per)].reshape(n, full, 512 + per), W[:, full * (512 + per):]
    codes = torch.cat([steps[..., :512].flatten(1), last[:, :C % 512]], 1)
    scales = torch.cat([steps[..., 512:].flatten(1), last[:, C % 512:C % 512 + C % 512 * per // 512]], 1)
    return codes.view(n, n_in // BLOCK[fmt], -1), scales.view(n, n_in // BLOCK[fmt], -1)


def plain_weights(fmt, W, n_in):
    if fmt == "bf16":
        return W.view(torch.bfloat16)[:, :n_in].float()
    codes, scales = blocks(fmt, W, n_in)
    if fmt == "q8_0":
        return ((codes.float() - 128) * scales.view(torch.float16).float()).flatten(1)
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    if fmt == "q5_0":
        e = torch.arange(32, device=W.device)
        fifth = (scales[..., e % 8 // 2] >> (2 * (e // 8) + e % 2).to(torch.uint8)) & 1
        q, scales = q | (fifth << 4), scales[..., 4:].contiguous()
    d = scales.view(torch.float16).float()
    if fmt == "affine4_g64":
        return (q.float() * d[..., :1] + d[..., 1:]).flatten(1)
    return ((q.float() - (8 if fmt == "q4_0" else 16)) * d).flatten(1)


def activate(v, f):
    if f == "silu":
        return v / (1 + torch.exp(-v))
    if f == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if f == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if f == "swiglu":
        return v[..., 0::2] / (1 + torch.exp(-v[..., 0::2])) * v[..., 1::2]
    return v


def plain_gemm(s):
    c = s["case"]
    v = torch.matmul(s["x"].float(), plain_weights(c["fmt"], s["W"], c["n_in"]).t())
    if s["bias"] is not None:
        v = v + s["bias"]
    v = activate(v, c["f"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(ACT[c["act"]])


def plain_experts(s):
    """All experts' products at once, their rows padded to the most that one has."""
    c = s["case"]
    W = plain_weights(c["fmt"], s["W"], c["n_in"]).view(c["n_experts"], c["n_out"], c["n_in"])
    x = s["x"].float() if s["rows"] is None else s["x"].float()[s["rows"].long()]
    off = s["offsets"].long()
    j = torch.arange(s["most"], device=x.device)
    slot = off[:-1, None] + j
    real = slot < off[1:, None]
    v = torch.bmm(x[slot.clamp(max=x.shape[0] - 1)], W.transpose(1, 2))[real]
    return activate(v, c["f"]).to(ACT[c["act"]])


def plain_attention(s):
    """Every prompt padded to the longest."""
    c = s["case"]
    Hq, Hk, D, n, L = c["heads"], c["kv_heads"], c["dim"], c["n_seq"], s["longest"]
    cu = s["cu_seq"].long()
    j = torch.arange(L, device=cu.device)
    real = j < (cu[1:] - cu[:-1])[:, None]
    tok = (cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][tok].float().view(n, L, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).flatten(2, 3)      # [n, Hk, group L, D]
    k, v = s["k"][tok].float().transpose(1, 2), s["v"][tok].float().transpose(1, 2)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    hidden = j > j[:, None]
    if c["window"]:
        hidden |= j <= (j - c["window"])[:, None]
    score.view(n, Hk, Hq // Hk, L, L).masked_fill_(hidden, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out, lse = torch.matmul(p, v) / total, top + torch.log(total)

    def rows(x):
        return x.view(n, Hk, Hq // Hk, L, -1).permute(0, 3, 1, 2, 4)[real].flatten(1, 2)

    return {"out": rows(out).to(ACT[c["act"]]), "lse": rows(lse).squeeze(-1)}


PLAIN = {"gemm": plain_gemm, "experts": plain_experts, "attention": plain_attention}


# ------------------------------------------------------------------------------------ what it takes

def work(case):
    size = 4 if case["act"] == "f32" else 2
    if case["op"] == "attention":
        Hq, Hk, D, w = case["heads"], case["kv_heads"], case["dim"], case["window"]
        lens = lengths(case)
        pairs = sum(n * (n + 1) // 2 if not w or w >= n else w * (w + 1) // 2 + (n - w) * w for n in lens)
        return {"bytes": sum(lens) * (2 * (Hq + Hk) * D * size + 4 * Hq), "flops": 4 * pairs * Hq * D}
    n_out, n_in, fmt = case["n_out"], case["n_in"], case["fmt"]
    width = n_out // 2 if case["f"] == "swiglu" else n_out
    row = n_in * (CODES[fmt] + SCALES[fmt] / BLOCK[fmt])
    if case["op"] == "experts":
        counts = routing(case)
        n = sum(counts)
        n_x = min(n, case["ntok"]) if case["gather"] else n
        return {"bytes": int(sum(k > 0 for k in counts) * n_out * row) + (n_x * n_in + n * width) * size, "flops": 2 * n * n_out * n_in}
    n = case["ntok"]
    return {"bytes": int(n_out * row) + n * (n_in + width * (2 if case["residual"] else 1)) * size + (4 * n_out if case["bias"] else 0),
            "flops": 2 * n * n_out * n_in}


# ------------------------------------------------------------------------------------ in 64 bits

def exact_weights(fmt, W, rows, n_in):
    """Rows of W, each weight fetched from its own place."""
    W, i = W[rows], torch.arange(n_in, device=W.device)
    if fmt == "bf16":
        return (W[:, 2 * i].int() << 16 | W[:, 2 * i + 1].int() << 24).view(torch.float32).double()
    at = i if fmt == "q8_0" else i // 2
    C = n_in if fmt == "q8_0" else n_in // 2
    step, B = at // 512, BLOCK[fmt]
    per = {"q8_0": 512, "q4_0": 1024, "affine4_g64": 1024, "q5_0": 1024}[fmt]           # weights of a step
    start = step * (512 + per // B * SCALES[fmt])
    scale = start + torch.minimum(torch.full_like(at, 512), C - step * 512) + i % per // B * SCALES[fmt]
    q = W[:, start + at % 512].int()

    def half(offset):
        b = (W[:, scale + offset].int() | W[:, scale + offset + 1].int() << 8)
        return b.to(torch.int16).view(torch.float16).double()

    if fmt == "q8_0":
        return (q - 128).double() * half(0)
    q = (q >> (i % 2 * 4)) & 15
    if fmt == "q4_0":
        return (q - 8).double() * half(0)
    if fmt == "affine4_g64":
        return q.double() * half(0) + half(2)
    e = i % 32
    q = q + (((W[:, scale + e % 8 // 2].int() >> (e // 8 * 2 + e % 2)) & 1) << 4)
    return (q - 16).double() * half(4)


def exact_activation(v, f):
    if f == "swiglu":
        return torch.nn.functional.silu(v[:, ::2]) * v[:, 1::2]
    if f == "silu":
        return torch.nn.functional.silu(v)
    return torch.nn.functional.gelu(v, approximate="tanh" if f == "gelu_tanh" else "none") if f != "none" else v


def exact_attention(s):
    c = s["case"]
    Hq, Hk, D, w = c["heads"], c["kv_heads"], c["dim"], c["window"]
    out = torch.zeros(s["q"].shape[0], Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = out.new_zeros(out.shape[:2])
    cu = s["cu_seq"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k, v = s["k"][a:b, h].double(), s["v"][a:b, h].double()
            for t in range(a, b, 512):
                e = min(b, t + 512)
                first = max(a, t - w + 1) if w else a
                score = torch.einsum("thd,kd->htk", s["q"][t:e, heads].double(), k[first - a:e - a]) * s["scale"]
                pos, key = torch.arange(t, e, device=k.device)[:, None], torch.arange(first, e, device=k.device)
                see = (key <= pos) & ((key > pos - w) if w else True)
                score = torch.where(see, score, -math.inf)
                out[t:e, heads] = torch.einsum("htk,kd->thd", score.softmax(-1), v[first - a:e - a])
                lse[t:e, heads] = score.logsumexp(-1).t()
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return exact_attention(s)
    n_out, n_in, fmt, f = case["n_out"], case["n_in"], case["fmt"], case["f"]
    x = s["x"]
    if case["op"] == "experts":
        off = s["offsets"].tolist()
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=x.device)
        for e in range(case["n_experts"]):
            a, b = off[e], off[e + 1]
            if a < b:
                rows = x[a:b] if s["rows"] is None else x[s["rows"][a:b].long()]
                y[a:b] = exact_activation(rows.double() @ exact_weights(fmt, s["W"], slice(e * n_out, (e + 1) * n_out), n_in).t(), f)
        return y
    step = max(2, (1 << 26) // n_in // 2 * 2)
    y = []
    for r in range(0, n_out, step):
        v = x.double() @ exact_weights(fmt, s["W"], slice(r, r + step), n_in).t()
        if s["bias"] is not None:
            v += s["bias"][r:r + step].double()
        y.append(exact_activation(v, f))
    y = torch.cat(y, 1)
    return y if s["residual"] is None else y + s["residual"].double()
