"""CPU oracle of the attention path over a 4-bit key/value cache -- TEST INFRASTRUCTURE.

Written from the definitions in ``include/qgemv.h`` in plain numpy, with no code of the CUDA
library: block quantizer, byte layout of a cache page, page tables, norm and rotation of
heads, attention.  Arithmetic is fp64 unless a function says otherwise; ``norm_rope32`` and
``kv_blocks`` follow the definition's fp32 operations one by one, because codes (and with
them the cache's bytes) are defined through them.
"""
from __future__ import annotations

import numpy as np

CACHE_MAX = 65280.0
F32 = np.float32


# ------------------------------------------------------------------------------------ blocks

def _to_bf16(x):
    """fp32 -> the nearest bf16 (ties to even), as fp32; finite values only."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    u = (u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return u.view(np.float32)


def kv_blocks(x):
    """Codes (uint8, shape of x) and scales (fp16, last axis / 32) of fp32 values."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    b = x.reshape(-1, 32)
    codes = np.full(b.shape, 8, dtype=np.uint8)
    scale = np.zeros(b.shape[0], dtype=np.float16)
    for i, v in enumerate(b):
        if not np.all(np.isfinite(v)) or np.max(np.abs(v)) > CACHE_MAX:
            scale[i] = np.nan
            continue
        m = v[int(np.argmax(np.abs(v)))]                     # the first of the largest
        d = F32(m / F32(-8))
        if d == 0:
            continue
        scale[i] = np.float16(_to_bf16(np.array([d]))[0])
        t = (v / d).astype(np.float32)
        r = np.trunc(t)
        r = r + np.where(np.abs(t - r) >= F32(0.5), np.sign(t), F32(0))      # half away from zero
        codes[i] = np.clip(r + 8, 0, 15).astype(np.uint8)
    return codes.reshape(x.shape), scale.reshape(x.shape[:-1] + (x.shape[-1] // 32,))


def kv_values(codes, scale):
    """What blocks stand for, fp64."""
    d = np.repeat(np.asarray(scale, dtype=np.float64), 32, axis=-1)
    with np.errstate(invalid="ignore"):
        return (codes.astype(np.float64) - 8.0) * d


# ------------------------------------------------------------------------------------ layout

def record_bytes(D):
    return 18 * D


def pool_bytes(n_pages, page, heads, D):
    return n_pages * heads * (page // 16) * record_bytes(D)


def _record(slot, head, page, heads, D):
    p, t = divmod(int(slot), page)
    return ((p * heads + head) * (page // 16) + t // 16) * record_bytes(D), t % 16


def _places(D, t):
    """For token t of a record: byte and nibble shift of every key and value dim, byte of every scale."""
    G = D // 32
    I = min(G, 4)
    key, val, shift, ks, vs = [], [], [], [], []
    for dim in range(D):
        g, at = divmod(dim, 32)
        s, i = divmod(g, I)
        c, j = divmod(at, 8)
        key.append(((s * 16 + t) * 4 + c) * I * 4 + i * 4 + j // 2)
        r, n = divmod(at, 4)
        val.append(9 * D + ((((s * 2 + t // 8) * 8 + r) * 4 + t // 2 % 4) * I + i) * 4 + t % 2 * 2 + n // 2)
        shift.append(4 * (dim % 2))
    for g in range(G):
        ks.append(8 * D + ((t // 2) * G + g) * 4 + t % 2 * 2)
        vs.append(17 * D + ((t // 2) * G + g) * 4 + t % 2 * 2)
    return (np.array(key), np.array(val), np.array(shift, dtype=np.uint8), np.array(ks), np.array(vs))


def kv_store(pool, slot, head, page, heads, D, k, v):
    """Store one token's key and value (fp32 [D]) of one head."""
    base, t = _record(slot, head, page, heads, D)
    key, val, shift, ks, vs = _places(D, t)
    for x, at, sc in ((k, key, ks), (v, val, vs)):
        codes, scale = kv_blocks(x)
        for dim in range(D):
            b = base + at[dim]
            pool[b] = (pool[b] & ~np.uint8(15 << shift[dim])) | np.uint8(codes[dim] << shift[dim])
        raw = scale.view(np.uint8).reshape(-1, 2)
        for g in range(D // 32):
            pool[base + sc[g]:base + sc[g] + 2] = raw[g]


def kv_load(pool, slots, head, page, heads, D):
    """Keys and values (fp64 [n, D] each) of one head at the given slots."""
    K, V = np.empty((len(slots), D)), np.empty((len(slots), D))
    places = [_places(D, t) for t in range(16)]
    for i, s in enumerate(slots):
        base, t = _record(s, head, page, heads, D)
        key, val, shift, ks, vs = places[t]
        for out, at, sc in ((K, key, ks), (V, val, vs)):
            raw = np.stack([pool[base + sc], pool[base + sc + 1]], 1)
            out[i] = kv_values((pool[base + at] >> shift) & 15, np.ascontiguousarray(raw).view(np.float16)[:, 0])
    return K, V


# ------------------------------------------------------------------------------------ pages

def cache_pages(held, fresh, free, begin, table, page, n_tok):
    """New table, seq_len, cu_new, slots, positions and the free list's new begin."""
    table = np.array(table)
    slots, positions = np.full(n_tok, -1, np.int64), np.full(n_tok, -1, np.int32)
    cu, at, tok = [0], begin, 0
    for r, (h, f) in enumerate(zip(held, fresh)):
        for i in range(-(-h // page), -(-(h + f) // page)):
            table[r, i] = free[at]
            at += 1
        for j in range(f):
            slots[tok] = int(table[r, (h + j) // page]) * page + (h + j) % page
            positions[tok] = h + j
            tok += 1
        cu.append(tok)
    return table, np.array(held) + np.array(fresh), np.array(cu), slots, positions, at


# ------------------------------------------------------------------------------------ heads

def norm_rope(x, weight, eps, positions, cos_sin, unit=False, interleaved=False, norm=True):
    """x [n, heads, D] in fp64."""
    y = np.array(x, dtype=np.float64)
    D = y.shape[-1]
    if norm:
        y = y / np.sqrt((y ** 2).sum(-1, keepdims=True) / D + np.float64(F32(eps)))
        if weight is not None:
            y = y * (np.asarray(weight, np.float64) + (1.0 if unit else 0.0))
    if cos_sin is not None:
        R = cos_sin.shape[1]
        cs = np.asarray(cos_sin, np.float64)[positions][:, None]
        c, s = cs[..., :R // 2], cs[..., R // 2:]
        ia = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
        ib = ia + (1 if interleaved else R // 2)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def norm_rope32(x, weight, eps, positions, cos_sin, unit=False, interleaved=False, norm=True):
    """The same, every fp32 operation rounded as the definition orders them."""
    y = np.array(x, dtype=np.float32)
    D = y.shape[-1]
    if norm:
        s = y * y
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        r = F32(1) / np.sqrt(s * F32(1.0 / D) + F32(eps))
        y = y * r
        if weight is not None:
            w = np.asarray(weight, np.float32)
            y = y * (w + F32(1) if unit else w)
    if cos_sin is not None:
        R = cos_sin.shape[1]
        cs = np.asarray(cos_sin, np.float32)[positions][:, None]
        c, s = cs[..., :R // 2], cs[..., R // 2:]
        ia = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
        ib = ia + (1 if interleaved else R // 2)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ------------------------------------------------------------------------------------ attention

def visible(keys, seq, fresh, j, window=0, bits=None):
    """Which of keys 0..keys-1 the request's new token j sees."""
    k = np.arange(keys)
    pos = seq - fresh + j
    see = (k <= pos) & (k < seq)
    if window:
        see &= k > pos - window
    if bits is not None:
        at = k - (seq - fresh)
        see &= (at < 0) | ((int(bits) >> np.clip(at, 0, 31)) & 1).astype(bool)
    return see


def attention(q, K, V, see, scale):
    """One query row: q [D], keys and values [n, D], see [n] -> (out, lse, p).  Keys and values
    that are not seen take no part, whatever they hold."""
    q, K, V = np.asarray(q, np.float64), K[see], V[see]
    if not see.any():
        return np.zeros(q.shape[0]), -np.inf, np.zeros(0)
    with np.errstate(invalid="ignore", over="ignore"):
        s = scale * (K @ q)
        m = s.max()
        p = np.exp(s - m)
        total = p.sum()
        return (p / total) @ V, m + np.log(total), p / total
