"""The attention path's oracle against closed forms, hand-worked blocks and brute force (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as ORC
from oracle import attention_oracle as AO


def test_block_by_hand():
    x = np.zeros(32, np.float32)
    x[3], x[7], x[9] = -4.0, 4.0, 1.25                      # first of the largest magnitude is -4: d = 0.5
    codes, scale = AO.kv_blocks(x)
    assert float(scale[0]) == 0.5
    assert codes[3] == 0 and codes[7] == 15 and codes[0] == 8
    assert codes[9] == 11                                    # 1.25 / 0.5 = 2.5, half away from zero
    assert AO.kv_values(codes, scale)[3] == -4.0 and AO.kv_values(codes, scale)[7] == 3.5


def test_codes_are_those_of_q4_0():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((64, 128)) * np.exp(rng.uniform(-6, 6, (64, 1)))).astype(np.float32)
    codes, _ = AO.kv_blocks(x)
    canon = ORC.quantize("q4_0", x)
    deq = ORC.dequantize("q4_0", canon, 64, 128)
    raw = np.frombuffer(canon.tobytes(), np.uint8).reshape(-1, 18)
    q = np.concatenate([raw[:, 2:] & 15, raw[:, 2:] >> 4], 1)
    assert np.array_equal(q.reshape(64, 128), codes)
    d = np.ascontiguousarray(raw[:, :2]).view(np.float16).astype(np.float64)
    assert np.allclose(((q - 8.0) * d).reshape(64, 128), deq)


def test_values_are_fp16_numbers():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((500, 32)) * np.exp(rng.uniform(-18, 9, (500, 1)))).astype(np.float32)
    v = AO.kv_values(*AO.kv_blocks(x))
    assert np.array_equal(v, v.astype(np.float16).astype(np.float64))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 65281.0, -1e30])
def test_bad_values_spoil_their_block_only(bad):
    x = np.ones((1, 64), np.float32)
    x[0, 40] = bad
    v = AO.kv_values(*AO.kv_blocks(x))
    assert np.all(np.isnan(v[0, 32:])) and np.all(v[0, :32] == v[0, 0])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_is_a_bijection(D):
    """Every nibble and scale byte of a record belongs to exactly one token's dim or block."""
    seen = np.zeros(2 * AO.record_bytes(D), int)
    for t in range(16):
        key, val, shift, ks, vs = AO._places(D, t)
        for at in (key, val):
            np.add.at(seen, 2 * at + (shift > 0), 1)
        for sc in (ks, vs):
            for b in (0, 1):
                np.add.at(seen, 2 * (sc + b), 1)
                np.add.at(seen, 2 * (sc + b) + 1, 1)
    assert np.all(seen == 1)


@pytest.mark.parametrize("D,page,heads", [(64, 16, 1), (128, 48, 3), (256, 32, 2)])
def test_store_then_load(D, page, heads):
    rng = np.random.default_rng(D)
    pool = rng.integers(0, 256, AO.pool_bytes(3, page, heads, D)).astype(np.uint8)
    slots = rng.permutation(3 * page)[:10]
    K, V = rng.standard_normal((2, 10, heads, D)).astype(np.float32)
    for i, s in enumerate(slots):
        for h in range(heads):
            AO.kv_store(pool, s, h, page, heads, D, K[i, h], V[i, h])
    for h in range(heads):
        k, v = AO.kv_load(pool, slots, h, page, heads, D)
        assert np.array_equal(k, AO.kv_values(*AO.kv_blocks(K[:, h])))
        assert np.array_equal(v, AO.kv_values(*AO.kv_blocks(V[:, h])))


def test_pages_by_hand():
    table = np.full((3, 4), -1)
    table[0, 0], table[2, 0] = 9, 8
    t, seq, cu, slots, pos, end = AO.cache_pages([15, 0, 16], [2, 0, 17], [3, 4, 5, 6, 7], 1, table, 16, 21)
    assert t.tolist() == [[9, 4, -1, -1], [-1, -1, -1, -1], [8, 5, 6, -1]] and end == 4
    assert seq.tolist() == [17, 0, 33] and cu.tolist() == [0, 2, 2, 19]
    assert slots[:3].tolist() == [9 * 16 + 15, 4 * 16, 5 * 16] and slots[18:].tolist() == [6 * 16, -1, -1]
    assert pos[:3].tolist() == [15, 16, 16] and pos[19:].tolist() == [-1, -1]


def test_norm_rope_closed_forms():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 2, 64))
    y = AO.norm_rope(x, None, 0.0, None, None)
    assert np.allclose((y ** 2).mean(-1), 1.0)
    ang = rng.uniform(0, 6, (9, 32))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([0, 8, 3, 3])
    for inter in (False, True):
        z = AO.norm_rope(x, None, 0.0, pos, cs, norm=False, interleaved=inter)
        assert np.allclose((z ** 2).sum(-1), (x ** 2).sum(-1))               # rotations keep lengths
        back = np.concatenate([cs[:, :32], -cs[:, 32:]], 1)
        assert np.allclose(AO.norm_rope(z, None, 0.0, pos, back, norm=False, interleaved=inter), x)
        f = AO.norm_rope32(x, None, 0.0, pos, cs.astype(np.float32), norm=False, interleaved=inter)
        assert np.allclose(f, z, atol=1e-5)


def test_attention_closed_forms():
    rng = np.random.default_rng(6)
    V = rng.standard_normal((50, 8))
    see = np.ones(50, bool)
    out, lse, p = AO.attention(np.zeros(8), rng.standard_normal((50, 8)), V, see, 0.3)
    assert np.allclose(out, V.mean(0)) and np.isclose(lse, np.log(50.0)) and np.isclose(p.sum(), 1)
    K = np.zeros((50, 8))
    K[17, 0] = 1.0
    out, _, _ = AO.attention(np.array([1000.0] + [0] * 7), K, V, see, 1.0)
    assert np.allclose(out, V[17])
    V[3] = np.nan
    see[3] = False
    assert np.all(np.isfinite(AO.attention(np.ones(8), K, V, see, 1.0)[0]))
    out, lse, _ = AO.attention(np.ones(8), K, V, np.zeros(50, bool), 1.0)
    assert np.all(out == 0) and lse == -np.inf


def test_visibility_by_hand():
    see = AO.visible(12, 10, 3, 1)                           # new tokens 7, 8, 9; token 8 sees 0..8
    assert see.tolist() == [True] * 9 + [False] * 3
    assert AO.visible(12, 10, 3, 1, window=4).tolist() == [False] * 5 + [True] * 4 + [False] * 3
    assert AO.visible(12, 10, 3, 2, bits=0b101).tolist() == [True] * 8 + [False, True] + [False] * 2
