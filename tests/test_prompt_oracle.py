"""The 64-bit implementation of the whole-prompt calls against closed forms and brute force."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
from oracle import prompt_oracle as PO


@pytest.mark.parametrize("f,v,want", [("silu", 0.0, 0.0), ("silu", 2.0, 2.0 / (1.0 + math.exp(-2.0))), ("gelu", 1.0, 0.8413447460685429),
                                      ("gelu", -1.0, -0.15865525393145707), ("gelu_tanh", 1.0, 0.8411919906082768), ("none", -3.0, -3.0)])
def test_activations(f, v, want):
    assert abs(float(PO.activation(np.array([v]), f)[0]) - want) < 1e-12


def test_swiglu_pairs():
    y = PO.activation(np.array([[1.0, 3.0, -2.0, 5.0]]), "swiglu")
    assert np.allclose(y, [[3.0 / (1 + math.exp(-1.0)), -10.0 / (1 + math.exp(2.0))]], rtol=1e-14)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "affine4_g64", "bf16", "q5_0"])
def test_gemm_is_the_mat_vec(fmt):
    rng = np.random.default_rng(3)
    W, x = rng.standard_normal((6, 128)).astype(np.float32), rng.standard_normal((3, 128)).astype(np.float32)
    c = oracle.quantize(fmt, W)
    y = PO.gemm(fmt, c, 6, 128, x)
    assert np.allclose(y, oracle.gemv(fmt, c, 6, 128, x), rtol=1e-13, atol=1e-13)
    assert (PO.gemm_abs(fmt, c, 6, 128, x) >= np.abs(y) - 1e-12).all()
    b, r = rng.standard_normal(6), rng.standard_normal((3, 6))
    assert np.allclose(PO.gemm(fmt, c, 6, 128, x, b, "silu", r), PO.activation(y + b, "silu") + r)


def test_experts_pick_their_rows():
    rng = np.random.default_rng(4)
    W, x = rng.standard_normal((3 * 2, 64)).astype(np.float32), rng.standard_normal((4, 64))
    c = oracle.quantize("bf16", W)
    full = oracle.dequantize("bf16", c, 6, 64)
    got = PO.gemm_experts("bf16", c, 3, 2, 64, x, [1, 3, 3, 4], rows=[9, 2, 0, 3])
    assert sorted(got) == [1, 2, 3]
    assert np.allclose(got[1], full[0:2] @ x[2]) and np.allclose(got[2], full[0:2] @ x[0]) and np.allclose(got[3], full[4:6] @ x[3])


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attention_by_hand(window):
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    out, lse, _ = PO.prompt_attention(q, k, v, [1, 4, 4, 6], 0.3, window)
    assert np.isnan(out[0]).all() and np.isnan(out[6]).all()
    for a, b in ((1, 4), (4, 6)):
        for i in range(a, b):
            for h in range(4):
                w = [(j, math.exp(0.3 * float(q[i, h] @ k[j, h // 2]))) for j in range(a, i + 1) if not window or j > i - window]
                t = sum(x for _, x in w)
                assert np.allclose(out[i, h], sum(x / t * v[j, h // 2] for j, x in w)) and abs(lse[i, h] - math.log(t)) < 1e-12
    # values that are not seen may be anything
    v2 = v.copy()
    v2[[0, 6]] = np.nan
    assert np.array_equal(PO.prompt_attention(q, k, v2, [1, 4, 4, 6], 0.3, window)[0][1:6], out[1:6])
