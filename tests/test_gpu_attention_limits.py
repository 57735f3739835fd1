"""GPU parity of the attention path at the ends of its ranges: what the cache may hold at most, scores
of any size, long chunks in large batches, lengths near 2^31, inconsistent device data.

Tolerances are those of ``test_gpu_attention`` (derived there); others are derived beside their test.
"""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import attention_oracle as AO

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_token_format_gb300 as qg  # noqa: E402
from test_gpu_attention import Case, _cuda, dev, heads_input, host, ints, rotation, run_pages  # noqa: E402, F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------------------------ values

# Scales of 2720 (the last whose 24-fold is finite in fp16), 2736 (the next one), and the largest.
TOPS = [21760.0, 21888.0, 32768.0, 65280.0]


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("D,heads,kv,new,act", [(64, 4, 2, 1, "f32"), (128, 2, 2, 3, "f32"), (128, 12, 2, 2, "f32"), (256, 6, 1, 4, "f32"),
                                                (128, 8, 1, 1, "bf16"), (64, 8, 1, 2, "bf16"), (256, 12, 1, 1, "bf16")])
def test_largest_values_the_cache_takes(top, D, heads, kv, new, act):
    """Every magnitude up to QG_CACHE_MAX takes part as the finite number that the cache gives back."""
    c = Case(int(top) + D, D, heads, kv, [90, 3, 700], [new, 1, new], page=48, act=act, v_scale=1.0)
    v = c.rng.uniform(-1, 1, c.v.shape) * top
    v.reshape(-1, 32)[:, 5] = top * c.rng.choice([-1, 1], v.size // 32)
    pick = c.rng.random(v.shape[0]) < 0.5                    # others stay small: both kinds in one unit
    c.v[pick] = v[pick].astype(np.float32)
    c.append()
    got = c.run()
    assert bool(torch.isfinite(got).all())
    c.check(got)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_large_values_stay_where_they_are_seen(act):
    """A large value that only some rows of a tile see reaches no other row."""
    c = Case(3, 128, 4, 2, [60, 40], [4, 4], page=16, window=30, tree=True, act=act, v_scale=1.0)
    c.bits[:] = [1, 2, 4, 8] * 2                             # every new token sees itself only
    c.v[61, 1] = 65280.0                                     # request 0's token 61: its row alone
    c.v[64 + 42, 0, 40] = -30000.0                           # request 1's token 42
    c.v[20] = 65280.0                                        # outside every window
    c.append()
    got = c.run()
    c.check(got)
    big = got.abs().amax(-1) > 100
    want = np.zeros(tuple(big.shape), dtype=bool)
    want[1, 2:] = want[6, :2] = True
    assert np.array_equal(big.cpu().numpy(), want)
