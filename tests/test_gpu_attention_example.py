"""The example runs the attention sublayer end to end: prompt, decode as a replayed graph, verify."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_step.py")


def test_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("attention_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.main(prompt=70, decode=6)
    # 70 prompt tokens each, one decode step before the graph, 5 replays, 4 verified by the first
    assert r["lengths"] == [70 + 6 + 4, 70 + 6]
    assert r["pages"] == 4                                   # two pages of 64 each
    for y in (r["decode"], r["verify"]):
        assert torch.isfinite(y).all() and float(y.abs().max()) > 0
