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


@pytest.mark.parametrize("prompt", [1, 70, 71])
def test_prompts_whole_and_in_steps(prompt):
    """Both ways in give the same lengths, pages and, but for the cache's rounding, outputs.  The mat-vec's inputs have
    16 bits of their largest: keys and values differ by 2^-14 of their root mean square or so, the cached ones by a whole
    step (a seventh of a group's largest, half of its root mean square) in 2^-12 of the places: 2^-7 of the norm
    for keys and values each, 2^-5 of the outputs'."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("attention_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    a, b = mod.main(prompt=prompt, decode=2), mod.main(prompt=prompt, decode=2, whole=False)
    assert a["lengths"] == b["lengths"] == [prompt + 2 + 4, prompt + 2] and a["pages"] == b["pages"]
    assert a["prompt"].shape == b["prompt"].shape == (2, prompt, mod.D_MODEL)
    assert torch.isfinite(a["prompt"]).all() and float(a["prompt"].abs().max()) > 0
    assert float((a["prompt"] - b["prompt"]).norm()) <= 2.0 ** -5 * float(b["prompt"].norm())
