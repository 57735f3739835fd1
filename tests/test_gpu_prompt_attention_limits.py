"""qg_prompt_attention where values leave the ordinary range: large finite values that a row does not
see, scores that are not finite, values next to the largest number, a factor of zero.

Tolerances (derived from the arithmetic, before any run), with A = |scale| sum |q| |k| of a score, the
largest of those that the row sees, V = sum p |v| and M the largest |v| that the row sees in the head:
* a score: D / 16 additions on the tensor cores that may cut off a bit, D / 16 * 2^-23 A; fp32's terms
  carry 22 bits of their row's largest, 2^-20 A more; the exponent's argument and the exponential 2^-20.
  ds is their sum; a probability is off by ds, an output by twice that of V.
* bf16: a probability rounded 2^-8, n / 16 additions 2^-23 each; the output's rounding 2^-8 |out|.
* fp32: probabilities in two terms 2^-21, sums by tiles 2^-18 V; terms of a value 2^-22 of the token's
  largest, terms of a small probability 2^-31 of the row's largest: 2^-22 M together.
* lse: ds + 2^-21 |lse| + 2^-20.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import prompt_oracle as PO

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_quantized_token_format_gb300 as qg  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qg.qg_device_status(clear=True)
    yield
    qg.qg_device_status(clear=True)


def host(t):
    return t.double().cpu().numpy()


def inputs(rng, n, hq, hk, D, act):
    x = torch.tensor(rng.standard_normal((n, hq + 2 * hk, D)), dtype=torch.float32, device="cuda").to(DT[act])
    return [t.clone() for t in (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])]


def run(q, k, v, cu, scale, window=0):
    n, hq, D = q.shape
    act = "f32" if q.dtype == torch.float32 else "bf16"
    out, lse = torch.full((n, hq, D), 5.0, dtype=q.dtype, device="cuda"), torch.full((n, hq), 5.0, device="cuda")
    ws = torch.full((qg.qg_prompt_attention_workspace_bytes(act, n, hq, k.shape[1], D),), 0xFF, dtype=torch.uint8, device="cuda")
    qg.qg_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out, ws, scale, max(np.diff(cu)), window=window, lse=lse)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == 0
    return out, lse


def check(q, k, v, cu, scale, window, out, lse, rows=None):
    act = "f32" if q.dtype == torch.float32 else "bf16"
    D, group = q.shape[2], q.shape[1] // k.shape[1]
    hq, hk, hv = host(q), host(k), host(v)
    want, wl, V = PO.prompt_attention(hq, hk, hv, cu, scale, window)
    A, M, n = np.zeros(want.shape[:2]), np.zeros(want.shape[:2]), np.zeros(len(want))
    for a, b in zip(cu[:-1], cu[1:]):
        for i in range(a, b):
            lo = max(a, i - window + 1) if window else a
            A[i] = [abs(scale) * (np.abs(hk[lo:i + 1, h // group]) @ np.abs(hq[i, h])).max() for h in range(hq.shape[1])]
            M[i] = np.repeat(np.abs(hv[lo:i + 1]).max(axis=(0, 2)), group)
            n[i] = i + 1 - lo
    ds = D / 16 * 2.0 ** -23 * A + 2.0 ** -20 + (2.0 ** -20 * A if act == "f32" else 0.0)
    if act == "f32":
        t = (2 * ds + 2.0 ** -18 + 2.0 ** -21)[..., None] * V + 2.0 ** -22 * M[..., None]
    else:
        t = (2 * ds + 2.0 ** -8 + n[:, None] / 16 * 2.0 ** -23)[..., None] * V + 2.0 ** -8 * np.abs(want)
    sel = np.arange(cu[0], cu[-1]) if rows is None else np.asarray(rows)
    assert (np.abs(host(out) - want)[sel] <= t[sel] + 1e-30).all()
    assert (np.abs(host(lse) - wl)[sel] <= (ds + 2.0 ** -21 * np.abs(wl) + 2.0 ** -20)[sel]).all()


# ------------------------------------------------------------------- what a row does not see

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [1e6, 1e20, 1e30])
@pytest.mark.parametrize("window", [0, 20])
def test_large_values_that_a_row_does_not_see(act, D, size, window):
    """A later token, a token beyond the window, another prompt and padding may hold any finite value: the
    rows that do not see it keep every bit."""
    rng = np.random.default_rng(41)
    cu = [2, 90, 150]
    q, k, v = inputs(rng, 200, 4, 2, D, act)
    clean, lse_clean = run(q, k, v, cu, 0.1, window)
    check(q, k, v, cu, 0.1, window, clean, lse_clean)
    for t in (q, k, v):
        t[:2], t[150:] = size, -size
    k[40, 0] *= size
    v[40] *= size
    k[75] *= -size
    v[75, 1, 3] = size
    v[149] *= size
    out, lse = run(q, k, v, cu, 0.1, window)
    sees = np.zeros(200, bool)
    sees[:2] = sees[149:] = True                                     # (149 sees itself; padding is not looked at)
    for at in (40, 75):
        sees[at:min(90, at + window) if window else 90] = True
    hidden = ~sees
    assert hidden[:40].sum() == 38 and hidden[90:149].all()
    assert np.array_equal(host(out)[hidden], host(clean)[hidden]) and np.array_equal(host(lse)[hidden], host(lse_clean)[hidden])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 70])
def test_fp32_tokens_of_any_size(D, window):
    """Every key and value token has its own size: an output is as exact as the values that its row sees allow."""
    rng = np.random.default_rng(42)
    cu = [0, 130, 300]
    q, k, v = inputs(rng, 300, 4, 2, D, "f32")
    v *= torch.tensor(10.0 ** rng.uniform(-20, 20, (300, 2, 1)), device="cuda").float()
    k *= torch.tensor(10.0 ** rng.uniform(-6, 0, (300, 2, 1)), device="cuda").float()
    v[50] = 0.0
    v[131] = k[131] = 0.0
    out, lse = run(q, k, v, cu, 0.1, window)
    check(q, k, v, cu, 0.1, window, out, lse)


def test_values_that_grow_along_a_prompt():
    """Each value 1.3 times the one before: 1e-10 to 1e24 in one prompt, the first ones as exact as the last."""
    rng = np.random.default_rng(43)
    q, k, v = inputs(rng, 300, 2, 1, 128, "f32")
    v *= torch.tensor(1e-10 * 1.3 ** np.arange(300), device="cuda").float()[:, None, None]
    out, lse = run(q, k, v, [0, 300], 0.1)
    check(q, k, v, [0, 300], 0.1, 0, out, lse)


# ----------------------------------------------------------------- scores that are not finite

@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_that_are_not_finite_bf16(D):
    """A score of -infinity has weight 0; a row of nothing else has no average; one of +infinity or NaN none either."""
    rng = np.random.default_rng(45)
    q, k, v = inputs(rng, 200, 2, 1, D, "bf16")
    q[:, 0, 5], q[:, 1, 5] = 1.0, -1.0
    q[:100, :, 6] = 1.0
    k[0, 0, 5] = float("-inf")                                       # head 0: -infinity, head 1: +infinity
    k[100, 0, 6] = float("nan")
    out, lse = run(q, k, v, [0, 70, 200], 0.1)
    o, l = host(out), host(lse)
    assert np.isnan(o[0, 0]).all() and l[0, 0] == -np.inf
    assert np.isnan(o[:70, 1]).all() and not np.isfinite(l[:70, 1]).any()
    assert np.isnan(o[100:]).all() and np.isnan(l[100:]).all()
    k[0, 0, 5] = -3e38                                               # finite, and as little weight
    want, wl = run(q, k, v, [0, 70, 200], 0.1)
    assert np.array_equal(o[1:70, 0], host(want)[1:70, 0]) and np.array_equal(l[1:70, 0], host(wl)[1:70, 0])
    assert np.isfinite(o[70:100]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("-inf"), float("inf"), float("nan")])
def test_keys_and_queries_that_are_not_finite_fp32(D, bad):
    """The rows that see one are NaN, the others keep every bit."""
    rng = np.random.default_rng(46)
    q, k, v = inputs(rng, 300, 4, 2, D, "f32")
    clean, lse_clean = run(q, k, v, [0, 70, 300], 0.1)
    k[0, 0, 5] = k[150, 1, 6] = q[290, 0, 7] = bad
    out, lse = run(q, k, v, [0, 70, 300], 0.1)
    nan = np.zeros((300, 4), bool)
    nan[:70, :2] = nan[150:, 2:] = nan[290, 0] = True
    o, l = host(out), host(lse)
    assert np.isnan(o[nan]).all() and np.isnan(l[nan]).all()
    assert np.array_equal(o[~nan], host(clean)[~nan]) and np.array_equal(l[~nan], host(lse_clean)[~nan])


# ------------------------------------------------------------------------- the range's end

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_fp32_values_next_to_the_largest(D, n):
    """Outputs are averages: they are finite where the values are."""
    rng = np.random.default_rng(44)
    q, k, v = inputs(rng, n, 2, 1, D, "f32")
    v = torch.tensor(rng.uniform(0.5, 0.99, (n, 1, D)) * 2.0 ** 128, dtype=torch.float32, device="cuda")
    q[:, 1] = 0.0                                                    # even weights
    out, lse = run(q, k, v, [0, n], 0.1)
    assert torch.isfinite(out).all()
    check(q, k, v, [0, n], 0.1, 0, out, lse)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_rise_under_large_values(act, D):
    """Weights grow 2^7 from the first 64 keys to the next: sums of weights times values stay within what the
    weights' largest being 1 allows."""
    n = 128
    q = torch.zeros(n, 1, D, dtype=DT[act], device="cuda")
    k, v = torch.zeros_like(q), torch.full_like(q, 1e36)
    q[:, 0, 0] = 7.0
    k[64:, 0, 0] = 1.0
    scale = float(np.log(2.0))
    out, lse = run(q, k, v, [0, n], scale)
    assert torch.isfinite(out).all()
    check(q, k, v, [0, n], scale, 0, out, lse)


# ------------------------------------------------------------------------------ factors

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_factor_of_zero(act, D):
    """Every score is zero, however large the products are: averages of the values."""
    rng = np.random.default_rng(47)
    q, k, v = inputs(rng, 200, 2, 1, D, act)
    q[:], k[:] = 0.0, 0.0
    big = 1.6e19 if act == "bf16" else 1e35                          # (bf16: the products are fp32 numbers)
    q[:, :, 0] = big
    k[:, 0, 0] = torch.tensor(rng.choice([-big, big], 200), device="cuda").to(DT[act])
    out, lse = run(q, k, v, [0, 200], 0.0)
    assert np.abs(host(lse) - np.log(np.arange(1, 201))[:, None]).max() <= 2.0 ** -18
    check(q, k, v, [0, 200], 0.0, 0, out, lse)


# ------------------------------------------------------------------------------ lengths

@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_prompts_are_reported_fp32(D):
    """Lengths that shrink or leave the tokens, whose powers of two nobody has written, are reported."""
    rng = np.random.default_rng(48)
    q, k, v = inputs(rng, 40, 2, 1, D, "f32")
    out, ws = torch.zeros(40, 2, D, device="cuda"), torch.full((qg.qg_prompt_attention_workspace_bytes("f32", 40, 2, 1, D),), 0xFF,
                                                               dtype=torch.uint8, device="cuda")
    for cu in ([0, 20, 10, 40], [-1, 20, 40], [0, 20, 41], [30, 10], [0, 1 << 30]):
        qg.qg_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out, ws, 0.1, 40)
        torch.cuda.synchronize()
        assert qg.qg_device_status(clear=True) == qg.QG_DEVICE_BAD_LENGTH
    good, lse = run(q, k, v, [0, 40], 0.1)
    check(q, k, v, [0, 40], 0.1, 0, good, lse)
