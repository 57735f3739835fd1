"""qgemm and qgemm_experts at the ends of their range: long sums.

Tolerances (derived from the arithmetic, before any run), with S = sum |w x|: the tensor cores may cut off the
last bit of a sum that they add to, 2^-23 of S for each addition of 16 products.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle
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


def space(fmt, act, n_out, n_in, n, n_experts=0):
    return torch.full((qg.qgemm_workspace_bytes(fmt, act, n_out, n_in, n, n_experts),), 0xFF, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------ long sums

def products_of_one_sign(rng, fmt, rows, n_in):
    c = oracle.quantize(fmt, rng.uniform(0.25, 1.0, (rows, n_in)).astype(np.float32))
    return c, torch.from_numpy(qg.qg_to_device_layout(fmt, c, rows, n_in)).cuda()


def tolerance(y, n_in, act):
    """Of sums of one sign (S = y).  bf16: weights rounded 2^-11, chains of 8192 products (512 additions, 2^-14) whose
    sums are added in fp32, the output's rounding 2^-8.  fp32: terms 2^-21, chains of 256 and their small products'
    2^-18, their sums in fp32."""
    if act == "bf16":
        return (2.0 ** -11 + 2.0 ** -14 + n_in / 8192 * 2.0 ** -24 + 2.0 ** -8) * y
    return (2.0 ** -21 + 2.0 ** -18 + (n_in / 256 + 8) * 2.0 ** -24) * y


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "affine4_g64", "bf16", "q5_0"])
def test_long_sums(fmt, act):
    """Four million products of one sign, by one CTA and by a cluster.  The tokens are one, times powers of two."""
    rng = np.random.default_rng(51)
    n_out, n_in, ntok = 3, 1 << 22, 130
    c, W = products_of_one_sign(rng, fmt, 2 * n_out, n_in)
    one = torch.tensor(rng.uniform(0.5, 2.0, n_in), dtype=torch.float32, device="cuda").bfloat16()
    size = 2.0 ** rng.integers(-3, 4, ntok)
    x = (one * torch.tensor(size[:, None], device="cuda").bfloat16()).to(DT[act])
    want = PO.gemm(fmt, c, 2 * n_out, n_in, host(one)[None]).reshape(2, n_out)
    y = torch.zeros(ntok, n_out, dtype=DT[act], device="cuda")
    qg.qgemm_experts(fmt, W, 2, n_out, n_in, x, torch.tensor([0, 50, ntok], dtype=torch.int32, device="cuda"), y,
                     space(fmt, act, n_out, n_in, ntok, 2))
    exact = np.concatenate([np.tile(want[0], (50, 1)), np.tile(want[1], (ntok - 50, 1))]) * size[:, None]
    assert (np.abs(host(y) - exact) <= tolerance(exact, n_in, act)).all()
    y = torch.zeros(ntok, 2 * n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, 2 * n_out, n_in, x, y, space(fmt, act, 2 * n_out, n_in, ntok))
    exact = want.reshape(1, -1) * size[:, None]
    assert (np.abs(host(y) - exact) <= tolerance(exact, n_in, act)).all()
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "affine4_g64", "bf16", "q5_0"])
@pytest.mark.parametrize("n_in", [16384, 16384 + 64, 24576 - 64, 24576, 24576 + 64, 32768 + 8192])
def test_sums_around_a_chain(fmt, n_in):
    """One chain, chains with a step at the end and without, several tiles to a CTA; random signs."""
    rng = np.random.default_rng(n_in)
    n_experts, n_out, counts = 3, 129, [300, 0, 17]
    c = oracle.quantize(fmt, (rng.standard_normal((n_experts * n_out, n_in)) * 0.02).astype(np.float32))
    W = torch.from_numpy(qg.qg_to_device_layout(fmt, c, n_experts * n_out, n_in)).cuda()
    off = [0] + list(np.cumsum(counts))
    x = torch.tensor(rng.standard_normal((off[-1], n_in)), dtype=torch.float32, device="cuda").bfloat16()
    y = torch.zeros(off[-1], n_out, dtype=torch.bfloat16, device="cuda")
    qg.qgemm_experts(fmt, W, n_experts, n_out, n_in, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y,
                     space(fmt, "bf16", n_out, n_in, off[-1], n_experts))
    args = (fmt, c, n_experts, n_out, n_in, host(x), off)
    v, S = PO.gemm_experts(*args), PO.gemm_experts(*args, product=PO.gemm_abs)
    got = host(y)
    for s in range(off[-1]):
        assert (np.abs(got[s] - v[s]) <= (2.0 ** -11 + 2.0 ** -13) * S[s] + 2.0 ** -8 * np.abs(v[s])).all()
    assert qg.qg_device_status() == 0
