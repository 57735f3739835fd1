"""qgemm and qgemm_experts at the ends of their range: long sums, tiles of every width.

Tolerances (derived from the arithmetic, before any run), with S = sum |w x|: the tensor cores may cut off the
last bit of a sum that they add to, 2^-23 of S for each addition of 16 products.
"""
from __future__ import annotations

import functools

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


# --------------------------------------------------------------------------- wide tiles

QUANT = ["q8_0", "q4_0", "affine4_g64", "q5_0"]
N_IN = {"q8_0": 1120, "q4_0": 1120, "q5_0": 1120, "affine4_g64": 1152, "bf16": 1136}      # half a step, or two, at the end
LONG = {"q8_0": 4640, "q4_0": 4640, "q5_0": 4640, "affine4_g64": 4672, "bf16": 4656}


def tile(*a):
    return {k: int(v) for k, v in (p.split("=") for p in qg.qg_describe_gemm_tile(*a).split(","))}


@functools.lru_cache(maxsize=2)
def weights(fmt, rows, n_in):
    """Canonical bytes, packed bytes and the weights themselves in 64 bits."""
    c = oracle.quantize(fmt, (np.random.default_rng(rows).standard_normal((rows, n_in)) * 0.02).astype(np.float32))
    return c, torch.from_numpy(qg.qg_to_device_layout(fmt, c, rows, n_in)).cuda(), torch.from_numpy(oracle.dequantize(fmt, c, rows, n_in)).cuda()


def tokens(rng, n, n_in, act):
    return torch.tensor(rng.standard_normal((n, n_in)) * rng.uniform(0.5, 2.0, (n, 1)), dtype=torch.float32, device="cuda").to(DT[act])


def check(x, W, y, act):
    """bf16: a weight rounded to fp16 2^-11 of S, n_in / 16 additions that may cut off a bit, the output's rounding
    2^-8 of it.  fp32: terms 2^-21, chains of 256 and their small products' 2^-18, their sums in fp32."""
    want, S, n_in = x.double() @ W.t(), x.double().abs() @ W.abs().t(), x.shape[1]
    if act == "bf16":
        t = S * (2.0 ** -11 + n_in / 16 * 2.0 ** -23) + 2.0 ** -8 * want.abs()
    else:
        t = S * (2.0 ** -21 + 2.0 ** -18 + (n_in / 256 + 8) * 2.0 ** -24)
    assert bool(((y.double() - want).abs() <= t).all())


WIDE = ([(f, "bf16", *c) for f in QUANT for c in ((96, 3967, 776), (112, 3967, 875), (128, 3583, 1139), (144, 3967, 1172), (160, 3967, 1304),
                                                  (176, 3583, 1601), (192, 3583, 1766))] +
        [(f, "f32", *c) for f in QUANT for c in ((48, 2815, 578), (64, 3967, 446), (80, 3967, 578), (96, 3583, 809))] +
        [("bf16", "bf16", *c) for c in ((128, 3967, 1040), (144, 3967, 1172), (176, 3583, 1601), (208, 3967, 1733), (240, 3967, 2030), (256, 3967, 2162))] +
        [("bf16", "f32", *c) for c in ((64, 3327, 644), (80, 3967, 578), (96, 3583, 809), (112, 3967, 875), (128, 3583, 1139))])


@pytest.mark.parametrize("fmt,act,width,n_out,ntok", sorted(WIDE))
def test_tiles_of_every_width(fmt, act, width, n_out, ntok):
    """More tiles than SMs, so that CTAs take a second one; the last ones partly filled in both directions."""
    n_in = N_IN[fmt]
    got = tile(fmt, act, n_out, n_in, ntok)
    assert got["tokens"] == width and got["parts"] == 1 and -(-n_out // 128) * -(-ntok // width) > 152
    _, packed, W = weights(fmt, n_out, n_in)
    x = tokens(np.random.default_rng(width), ntok, n_in, act)
    y = torch.zeros(ntok, n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, packed, n_out, n_in, x, y, space(fmt, act, n_out, n_in, ntok))
    check(x, W, y, act)
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("n_out,ntok", [(127, 1), (1023, 53), (1023, 66), (1919, 105), (1919, 183), (2047, 92), (2431, 105), (2431, 196)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", QUANT + ["bf16"])
def test_clusters(fmt, act, n_out, ntok):
    """CTAs that share K, in numbers that do not divide it, with tiles of one width and another."""
    n_in = LONG[fmt]
    assert tile(fmt, act, n_out, n_in, ntok)["parts"] > 1
    _, packed, W = weights(fmt, n_out, n_in)
    x = tokens(np.random.default_rng(ntok), ntok, n_in, act)
    y = torch.zeros(ntok, n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, packed, n_out, n_in, x, y, space(fmt, act, n_out, n_in, ntok))
    check(x, W, y, act)
    assert qg.qg_device_status() == 0


def test_clusters_of_many_sizes():
    """The cases above are of several numbers of CTAs and widths."""
    for act, fmts in (("bf16", QUANT + ["bf16"]), ("f32", QUANT + ["bf16"])):
        got = [tile(f, act, n_out, LONG[f], ntok) for f in fmts for n_out, ntok in
               ((127, 1), (1023, 53), (1023, 66), (1919, 105), (1919, 183), (2047, 92), (2431, 105), (2431, 196))]
        assert len({g["parts"] for g in got}) >= 3 and len({g["tokens"] for g in got}) >= 4 and max(g["tokens"] for g in got) >= 96


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", QUANT + ["bf16"])
def test_experts_in_wide_tiles(fmt, act):
    """Experts' rows around every multiple of sixteen that a tile takes, some more than a tile has; more tiles than SMs."""
    counts = [16, 1, 0, 15, 17, 31, 32, 33, 48, 49, 64, 100, 192, 193, 95, 96, 97, 111, 112, 113, 127, 128, 129, 143, 144, 145, 159, 160, 161, 175, 176,
              177, 191, 208, 255, 256, 257]
    n_experts, n_out, n_in, off = len(counts), 515, 1152, [0] + list(np.cumsum(counts))
    width = tile(fmt, act, n_out, n_in, int(off[-1]), n_experts)["tokens"]
    assert width >= (80 if act == "f32" else 128) and 5 * sum(-(-k // width) for k in counts) > 152
    _, packed, W = weights(fmt, n_experts * n_out, n_in)
    x = tokens(np.random.default_rng(3), int(off[-1]), n_in, act)
    y = torch.zeros(int(off[-1]), n_out, dtype=DT[act], device="cuda")
    qg.qgemm_experts(fmt, packed, n_experts, n_out, n_in, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y,
                     space(fmt, act, n_out, n_in, int(off[-1]), n_experts))
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        check(x[a:b], W[e * n_out:(e + 1) * n_out], y[a:b], act)
    assert qg.qg_device_status() == 0
