"""GPU parity of qgemm and qgemm_experts against the fp64 oracle.

Tolerances (derived from the arithmetic, before any run), with S = sum |w x|:
* fp32: x has 22 bits of the row's largest value in two terms, the third product of small terms is
  left out: 2^-21 of S (and 2^-40 of the row's largest times sum |w|: nothing against S here); a chain
  of 16 additions on the tensor cores, which may cut off the last bit each, and as many small
  ones: 2^-18 of S; the parts in fp32: (n_in / 256 + 8) 2^-24 of S.
* bf16: a weight rounded to fp16 2^-11 of S; n_in / 16 additions that may cut off a bit: n_in / 16 *
  2^-23 of S; the output's rounding 2^-8 of it.
* bias, activation, residual in fp32: 2^-20 of what they are made of.  Slopes of silu and both gelu are
  below 1.13; silu(g) u is off by 1.13 |u| dg + |silu(g)| du + 1.13 dg du.
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
FMTS = ["q8_0", "q4_0", "affine4_g64", "bf16", "q5_0"]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qg.qg_device_status(clear=True)
    yield
    qg.qg_set_wait_limit(0, 0)
    qg.qg_set_launch_options(0)
    qg.qg_device_status(clear=True)


def host(t):
    return t.double().cpu().numpy()


def packed(rng, fmt, n_out, n_in, spread=0.02):
    W = (rng.standard_normal((n_out, n_in)) * spread).astype(np.float32)
    c = oracle.quantize(fmt, W)
    return c, torch.from_numpy(qg.qg_to_device_layout(fmt, c, n_out, n_in)).cuda()


def tokens(rng, n, width, act, lo=0.5, hi=2.0):
    x = rng.standard_normal((n, width)) * rng.uniform(lo, hi, (n, 1))
    return torch.tensor(x, dtype=torch.float32, device="cuda").to(DT[act])


def space(fmt, act, n_out, n_in, n, n_experts=0):
    return torch.full((qg.qgemm_workspace_bytes(fmt, act, n_out, n_in, n, n_experts),), 0xFF, dtype=torch.uint8, device="cuda")


def product_tolerance(S, n_in, act):
    if act == "f32":
        return S * (2.0 ** -21 + 2.0 ** -18 + (n_in / 256 + 8) * 2.0 ** -24)
    return S * (2.0 ** -11 + n_in / 16 * 2.0 ** -23)


def tolerance(S, v, y, n_in, act, f, bias=None, residual=None):
    """v: the exact products with bias, y: the exact outputs."""
    t = product_tolerance(S, n_in, act) + 2.0 ** -20 * np.abs(v)
    if bias is not None:
        t = t + 2.0 ** -20 * np.abs(bias)
    if f == "swiglu":
        g, u, dg, du = v[..., 0::2], v[..., 1::2], 1.13 * t[..., 0::2], t[..., 1::2]
        t = dg * np.abs(u) + np.abs(PO.activation(g, "silu")) * du + dg * du
    elif f not in (None, "none"):
        t = 1.13 * t
    t = t + 2.0 ** -20 * np.abs(y)
    if residual is not None:
        t = t + 2.0 ** -20 * np.abs(residual)
    return t + (2.0 ** -8 * np.abs(y) if act == "bf16" else 0.0) + 1e-30


CASES = [  # n_out, n_in, ntok, f, bias, residual
    (1, 64, 1, "none", False, False), (128, 64, 1, "none", True, False), (2, 128, 3, "swiglu", True, True), (129, 192, 33, "silu", False, True),
    (300, 640, 77, "none", False, False), (257, 1088, 130, "gelu", True, False), (64, 2560, 241, "gelu_tanh", False, True),
    (1000, 1280, 5, "none", True, True), (640, 4096, 17, "swiglu", False, False), (96, 704, 300, "silu", True, False),
    (200, 10240, 9, "none", False, False)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_out,n_in,ntok,f,bias,residual", CASES)
def test_gemm(fmt, act, n_out, n_in, ntok, f, bias, residual):
    rng = np.random.default_rng(n_out + ntok)
    c, W = packed(rng, fmt, n_out, n_in)
    x = tokens(rng, ntok, n_in, act)
    width = n_out // 2 if f == "swiglu" else n_out
    b = torch.tensor(rng.standard_normal(n_out), dtype=torch.float32, device="cuda") if bias else None
    r = tokens(rng, ntok, width, act) if residual else None
    y = torch.full((ntok, width), 7.0, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, n_out, n_in, x, y, space(fmt, act, n_out, n_in, ntok), bias=b, activation=f, residual=r)
    hb, hr = None if b is None else host(b), None if r is None else host(r)
    v = PO.gemm(fmt, c, n_out, n_in, host(x), hb)
    want = PO.activation(v, f) if hr is None else PO.activation(v, f) + hr
    t = tolerance(PO.gemm_abs(fmt, c, n_out, n_in, host(x)), v, want, n_in, act, f, hb, hr)
    assert (np.abs(host(y) - want) <= t).all()
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "q5_0"])
@pytest.mark.parametrize("n_in", [32, 96, 544, 1056, 2080])
def test_half_a_step_at_the_end(fmt, act, n_in):
    """n_in an odd number of blocks: what lies behind a row's codes does not count."""
    rng = np.random.default_rng(n_in)
    c, W = packed(rng, fmt, 131, n_in)
    x = tokens(rng, 40, n_in, act)
    y = torch.zeros(40, 131, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, 131, n_in, x, y, space(fmt, act, 131, n_in, 40))
    want = PO.gemm(fmt, c, 131, n_in, host(x))
    assert (np.abs(host(y) - want) <= tolerance(PO.gemm_abs(fmt, c, 131, n_in, host(x)), want, want, n_in, act, None)).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_bf16_rows_that_are_no_multiple_of_a_step(act):
    rng = np.random.default_rng(2)
    for n_in in (16, 48, 272):
        c, W = packed(rng, "bf16", 70, n_in)
        x = tokens(rng, 9, n_in, act)
        y = torch.zeros(9, 70, dtype=DT[act], device="cuda")
        qg.qgemm("bf16", W, 70, n_in, x, y, space("bf16", act, 70, n_in, 9))
        want = PO.gemm("bf16", c, 70, n_in, host(x))
        assert (np.abs(host(y) - want) <= tolerance(PO.gemm_abs("bf16", c, 70, n_in, host(x)), want, want, n_in, act, None)).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
def test_strides_and_what_lies_between(fmt, act):
    rng = np.random.default_rng(6)
    n_out, n_in, n = 72, 256, 50
    c, W = packed(rng, fmt, n_out, n_in)
    wide = tokens(rng, n, n_in + 64, act)
    x = wide[:, 32:32 + n_in]
    out = torch.full((n + 2, n_out + 5), 3.0, dtype=DT[act], device="cuda")
    y = out[1:n + 1, 2:2 + n_out]
    y.copy_(tokens(rng, n, n_out, act))
    before = host(y)
    qg.qgemm(fmt, W, n_out, n_in, x, y, space(fmt, act, n_out, n_in, n), residual=y)             # in place
    v = PO.gemm(fmt, c, n_out, n_in, host(x))
    t = tolerance(PO.gemm_abs(fmt, c, n_out, n_in, host(x)), v, v + before, n_in, act, None, None, before)
    assert (np.abs(host(y) - (v + before)) <= t).all()
    rest = host(out)
    rest[1:n + 1, 2:2 + n_out] = 3.0
    assert (rest == 3.0).all()


@pytest.mark.parametrize("fmt", ["q8_0", "affine4_g64", "bf16"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_values_of_any_size(fmt, act):
    """Each token's scale is its own: huge, tiny and zero rows beside ordinary ones."""
    rng = np.random.default_rng(7)
    n_out, n_in, n = 40, 512, 24
    c, W = packed(rng, fmt, n_out, n_in)
    size = 10.0 ** rng.integers(-30, 30, n)
    size[3] = 0.0
    x = torch.tensor(rng.standard_normal((n, n_in)) * size[:, None], dtype=torch.float32, device="cuda").to(DT[act])
    x[5, 7] *= 2.0 ** 20                                             # one value far above its row
    y = torch.ones(n, n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, n_out, n_in, x, y, space(fmt, act, n_out, n_in, n))
    want = PO.gemm(fmt, c, n_out, n_in, host(x))
    S = PO.gemm_abs(fmt, c, n_out, n_in, host(x))
    t = tolerance(S, want, want, n_in, act, None) + 2.0 ** -38 * np.abs(host(x)).max(1, keepdims=True) * np.abs(oracle.dequantize(fmt, c, n_out, n_in)).sum(1)
    assert (np.abs(host(y) - want) <= t + 1e-38).all() and (host(y)[3] == 0).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_weights_of_any_scale(act):
    """fp16 scales from the smallest to those whose weights are 60000."""
    rng = np.random.default_rng(8)
    n_in = 256
    W = (rng.standard_normal((64, n_in)) * 10.0 ** rng.uniform(-6, 3.5, (64, 1))).astype(np.float32).clip(-60000, 60000)
    for fmt in ("q8_0", "q4_0", "q5_0", "affine4_g64"):
        c = oracle.quantize(fmt, W)
        Wd = torch.from_numpy(qg.qg_to_device_layout(fmt, c, 64, n_in)).cuda()
        x = tokens(rng, 20, n_in, act)
        y = torch.zeros(20, 64, dtype=DT[act], device="cuda")
        qg.qgemm(fmt, Wd, 64, n_in, x, y, space(fmt, act, 64, n_in, 20))
        want = PO.gemm(fmt, c, 64, n_in, host(x))
        S = PO.gemm_abs(fmt, c, 64, n_in, host(x))
        # (weights below 2^-14 are multiples of 2^-24, which fp16 holds)
        assert (np.abs(host(y) - want) <= tolerance(S, want, want, n_in, act, None) + 2.0 ** -36 * n_in).all()


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_values_that_are_not_finite_stay_in_their_token(fmt, act):
    rng = np.random.default_rng(9)
    c, W = packed(rng, fmt, 33, 128)
    x = tokens(rng, 40, 128, act)
    x[4, 3], x[9, 100], x[20] = float("nan"), float("inf"), float("-inf")
    ws = space(fmt, act, 33, 128, 40)
    y, clean = torch.zeros(40, 33, dtype=DT[act], device="cuda"), torch.zeros(40, 33, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, 33, 128, x, y, ws)
    qg.qgemm(fmt, W, 33, 128, torch.where(torch.isfinite(x), x, torch.zeros_like(x)), clean, ws)
    bad = [4, 9, 20]
    ok = [i for i in range(40) if i not in bad]
    assert not torch.isfinite(y[bad]).any() and torch.equal(y[ok], clean[ok])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_outputs_are_the_same_on_every_run_stream_and_replay(act):
    rng = np.random.default_rng(10)
    fmt, n_out, n_in, n = "q8_0", 512, 2560, 70
    _, W = packed(rng, fmt, n_out, n_in)
    x = tokens(rng, n, n_in, act)
    ws, other = space(fmt, act, n_out, n_in, n), space(fmt, act, n_out, n_in, n)
    y = torch.zeros(n, n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, n_out, n_in, x, y, ws)
    want = y.clone()
    for _ in range(5):
        y.zero_()
        qg.qgemm(fmt, W, n_out, n_in, x, y, ws)
        assert torch.equal(y, want)
    side, z = torch.cuda.Stream(), torch.zeros_like(y)
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y.zero_()
        side.wait_stream(torch.cuda.current_stream())
        qg.qgemm(fmt, W, n_out, n_in, x, z, other, stream=stream)                    # two at once, a workspace each
        qg.qgemm(fmt, W, n_out, n_in, x, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want)
    for early in (0, qg.QG_LAUNCH_EARLY_START):
        qg.qg_set_launch_options(early)
        graph = torch.cuda.CUDAGraph()
        y.zero_()
        z.zero_()
        with torch.cuda.graph(graph):
            qg.qgemm(fmt, W, n_out, n_in, x, y, ws)
            qg.qgemm(fmt, W, n_out, n_in, x, z, ws)                                  # one after the other: one workspace
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want)
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("fmt,act,n_out,n", [("q8_0", "bf16", 256, 40), ("q8_0", "f32", 5000, 900), ("bf16", "bf16", 128, 300)])
def test_a_wait_that_runs_out_is_reported(fmt, act, n_out, n):
    rng = np.random.default_rng(11)
    _, W = packed(rng, fmt, n_out, 1024)
    x = tokens(rng, n, 1024, act)
    ws = space(fmt, act, n_out, 1024, n)
    y, z = torch.zeros(n, n_out, dtype=DT[act], device="cuda"), torch.zeros(n, n_out, dtype=DT[act], device="cuda")
    qg.qgemm(fmt, W, n_out, 1024, x, y, ws)
    torch.cuda.synchronize()
    qg.qg_set_wait_limit(2000, 16)
    qg.qgemm(fmt, W, n_out, 1024, x, z, ws)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == qg.QG_DEVICE_WAIT_TIMEOUT
    qg.qg_set_wait_limit(0, 0)
    qg.qgemm(fmt, W, n_out, 1024, x, z, ws)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == 0 and torch.equal(y, z)


def test_no_tokens():
    y = torch.zeros(0, 64, device="cuda")
    rng = np.random.default_rng(12)
    _, W = packed(rng, "q8_0", 64, 64)
    qg.qgemm("q8_0", W, 64, 64, torch.zeros(0, 64, device="cuda"), y, space("q8_0", "f32", 64, 64, 0))


# ------------------------------------------------------------------------------------ experts

def spread_offsets(rng, n_experts, most, first=0):
    counts = rng.integers(0, most + 1, n_experts)
    counts[rng.integers(n_experts)] = 0                              # an expert without rows
    return np.concatenate([[first], first + np.cumsum(counts)])


EXPERTS = [  # n_experts, n_out, n_in, most rows, gather, f
    (1, 130, 64, 40, False, "none"), (7, 200, 640, 50, True, "swiglu"), (40, 128, 320, 3, True, "silu"), (16, 34, 1088, 260, False, "none"),
    (300, 6, 128, 4, True, "gelu")]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_experts,n_out,n_in,most,gather,f", EXPERTS)
def test_experts(fmt, act, n_experts, n_out, n_in, most, gather, f):
    rng = np.random.default_rng(n_experts + n_in)
    c, W = packed(rng, fmt, n_experts * n_out, n_in)
    off = spread_offsets(rng, n_experts, most, first=2)
    n_slots = int(off[-1]) + 3
    n_x = 29 if gather else n_slots
    x = tokens(rng, n_x, n_in, act)
    rows = rng.integers(0, n_x, n_slots)
    rows[:2] = rows[int(off[-1]):] = -5                              # slots of no expert: not looked at
    width = n_out // 2 if f == "swiglu" else n_out
    y = torch.full((n_slots, width), 9.0, dtype=DT[act], device="cuda")
    at = torch.tensor(rows, dtype=torch.int32, device="cuda") if gather else None
    qg.qgemm_experts(fmt, W, n_experts, n_out, n_in, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y,
                     space(fmt, act, n_out, n_in, n_slots, n_experts), rows=at, activation=f)
    args = (fmt, c, n_experts, n_out, n_in, host(x), off, rows if gather else None)
    v, S = PO.gemm_experts(*args), PO.gemm_experts(*args, product=PO.gemm_abs)
    got = host(y)
    for s in range(n_slots):
        if s not in v:
            assert (got[s] == 9.0).all()
            continue
        want = PO.activation(v[s], f)
        assert (np.abs(got[s] - want) <= tolerance(S[s], v[s], want, n_in, act, f)).all()
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("fmt,act", [("q8_0", "bf16"), ("q4_0", "f32"), ("bf16", "bf16")])
def test_few_experts_with_thousands_of_rows(fmt, act):
    rng = np.random.default_rng(33)
    n_out, n_in, n_x, off = 130, 64, 29, [0, 15001, 15001, 20000]
    c, W = packed(rng, fmt, 3 * n_out, n_in)
    x = tokens(rng, n_x, n_in, act)
    rows = rng.integers(0, n_x, off[-1])
    y = torch.zeros(off[-1], n_out, dtype=DT[act], device="cuda")
    qg.qgemm_experts(fmt, W, 3, n_out, n_in, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y,
                     space(fmt, act, n_out, n_in, off[-1], 3), rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    got = host(y)
    for e in (0, 2):                                                 # equal rows of an expert are equal
        first = {}
        for s in range(off[e], off[e + 1]):
            assert (got[s] == got[first.setdefault(rows[s], s)]).all()
        slots = sorted(first.values())
        args = (fmt, c, 3, n_out, n_in, host(x), [0] * (e + 1) + [len(slots)] * (3 - e), rows[slots])
        v, S = PO.gemm_experts(*args), PO.gemm_experts(*args, product=PO.gemm_abs)
        for i, s in enumerate(slots):
            assert (np.abs(got[s] - v[i]) <= tolerance(S[i], v[i], v[i], n_in, act, "none")).all()
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
def test_experts_with_rows_around_sixteens(fmt, act):
    """A tile takes its expert's rows in sixteens: one more, one less and just as many."""
    rng = np.random.default_rng(34)
    counts = [16, 1, 0, 15, 17, 31, 32, 33, 48, 49, 64, 100, 192, 193]
    n_experts, n_out, n_in, off = len(counts), 130, 576, [0] + list(np.cumsum(counts))
    c, W = packed(rng, fmt, n_experts * n_out, n_in)
    x = tokens(rng, int(off[-1]), n_in, act)
    y = torch.zeros(int(off[-1]), n_out, dtype=DT[act], device="cuda")
    qg.qgemm_experts(fmt, W, n_experts, n_out, n_in, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y,
                     space(fmt, act, n_out, n_in, int(off[-1]), n_experts))
    args = (fmt, c, n_experts, n_out, n_in, host(x), off)
    v, S = PO.gemm_experts(*args), PO.gemm_experts(*args, product=PO.gemm_abs)
    got = host(y)
    for s in range(int(off[-1])):
        assert (np.abs(got[s] - v[s]) <= tolerance(S[s], v[s], v[s], n_in, act, "none")).all()
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("off", [[0, 5, 3, 9], [-1, 2, 4, 6], [0, 4, 8, 11], [0, 2, 1, 0]])
def test_offsets_that_are_no_offsets(off):
    rng = np.random.default_rng(13)
    _, W = packed(rng, "q8_0", 3 * 16, 64)
    x = tokens(rng, 10, 64, "bf16")
    y = torch.full((10, 16), 9.0, dtype=torch.bfloat16, device="cuda")
    qg.qgemm_experts("q8_0", W, 3, 16, 64, x, torch.tensor(off, dtype=torch.int32, device="cuda"), y, space("q8_0", "bf16", 16, 64, 10, 3))
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PLAN and (y == 9.0).all()


def test_rows_that_are_no_rows():
    rng = np.random.default_rng(14)
    c, W = packed(rng, "q8_0", 2 * 16, 64)
    x = tokens(rng, 4, 64, "f32")
    rows = torch.tensor([0, 4, 3, -1], dtype=torch.int32, device="cuda")
    y = torch.full((4, 16), 9.0, device="cuda")
    qg.qgemm_experts("q8_0", W, 2, 16, 64, x, torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"), y, space("q8_0", "f32", 16, 64, 4, 2), rows=rows)
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PLAN
    assert (y[[1, 3]] == 0).all() and (y[[0, 2]] != 9.0).all() and (y[[0, 2]] != 0).any()


def test_binding_refuses():
    rng = np.random.default_rng(15)
    _, W = packed(rng, "q8_0", 64, 64)
    x, y, ws = tokens(rng, 8, 64, "f32"), torch.zeros(8, 64, device="cuda"), space("q8_0", "f32", 64, 64, 8, 2)
    off, bias = torch.tensor([0, 8], dtype=torch.int32, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (dict(x=x[:, :32]), dict(x=x.t()), dict(x=x[None]), dict(y=y[:4]), dict(y=y.bfloat16()), dict(y=y[:, :32]), dict(y=None), dict(bias=bias[:8]),
                dict(bias=bias.bfloat16()), dict(residual=y[:4]), dict(residual=y.bfloat16()), dict(W=W[:100]), dict(W=W.cpu()), dict(workspace=ws.cpu()),
                dict(activation="swiglu")):
        a = dict(fmt="q8_0", W=W, n_out=64, n_in=64, x=x, y=y, workspace=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            qg.qgemm(**a)
    with pytest.raises(qg.QGError):
        qg.qgemm("q8_0", W, 64, 64, x, y, ws[:16])
    with pytest.raises(qg.QGError):
        qg.qgemm("q8_0", W, 64, 64, x, y, None)
    for bad in (dict(offsets=off[:1]), dict(offsets=off.long()), dict(offsets=None), dict(rows=off), dict(y=y[:, :32]), dict(W=W[:100]), dict(n_experts=0)):
        a = dict(fmt="q8_0", W=W, n_experts=1, n_out=64, n_in=64, x=x, offsets=off, y=y, workspace=ws)
        a.update(bad)
        with pytest.raises((ValueError, qg.QGError)):
            qg.qgemm_experts(**a)
    torch.cuda.synchronize()
