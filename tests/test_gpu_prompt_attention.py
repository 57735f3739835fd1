"""GPU parity of qg_prompt_attention against the fp64 oracle, and a run of the prompt's calls
together with those of the cache.

Tolerances (derived from the arithmetic, before any run), with A = |scale| sum |q| |k| of a score, the
largest of the row's, and V = sum p |v|:
* a score is a sum of D products on the tensor cores in D / 16 additions that may cut off a bit: D / 16
  * 2^-23 A; fp32's terms carry 22 bits of the row's or tile's largest: 2^-20 A more.  The exponent's
  argument and the exponential: 2^-20.  ds is their sum; a probability is off by ds, an output by twice
  that of V.
* bf16: a probability rounded to bf16 2^-8, the additions of an output n / 16 * 2^-23, at most n of the
  keys; the output's rounding 2^-8 |out|.  fp32: two terms 2^-21, sums by tiles 2^-18 V; values have 22
  bits of their tile's largest, 2^-22 max |v|.
* lse: ds + 2^-21 |lse| + 2^-20.
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
    qg.qg_set_wait_limit(0, 0)
    qg.qg_set_launch_options(0)
    qg.qg_device_status(clear=True)


def host(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def space(act, n, hq, hk, D):
    return torch.full((qg.qg_prompt_attention_workspace_bytes(act, n, hq, hk, D),), 0xFF, dtype=torch.uint8, device="cuda")


def inputs(rng, n, hq, hk, D, act, size=1.0):
    x = torch.tensor(rng.standard_normal((n, hq + 2 * hk, D)) * size, dtype=torch.float32, device="cuda").to(DT[act])
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def run(q, k, v, cu, scale, window=0, lse=True, act=None):
    n, hq, D = q.shape
    out = torch.full((n, hq, D), 5.0, dtype=q.dtype, device="cuda")
    le = torch.full((n, hq), 5.0, device="cuda") if lse else None
    act = "f32" if q.dtype == torch.float32 else "bf16"
    longest = max(1, max(b - a for a, b in zip(cu[:-1], cu[1:])) if len(cu) > 1 else 1)
    qg.qg_prompt_attention(q, k, v, ints(cu), out, space(act, n, hq, k.shape[1], D), scale, longest, window=window, lse=le)
    return out, le


def check(q, k, v, cu, scale, window, out, lse, rows=None):
    act = "f32" if q.dtype == torch.float32 else "bf16"
    D, group = q.shape[2], q.shape[1] // k.shape[1]
    hq, hk, hv = host(q), host(k), host(v)
    want, wl, V = PO.prompt_attention(hq, hk, hv, cu, scale, window)
    got = host(out)
    inside = np.zeros(len(got), bool)
    inside[cu[0]:cu[-1]] = True
    assert (got[~inside] == 5.0).all() and (lse is None or (host(lse)[~inside] == 5.0).all())
    A, most = np.zeros(want.shape[:2]), np.zeros(want.shape[:2])
    for a, b in zip(cu[:-1], cu[1:]):
        for i in range(a, b):
            lo = max(a, i - window + 1) if window else a
            kk = np.abs(hk[lo:i + 1])
            A[i] = [abs(scale) * (kk[:, h // group] @ np.abs(hq[i, h])).max() for h in range(hq.shape[1])]
            most[i] = np.repeat(np.abs(hv[a:b]).max(axis=(0, 2)), group)
    ds = D / 16 * 2.0 ** -23 * A + 2.0 ** -20 + (2.0 ** -20 * A if act == "f32" else 0.0)
    n = int(max(b - a for a, b in zip(cu[:-1], cu[1:])))
    if act == "f32":
        t = (2 * ds + 2.0 ** -18 + 2.0 ** -21)[..., None] * V + 2.0 ** -22 * most[..., None]
    else:
        t = (2 * ds + 2.0 ** -8 + n / 16 * 2.0 ** -23)[..., None] * V + 2.0 ** -8 * np.abs(want)
    sel = inside if rows is None else rows
    assert (np.abs(got - want)[sel] <= t[sel] + 1e-30).all()
    if lse is not None:
        assert (np.abs(host(lse) - wl)[sel] <= (ds + 2.0 ** -21 * np.abs(wl) + 2.0 ** -20)[sel]).all()


CASES = [  # heads, kv_heads, D, lengths, window
    (1, 1, 128, [1], 0), (1, 1, 64, [2, 1, 3], 0), (4, 1, 128, [128], 0), (3, 1, 128, [43, 0, 85, 1], 0), (8, 2, 64, [65, 64, 63, 129], 0),
    (6, 2, 256, [70, 5, 131], 0), (2, 2, 128, [300], 0), (5, 5, 64, [17, 260], 0), (128, 1, 64, [9, 3], 0), (96, 1, 128, [12], 0),
    (4, 2, 128, [200, 7], 1), (4, 2, 128, [200, 70], 64), (6, 1, 64, [257, 33], 100), (2, 1, 256, [190], 65), (10, 2, 128, [150, 150], 1000)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,D,lens,window", CASES)
def test_attention(act, heads, kv, D, lens, window):
    rng = np.random.default_rng(sum(lens) + D)
    first = 3                                                        # tokens of no prompt before and behind
    cu = [first + sum(lens[:i]) for i in range(len(lens) + 1)]
    q, k, v = inputs(rng, cu[-1] + 4, heads, kv, D, act)
    out, lse = run(q, k, v, cu, D ** -0.5, window)
    check(q, k, v, cu, D ** -0.5, window, out, lse)
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale,size", [(-0.2, 1.0), (0.0, 1.0), (1.0, 4.0), (0.05, 30.0), (1e-3, 1e-3)])
def test_scores_of_any_size(act, scale, size):
    """Negative, zero and large factors: probabilities from even to a single key."""
    rng = np.random.default_rng(21)
    cu = [0, 150, 190]
    q, k, v = inputs(rng, 190, 4, 2, 128, act, size)
    out, lse = run(q, k, v, cu, scale)
    check(q, k, v, cu, scale, 0, out, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp32_rows_keys_and_prompts_of_other_sizes(D):
    """Each query row, key tile and prompt has its own power of two."""
    rng = np.random.default_rng(22)
    cu = [0, 100, 230, 240]
    q, k, v = inputs(rng, 240, 4, 2, D, "f32")
    k, v, q = k.clone(), v.clone(), q.clone()
    q *= torch.tensor(10.0 ** rng.integers(-3, 1, (240, 4, 1)), device="cuda").float()
    for (a, b), s in zip(zip(cu[:-1], cu[1:]), (1e-12, 1e9, 1.0)):
        v[a:b] *= s
        k[a:b] *= 0.5
    out, lse = run(q, k, v, cu, 0.1)
    check(q, k, v, cu, 0.1, 0, out, lse)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_places_may_hold_anything(act, D):
    """NaN and infinities in later tokens, in other prompts and behind the last one reach no row that
    does not see them."""
    rng = np.random.default_rng(23)
    cu = [2, 90, 150]
    q, k, v = [t.clone() for t in inputs(rng, 200, 4, 2, D, act)]
    clean, lse_clean = run(q, k, v, cu, 0.1)
    bad = float("nan"), float("inf"), float("-inf")
    for t in (q, k, v):
        t[:2], t[150:] = float("nan"), float("inf")                  # padding
    v[60, 0, 5], v[75, 0, 9], v[140, 1, 3] = bad                     # values of tokens that later ones see
    k[80, 1, 7] = float("nan")
    out, lse = run(q, k, v, cu, 0.1)
    o, c = host(out), host(clean)
    touched = np.zeros((200, 4, D), bool)
    touched[60:90, :2, 5] = touched[75:90, :2, 9] = touched[140:150, 2:, 3] = True
    touched[80:90, 2:] = True
    inside = np.zeros(200, bool)
    inside[2:150] = True
    assert not np.isfinite(o[touched & inside[:, None, None]]).any()
    same = ~touched & inside[:, None, None]
    assert np.array_equal(o[same], c[same])
    assert (o[~inside] == 5.0).all()
    assert np.isnan(o[60:90, :2, 5]).all() and (o[140:150, 2:, 3] == -np.inf).all()
    keep = np.ones((200, 4), bool)
    keep[80:90, 2:] = False
    assert np.array_equal(host(lse)[2:150][keep[2:150]], host(lse_clean)[2:150][keep[2:150]])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_windows_hide_what_is_not_finite(act):
    rng = np.random.default_rng(24)
    q, k, v = [t.clone() for t in inputs(rng, 300, 2, 1, 128, act)]
    v[100, 0, 1] = float("inf")
    out, _ = run(q, k, v, [0, 300], 0.1, window=50)
    o = host(out)
    assert np.isfinite(o[:100]).all() and np.isfinite(o[150:]).all()
    assert (o[100:150, :, 1] == np.inf).all() and np.isfinite(np.delete(o, 1, axis=2)).all()


def test_bad_prompts_are_reported():
    rng = np.random.default_rng(25)
    q, k, v = inputs(rng, 40, 2, 1, 64, "bf16")
    for cu in ([0, 20, 10, 40], [-1, 20, 40], [0, 20, 41]):
        out, _ = run(q, k, v, cu, 0.1, lse=False)
        assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH
        assert torch.isfinite(out).all()
    out, lse = run(q, k, v, [0], 0.1)
    assert (out == 5.0).all() and qg.qg_device_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_the_same_on_every_run_stream_and_replay(act):
    rng = np.random.default_rng(26)
    cu = [0, 260, 261, 700]
    q, k, v = inputs(rng, 700, 8, 2, 128, act)
    want, wl = run(q, k, v, cu, 0.1)
    for _ in range(3):
        out, lse = run(q, k, v, cu, 0.1)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    ws, other, c = space(act, 700, 8, 2, 128), space(act, 700, 8, 2, 128), ints(cu)
    out, two = torch.full_like(want, 5.0), torch.full_like(want, 5.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qg.qg_prompt_attention(q, k, v, c, two, other, 0.1, 439, stream=side)
    qg.qg_prompt_attention(q, k, v, c, out, ws, 0.1, 1)              # (any `longest` is right)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(two, want)
    for early in (0, qg.QG_LAUNCH_EARLY_START):
        qg.qg_set_launch_options(early)
        out.zero_()
        two.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qg.qg_prompt_attention(q, k, v, c, out, ws, 0.1, 439)
            qg.qg_prompt_attention(q, k, v, c, two, ws, 0.1, 439)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(two, want)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_is_reported(act, D):
    rng = np.random.default_rng(27)
    q, k, v = inputs(rng, 900, 4, 2, D, act)
    want, _ = run(q, k, v, [0, 400, 900], 0.1)
    torch.cuda.synchronize()
    qg.qg_set_wait_limit(2000, 16)
    run(q, k, v, [0, 400, 900], 0.1)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == qg.QG_DEVICE_WAIT_TIMEOUT
    qg.qg_set_wait_limit(0, 0)
    out, _ = run(q, k, v, [0, 400, 900], 0.1)
    assert torch.equal(out, want) and qg.qg_device_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_items_than_run_at_once(act, D):
    """CTAs take items that others would have had: hundreds of short prompts around a longer one, some
    empty; the same bits every time, and a wait that runs out in such a call ends all of it."""
    rng = np.random.default_rng(31)
    lens = list(rng.integers(0, 8, 500))
    lens[200] = 300
    cu = [int(sum(lens[:i])) for i in range(len(lens) + 1)]
    q, k, v = inputs(rng, cu[-1], 4, 2, D, act)
    out, lse = run(q, k, v, cu, D ** -0.5)
    check(q, k, v, cu, D ** -0.5, 0, out, lse)
    for _ in range(3):
        again, l2 = run(q, k, v, cu, D ** -0.5)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    qg.qg_set_launch_options(qg.QG_LAUNCH_EARLY_START)
    many = [run(q, k, v, cu, D ** -0.5)[0] for _ in range(4)]
    qg.qg_set_launch_options(0)
    assert all(torch.equal(m, out) for m in many)
    assert qg.qg_device_status() == 0
    qg.qg_set_wait_limit(2000, 16)
    run(q, k, v, cu, D ** -0.5)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == qg.QG_DEVICE_WAIT_TIMEOUT
    qg.qg_set_wait_limit(0, 0)
    again, _ = run(q, k, v, cu, D ** -0.5)
    assert torch.equal(again, out) and qg.qg_device_status() == 0


@pytest.mark.parametrize("at", [0, 31, 32, 400])
def test_one_wrong_length_among_many_prompts(at):
    """It is reported wherever it stands."""
    rng = np.random.default_rng(32)
    cu = list(range(0, 2 * 402, 2))
    q, k, v = inputs(rng, cu[-1], 2, 2, 64, "bf16")
    run(q, k, v, cu, 0.1)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == 0
    bad = list(cu)
    bad[at + 1] = -7
    run(q, k, v, bad, 0.1)
    torch.cuda.synchronize()
    assert qg.qg_device_status() & qg.QG_DEVICE_BAD_LENGTH


def test_binding_refuses():
    rng = np.random.default_rng(28)
    q, k, v = inputs(rng, 20, 4, 2, 64, "bf16")
    ok = dict(q=q, k=k, v=v, cu_seq=ints([0, 20]), out=torch.zeros(20, 4, 64, dtype=torch.bfloat16, device="cuda"), workspace=space("bf16", 20, 4, 2, 64),
              scale=0.1, longest=20)
    for bad in (dict(k=k.float()), dict(v=v[:10]), dict(k=None), dict(out=None), dict(v=k[:, :1]), dict(out=ok["out"][:10]), dict(out=ok["out"][:, :2]),
                dict(cu_seq=ints([0, 20]).long()), dict(cu_seq=ints([0, 20])[None]), dict(cu_seq=ints([])), dict(lse=torch.zeros(20, device="cuda")),
                dict(workspace=ok["workspace"].cpu()), dict(q=q.transpose(0, 1)), dict(q=q[..., ::2])):
        with pytest.raises(ValueError):
            qg.qg_prompt_attention(**{**ok, **bad})
    with pytest.raises(qg.QGError):
        qg.qg_prompt_attention(**{**ok, "workspace": None})
    with pytest.raises(qg.QGError):
        qg.qg_prompt_attention(**{**ok, "longest": 0})
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_prompt_through_a_layer_and_on(act):
    """Projection, page table, store, attention, output projection and experts of two prompts; then
    their last tokens attend once more over the cache, which holds what the prompts' attention read."""
    rng = np.random.default_rng(30)
    lens, page, heads, kv, D, width = [70, 33], 16, 6, 2, 128, 192
    n, n_pages, rows = sum(lens), 12, heads + 2 * kv
    c_qkv = oracle.quantize("q8_0", (rng.standard_normal((rows * D, width)) * 0.05).astype(np.float32))
    c_out = oracle.quantize("q4_0", (rng.standard_normal((width, heads * D)) * 0.05).astype(np.float32))
    W_qkv = torch.from_numpy(qg.qg_to_device_layout("q8_0", c_qkv, rows * D, width)).cuda()
    W_out = torch.from_numpy(qg.qg_to_device_layout("q4_0", c_out, width, heads * D)).cuda()
    x = torch.tensor(rng.standard_normal((n, width)), dtype=torch.float32, device="cuda").to(DT[act])
    i32 = dict(dtype=torch.int32, device="cuda")
    held, begin, table = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.full((2, 8), -1, **i32)
    free, seq, cu = torch.arange(n_pages, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32)
    slots, pos = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, **i32)
    pool = torch.zeros(qg.qg_cache_bytes(n_pages, page, kv, D), dtype=torch.uint8, device="cuda")
    cache = qg.qg_cache(pool, n_pages, page, kv, D)
    angle = rng.uniform(0, 6.0, (100, D // 2))
    cs = torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32, device="cuda")
    gemm_ws = torch.empty(max(qg.qgemm_workspace_bytes("q8_0", act, rows * D, width, n), qg.qgemm_workspace_bytes("q4_0", act, width, heads * D, n)),
                          dtype=torch.uint8, device="cuda")

    qg.qg_cache_pages(held, ints(lens), free, table, seq, cu, slots, pos, page, free_begin=begin, free_end=begin)
    qkv = torch.empty(n, rows, D, dtype=DT[act], device="cuda")
    qg.qgemm("q8_0", W_qkv, rows * D, width, x, qkv.view(n, -1), gemm_ws)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    k_back, v_back = [torch.empty(n, kv, D, dtype=DT[act], device="cuda") for _ in range(2)]
    qg.qg_cache_append(cache, k, v, slots, q=q, q_out=q, positions=pos, cos_sin=cs, k_back=k_back, v_back=v_back)
    out = torch.full((n, heads, D), 5.0, dtype=DT[act], device="cuda")
    lse = torch.full((n, heads), 5.0, device="cuda")
    qg.qg_prompt_attention(q, k_back, v_back, cu, out, space(act, n, heads, kv, D), D ** -0.5, max(lens), lse=lse)
    y = x.clone()
    qg.qgemm("q4_0", W_out, width, heads * D, out.view(n, -1), y, gemm_ws, residual=y)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == 0 and cu.tolist() == [0, 70, 103]
    check(q, k_back, v_back, [0, 70, 103], D ** -0.5, 0, out, lse)
    want = PO.gemm("q4_0", c_out, width, heads * D, host(out).reshape(n, -1), residual=host(x))
    S = PO.gemm_abs("q4_0", c_out, width, heads * D, host(out).reshape(n, -1))
    t = S * (2.0 ** -11 + heads * D / 16 * 2.0 ** -23 if act == "bf16" else 2.0 ** -17) + 2.0 ** -19 * np.abs(want) + (2.0 ** -8 * np.abs(want) if act == "bf16" else 0)
    assert (np.abs(host(y) - want) <= t).all()

    # The last tokens over the cache: the same keys and values, another kernel.
    last = torch.tensor([69, 102], device="cuda")
    q1, o1, l1 = q[last].contiguous(), torch.empty(2, heads, D, dtype=DT[act], device="cuda"), torch.empty(2, heads, device="cuda")
    ws = torch.zeros(qg.qg_attention_workspace_bytes(heads, kv, D), dtype=torch.uint8, device="cuda")
    qg.qg_attention(cache, q1, table, seq, ints([0, 1, 2]), o1, ws, D ** -0.5, max_new=1, lse=l1)
    # A cached key is a 4-bit code times a scale of 8 significant bits, 12 bits together.  In fp32 k_back holds
    # it; in bf16 it is rounded to 8 bits, 2^-8 of each value at most (values likewise): a score of the
    # prompt's attention is off by 2^-8 of A = scale sum |q| |k|, lse by as much, a probability by that factor.
    # The kernels themselves are within 2^-18 A + 2^-19 (fp32) of the score; bf16 rounds probabilities (2^-8
    # and 2^-11) and outputs (2^-8 each).
    group, hq, hk = heads // kv, host(q1), host(k_back)
    A = max(D ** -0.5 * (np.abs(hk[a:b, h // group]) @ np.abs(hq[i, h])).max() for i, (a, b) in enumerate(((0, 70), (70, 103))) for h in range(heads))
    ds, rounding = (2.0 ** -8 * A + 2.0 ** -12, 5 * 2.0 ** -8) if act == "bf16" else (2.0 ** -18 * A + 2.0 ** -19, 2.0 ** -17)
    assert np.abs(host(o1) - host(out[last])).max() <= (2 * ds + rounding) * np.abs(host(v_back)).max()
    assert np.abs(host(l1) - host(lse[last])).max() <= ds + 2.0 ** -18
