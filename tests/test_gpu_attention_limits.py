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


# ------------------------------------------------------------------------------------ the division of work

def expect_row(c, tok, h):
    """Output, its tolerance and the log-sum-exp of query head h of token tok (as Case.expect)."""
    r = int(np.searchsorted(c.cu, tok, side="right")) - 1
    s, j, hk = c.seq[r], tok - int(c.cu[r]), h // (c.heads // c.kv)
    see = AO.visible(s, s, c.fresh[r], j, c.window)
    if (r, hk) not in c.loaded:
        c.loaded[r, hk] = AO.kv_load(c.pool.cpu().numpy(), c.slots[r], hk, c.page, c.kv, c.D)
    K, V = c.loaded[r, hk]
    d = np.abs(K).reshape(s, -1, 32).max(-1).repeat(32, -1) / 7.0
    row = host(c.q)[tok, h]
    o, l, p = AO.attention(row, K, V, see, c.scale)
    ds = 2.0 ** -19 * abs(c.scale) * 23 * (d[see] @ np.abs(row)) + 2.0 ** -20
    return o, (2 * ds.max() + 2.0 ** -19) * (p @ np.abs(V[see])) + 2.0 ** -32 * np.abs(V[see]).sum(0), l


def test_a_long_chunk_in_a_large_batch():
    """A chunk takes as much of a launch as it needs, whatever the number of requests beside it:
    here 2.1 million places of work, more than 2^31 / 1024, beside 1023 single tokens."""
    n = 1024
    held, fresh = [5] * n, [1] * n
    held[300], fresh[300] = 65600, 1024
    c = Case(71, 64, 16, 2, held, fresh, page=64)
    c.loaded = {}
    got = host(c.run())
    assert qg.qg_device_status() == 0
    assert (2053 + 4) * (1024 * 8 // 16) * 2 > (1 << 31) // n
    at = int(c.cu[300])
    for tok in (0, 299, at, at + 1, at + 500, at + 1023, at + 1024, c.n_tok - 1):
        for h in (0, 9, 15):
            o, tol, _ = expect_row(c, tok, h)
            assert np.all(np.abs(got[tok, h] - o) <= tol), (tok, h)


def long_table(rows, width):
    """Every page of every request is page 0: a cache of 65536 tokens stands for any length."""
    return torch.zeros(rows, width, dtype=torch.int32, device=dev())


class LongCase:
    """One key/value head of 64 in a single page of 65536 tokens, which every entry of the tables names."""
    D, PAGE = 64, 65536

    def __init__(self, seed, rows):
        self.rng = np.random.default_rng(seed)
        pool = torch.zeros(qg.qg_cache_bytes(1, self.PAGE, 1, self.D), dtype=torch.uint8, device=dev())
        self.pool, self.cache = pool, qg.qg_cache(pool, 1, self.PAGE, 1, self.D)
        k, v = [torch.tensor(self.rng.standard_normal((self.PAGE, 1, self.D)).astype(np.float32), device=dev()) for _ in range(2)]
        qg.qg_cache_append(self.cache, k, v, torch.arange(self.PAGE, device=dev()), norm=False)
        self.q = torch.tensor(self.rng.standard_normal((rows, 1, self.D)).astype(np.float32), device=dev())
        self.ws = torch.zeros(qg.qg_attention_workspace_bytes(1, 1, self.D), dtype=torch.uint8, device=dev())

    def run(self, seq, cu, window=0, max_new=4):
        out = torch.full_like(self.q, 7)
        self.lse = torch.full((self.q.shape[0], 1), 7.0, device=dev())
        qg.qg_attention(self.cache, self.q, long_table(len(seq), (max(seq) + self.PAGE - 1) // self.PAGE), ints(seq), ints(cu), out, self.ws,
                        self.D ** -0.5, max_new=max_new, window=window, lse=self.lse)
        return out

    def check_row(self, got, tok, pos, window):
        keys = np.arange(max(0, pos - window + 1), pos + 1, dtype=np.int64)
        K, V = AO.kv_load(self.pool.cpu().numpy(), keys % self.PAGE, 0, self.PAGE, 1, self.D)
        row = host(self.q)[tok, 0]
        o, l, p = AO.attention(row, K, V, np.ones(len(keys), bool), self.D ** -0.5)
        d = np.abs(K).reshape(len(keys), -1, 32).max(-1).repeat(32, -1) / 7.0
        ds = 2.0 ** -19 * self.D ** -0.5 * 23 * (d @ np.abs(row)) + 2.0 ** -20
        assert np.all(np.abs(host(got)[tok, 0] - o) <= (2 * ds.max() + 2.0 ** -19) * (p @ np.abs(V)) + 2.0 ** -32 * np.abs(V).sum(0)), (tok, pos)
        assert abs(float(self.lse[tok, 0]) - l) <= ds.max() + 2.0 ** -20 * max(1.0, abs(l))


def test_only_what_does_not_fit_a_launch_is_left_out():
    """The work of a call is numbered with 31 bits: a request that no longer fits is reported and its
    rows stay as they are; those before and after it are computed."""
    last = (1 << 31) - 160                                   # (2^26 - 5 + 4) places a tile, 32 tiles of 4: 2^31 - 32
    fresh = [1] * 8 + [128, 1, 2]
    cu = np.concatenate([[0], np.cumsum(fresh)]).tolist()
    seq = [10 * (i + 1) for i in range(8)] + [last, 33, 40]
    c = LongCase(5, cu[-1])
    got = c.run(seq, cu)
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH
    assert bool((got[8:136] == 7).all()) and bool((c.lse[8:136] == 7).all())
    for r in [0, 1, 7, 9, 10]:
        for j in range(fresh[r]):
            pos = seq[r] - fresh[r] + j
            c.check_row(got, cu[r] + j, pos, pos + 1)
    # The same in a batch of more requests than a warp has lanes.
    fresh2, seq2 = [1] * 40 + fresh, [7] * 40 + seq
    c2 = LongCase(6, 40 + cu[-1])
    cu2 = np.concatenate([[0], np.cumsum(fresh2)]).tolist()
    got = c2.run(seq2, cu2)
    assert qg.qg_device_status(clear=True) == qg.QG_DEVICE_BAD_LENGTH
    assert bool((got[48:176] == 7).all())
    for tok, pos in ((0, 6), (39, 6), (40, 9), (176, 32), (178, 39)):
        c2.check_row(got, tok, pos, pos + 1)
    assert int(c.ws[:qg.QG_ATTENTION_ZERO_BYTES].max()) == 0 and int(c2.ws[:qg.QG_ATTENTION_ZERO_BYTES].max()) == 0


def test_more_requests_than_a_call_takes():
    """A batch in several calls: table, lengths and offsets advanced, queries and outputs as they are."""
    rng = np.random.default_rng(72)
    n = 1500
    c = Case(72, 64, 2, 1, rng.integers(0, 20, n).tolist(), rng.integers(0, 3, n).tolist(), page=16)
    cache = qg.qg_cache(c.pool, c.n_pages, 16, 1, 64)
    table, seq, cu = ints(c.table.ravel()).view(c.table.shape), ints(c.seq), ints(c.cu)
    out, c.lse = torch.full_like(c.q, 7), torch.full((c.n_tok, 2), 7.0, device=dev())
    c.ws = torch.zeros(qg.qg_attention_workspace_bytes(2, 1, 64), dtype=torch.uint8, device=dev())
    for r0, r1 in ((0, 1024), (1024, n)):
        qg.qg_attention(cache, c.q, table[r0:r1], seq[r0:r1], cu[r0:r1 + 1], out, c.ws, c.scale, max_new=2, lse=c.lse)
    c.check(out)


# ------------------------------------------------------------------------------------ lengths

@pytest.mark.parametrize("window", [0, 5])
def test_lengths_below_the_new_tokens_are_reported(window):
    """A request cannot have fewer tokens in the cache than it adds: it is left out."""
    c = Case(43, 128, 4, 2, [40, 20, 30], [3, 2, 1], page=16, window=window)
    want = c.run()
    for short in (0, 1, 2):
        got = c.run(seq=ints([short, 22, 31]))
        assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH
        assert bool((got[:3] == 7).all()) and torch.equal(got[3:], want[3:])
    c.check(c.run())


def test_lengths_near_the_end_of_32_bits():
    """Positions up to 2^31 - 2 through a table whose entries all name one page; windows up to 2^31 - 1."""
    for last in ((1 << 31) - 1, (1 << 31) - 2, (1 << 31) - 16, (1 << 31) - 17, (1 << 31) - 33):
        c = LongCase(last % 97, 5)
        got = c.run([last, 900], [0, 3, 5], window=100)
        assert qg.qg_device_status() == 0
        for tok, pos in ((0, last - 3), (1, last - 2), (2, last - 1), (3, 898), (4, 899)):
            c.check_row(got, tok, pos, 100)
    got = c.run([700, 900], [0, 3, 5], window=(1 << 31) - 1)
    assert qg.qg_device_status() == 0
    for tok, pos in ((0, 697), (1, 698), (2, 699), (3, 898), (4, 899)):
        c.check_row(got, tok, pos, (1 << 31) - 1)


# ------------------------------------------------------------------------------------ scores

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D,heads,new", [(64, 1, 1), (128, 2, 4), (128, 12, 1), (256, 3, 2)])
@pytest.mark.parametrize("power", [12, 16, 22, 26, 27, 28, 30, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_apart(act, D, heads, new, power, sign):
    """Scores that are whole multiples of 2^power, exact in every step: the keys with the largest share
    the weight, all others have none (exp(-2^12) is 0 in any of the formats).  Error: two fp16 terms
    of a probability and the sums, 2^-18 of the largest value; bf16: 2^-11 and the output's 2^-8."""
    c = Case(power + D, D, heads, 1, [333, 2, 90], [new, 1, new], page=32, act=act, v_scale=1.0, scale=1.0)
    c.k[:] = -8.0                                            # every block has the scale 1
    c.k[:, :, 0] = c.rng.integers(-8, 8, c.k.shape[:2])
    c.append()
    c.q.zero_()
    c.q[:, :, 0] = sign * 2.0 ** power
    got = host(c.run())
    want, _, lse, _ = c.expect()
    assert np.all(np.isfinite(got))
    assert np.abs(got - want).max() <= (2.0 ** -18 if act == "f32" else 2.0 ** -7) * np.abs(c.v).max()
    gl = host(c.lse)[:c.n_tok]
    assert np.all(np.abs(gl - lse) <= 2.0 ** -20 * np.abs(lse) + 2.0 ** -18)
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("q_scale", [1e3, 1e6, 3e7, 1e8, 1e9, 1e12])
@pytest.mark.parametrize("spread", [0.0, 1e-4])
def test_large_scores_weigh_no_more_than_one(q_scale, spread):
    """Scores up to 10^13 that differ by a few of their own last bits (the keys are copies of one, but for
    a small share): whatever the rounding, outputs are weighted means of the values."""
    c = Case(57, 128, 6, 2, [700, 40], [2, 4], page=32, v_scale=1.0, scale=0.3, q_scale=q_scale)
    c.k[:] = c.k[:1] + spread * c.k
    c.append()
    got = host(c.run())
    V = AO.kv_load(c.pool.cpu().numpy(), np.concatenate(c.slots), 0, c.page, c.kv, c.D)[1]
    V1 = AO.kv_load(c.pool.cpu().numpy(), np.concatenate(c.slots), 1, c.page, c.kv, c.D)[1]
    top = max(np.abs(V).max(), np.abs(V1).max())
    assert np.all(np.isfinite(got)) and np.abs(got).max() <= top * (1 + 2.0 ** -18)
    if spread == 0.0:                                        # equal keys, equal scores: the plain mean of what a row sees
        for r, (s, f) in enumerate(zip(c.seq, c.fresh)):
            at = int(sum(c.seq[:r]))
            for j in range(f):
                n = s - f + j + 1
                for h in range(6):
                    want = (V, V1)[h // 3][at:at + n].mean(0)
                    assert np.abs(got[int(c.cu[r]) + j, h] - want).max() <= 2.0 ** -18 * top


@pytest.mark.parametrize("q_scale,scale", [(0.0, 1e-20), (0.0, 1.0), (0.0, 1e38), (1e-30, 1e-15), (1e-38, 1e-38), (1.0, 1e-38),
                                           (1e-33, 1e33), (1e30, 1e-30), (1e-38, 3e38)])
def test_scales_of_every_size(q_scale, scale):
    """Masked units, rows of zeros and scales whose product with a query leaves fp32's range on the way."""
    c = Case(61, 128, 6, 2, [90, 3, 0], [2, 1, 3], q_scale=q_scale, scale=scale)
    c.check(c.run())


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_zero_scores_of_large_queries(act):
    """Keys of zeros: every score is 0, however large a query times the scale is."""
    c = Case(62, 128, 6, 2, [90, 3], [2, 1], q_scale=1e30, scale=1e10, act=act)
    c.k[:] = 0
    c.append()
    c.check(c.run())


# ------------------------------------------------------------------------------------ pages

PAGES = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
from test_gpu_attention import AO, run_pages, qg
for n in {sizes}:
    rng = np.random.default_rng(n)
    held, fresh = rng.integers(0, 40, n), rng.integers(0, 3, n)
    table = np.full((n, 3), -1)
    count = -(-held // 16)
    for r in range(n):
        table[r, :count[r]] = 100000 + 3 * r + np.arange(count[r])
    free = rng.permutation(n + 5)
    want = AO.cache_pages(held.tolist(), fresh.tolist(), free, 2, table, 16, int(fresh.sum()) + 1)
    got = run_pages(held, fresh, free, table, 16, int(fresh.sum()) + 1, begin=2, in_place={in_place})
    for w, g in zip(want, got):
        assert np.array_equal(np.asarray(w).reshape(-1), g.reshape(-1)), n
    assert qg.qg_device_status() == 0
print("same")
"""


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_of_every_number_of_requests(in_place):
    """Where the prefix arrays and the kernel's own shared memory together pass 48 KB (in a process of its own:
    a larger call before would raise the limit for the smaller ones)."""
    code = PAGES.format(root=ROOT, tests=os.path.join(ROOT, "tests"), sizes=[6111, 6112, 6143, 6144, 16384], in_place=in_place)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


@pytest.mark.parametrize("in_place", [False, True])
def test_a_free_page_that_is_none_is_reported(in_place):
    """A negative number in the list of free pages: its tokens have no slot, and the status says so."""
    t, seq, cu, slots, pos, end = run_pages([0, 3], [20, 2], [5, -1, 6], [[-1, -1], [9, -1]], 16, 22, begin=0, in_place=in_place)
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE
    assert slots[:16].tolist() == list(range(80, 96)) and (slots[16:20] == -1).all() and slots[20:].tolist() == [147, 148]
    assert cu.tolist() == [0, 20, 22] and seq.tolist() == [20, 5] and end[0] == 2


# ------------------------------------------------------------------------------------ tensors

class Elsewhere(torch.Tensor):
    """A tensor that says it is on another GPU; it has no memory, so nothing can be launched with it."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_wrapper_subclass(cls, t.shape, strides=t.stride(), dtype=t.dtype,
                                                   device=f"cuda:{torch.cuda.current_device() + 1}")

    __torch_dispatch__ = None


def test_tensors_of_another_device_are_refused():
    """Kernels go to the current device: every tensor of a call has to be there."""
    c = Case(63, 128, 4, 2, [40], [2], page=16)
    cache = qg.qg_cache(c.pool, c.n_pages, 16, 2, 128)
    n = c.seq[0]
    f = lambda *s: torch.ones(*s, device=dev())  # noqa: E731
    calls = [
        (qg.qg_cache_pages, dict(held=ints([1]), fresh=ints([1]), free_pages=ints([0]), table=ints([0]).view(1, 1), seq_len=ints([0]),
                                 cu_new=ints([0, 0]), slots=ints([0]).long(), positions=ints([0]), page_tokens=16, free_begin=ints([0]),
                                 free_end=ints([0]))),
        (qg.qg_qk_norm_rope, dict(q=c.q, k=c.q, q_out=f(2, 4, 128), k_out=f(2, 4, 128), positions=ints([0, 0]), cos_sin=f(4, 128),
                                  q_weight=f(128), k_weight=f(128))),
        (qg.qg_cache_append, dict(cache=cache, k=f(n, 2, 128), v=f(n, 2, 128), slots=torch.tensor(c.slots[0], device=dev()), q=f(n, 4, 128),
                                  q_out=f(n, 4, 128), positions=ints([0] * n), cos_sin=f(4, 128), q_weight=f(128), k_weight=f(128),
                                  k_back=f(n, 2, 128), v_back=f(n, 2, 128))),
        (qg.qg_attention, dict(cache=cache, q=c.q, table=ints(c.table.ravel()).view(c.table.shape), seq_len=ints(c.seq), cu_new=ints(c.cu),
                               out=f(2, 4, 128), workspace=torch.zeros(qg.qg_attention_workspace_bytes(4, 2, 128), dtype=torch.uint8, device=dev()),
                               scale=0.1, span_mask=ints([1, 3]), lse=f(2, 4)))]
    for call, good in calls:
        call(**good)
        for name, t in good.items():
            if torch.is_tensor(t):
                with pytest.raises(ValueError, match=f"{name}: not on the current CUDA device"):
                    call(**{**good, name: Elsewhere(t)})
        if "cache" in good:
            other = qg.qg_cache(c.pool, c.n_pages, 16, 2, 128)
            other.device += 1                                # as if its tensor were there
            with pytest.raises(ValueError, match="cache: not on the current CUDA device"):
                call(**{**good, "cache": other})
            call(**{**good, "cache": qg.qg_cache(c.pool.data_ptr(), c.n_pages, 16, 2, 128)})
    assert qg.qg_device_status() == 0


def test_one_token_may_have_any_stride():
    """The distance of the next token means nothing where there is none."""
    c = Case(67, 128, 4, 2, [50], [1], page=16)
    want = c.run()
    for extra in (1, 2, 130):
        wide = torch.zeros(1, 4 * 128 + extra, device=dev())
        wide[:, :512] = c.q.view(1, 512)
        q = wide.as_strided((1, 4, 128), (4 * 128 + extra, 128, 1))
        assert torch.equal(c.run(q=q), want)
        out = torch.zeros(1, 4 * 128 + extra, device=dev()).as_strided((1, 4, 128), (4 * 128 + extra, 128, 1))
        assert torch.equal(c.run(out=out), want)
        k0, k1 = torch.empty_like(c.q), torch.empty_like(c.q)
        qg.qg_qk_norm_rope(q, q, k0, k1)
        a0, a1 = torch.empty_like(c.q), torch.empty_like(c.q)
        qg.qg_qk_norm_rope(c.q, c.q, a0, a1)
        assert torch.equal(k0, a0) and torch.equal(k1, a1)


def test_one_token_as_a_bf16_row():
    c = Case(67, 64, 2, 1, [50], [1], page=16, act="bf16")
    want = c.run()
    wide = torch.zeros(1, 2 * 64 + 3, device=dev(), dtype=torch.bfloat16)
    q = wide.as_strided((1, 2, 64), (131, 64, 1))
    q.copy_(c.q)
    assert torch.equal(c.run(q=q), want)


def test_append_over_its_inputs():
    """What the cache now holds, written over the keys and values it was made of."""
    rng = np.random.default_rng(68)
    x = heads_input(rng, 40, 4, 2, 64, "f32", hv=2)
    q, k, v = [t.contiguous() for t in (x[:, :4], x[:, 4:6], x[:, 6:])]
    slots, pos, cs = torch.arange(40, device=dev()), ints(range(40)), torch.tensor(rotation(rng, 40, 64), device=dev())
    pools, outs = [], []
    for over in (False, True):
        pool = torch.zeros(AO.pool_bytes(3, 16, 2, 64), dtype=torch.uint8, device=dev())
        qq, kk, vv = q.clone(), k.clone(), v.clone()
        qo, kb, vb = (qq, kk, vv) if over else [torch.empty_like(t) for t in (qq, kk, vv)]
        qg.qg_cache_append(qg.qg_cache(pool, 3, 16, 2, 64), kk, vv, slots, q=qq, q_out=qo, positions=pos, cos_sin=cs, k_back=kb, v_back=vb)
        pools.append(pool)
        outs.append((qo, kb, vb))
    assert torch.equal(*pools) and all(torch.equal(a, b) for a, b in zip(*outs))
    wide = torch.randn(4, 6, 128, device=dev())
    with pytest.raises(qg.QGError):                          # the same first row, tokens at another distance
        qg.qg_qk_norm_rope(wide[:, :4], wide[:, 4:], wide.view(-1)[:4 * 4 * 128].view(4, 4, 128), torch.empty(4, 2, 128, device=dev()))


def test_append_of_positions_that_are_none():
    """A negative position, or one past the table of angles, stores zeros; the latter is reported."""
    rng = np.random.default_rng(69)
    x = heads_input(rng, 3, 0, 1, 64, "f32", hv=1)
    cs = torch.tensor(rotation(rng, 10, 64), device=dev())
    for bad, status in ((-1, 0), (10, qg.QG_DEVICE_BAD_LENGTH)):
        pool = torch.full((AO.pool_bytes(1, 16, 1, 64),), 0xFF, dtype=torch.uint8, device=dev())
        kb, vb = [torch.full((3, 1, 64), 7.0, device=dev()) for _ in range(2)]
        qg.qg_cache_append(qg.qg_cache(pool, 1, 16, 1, 64), x[:, :1], x[:, 1:], torch.arange(3, device=dev()), positions=ints([4, bad, 9]),
                           cos_sin=cs, k_back=kb, v_back=vb)
        assert qg.qg_device_status() == status
        K, V = AO.kv_load(pool.cpu().numpy(), [0, 1, 2], 0, 16, 1, 64)
        assert not K[1].any() and not V[1].any() and K[[0, 2]].any(1).all() and np.isfinite(K).all() and np.isfinite(V).all()
        assert not bool(kb[1].any()) and not bool(vb[1].any())
        assert np.array_equal(host(kb)[:, 0], K) and np.array_equal(host(vb)[:, 0], V)


# ------------------------------------------------------------------------------------ branches that other tests do not reach

@pytest.mark.parametrize("n,hq,hk,D,rot,act,norm", [
    (3, 2, 1, 64, 48, "f32", True), (40, 6, 2, 128, 96, "f32", True), (5, 3, 3, 128, 112, "bf16", True), (7, 2, 1, 256, 144, "f32", False),
    (2000, 9, 2, 128, 80, "bf16", True), (900, 21, 3, 256, 240, "f32", True), (1500, 12, 4, 64, 48, "bf16", True)])
def test_rotation_of_more_than_half_the_head(n, hq, hk, D, rot, act, norm):
    """Half-split pairs that lie in two lanes and in both halves of the row; the append computes the same bits."""
    rng = np.random.default_rng(n + rot)
    x = heads_input(rng, n, hq, hk, D, act, hv=hk)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    cs, pos = rotation(rng, 50, rot), rng.integers(0, 50, n)
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    up = lambda a: torch.tensor(a, device=dev())  # noqa: E731
    qo, ko = torch.full_like(q, 7).contiguous(), torch.full_like(k, 7).contiguous()
    qg.qg_qk_norm_rope(q, k, qo, ko, ints(pos), up(cs), up(w), up(w), 1e-5, norm)
    page = 16
    pool = torch.zeros(AO.pool_bytes(-(-n // page), page, hk, D), dtype=torch.uint8, device=dev())
    qa, kb = torch.full_like(qo, 7), torch.full_like(ko, 7)
    qg.qg_cache_append(qg.qg_cache(pool, -(-n // page), page, hk, D), k, v, torch.arange(n, device=dev()), q=q, q_out=qa, positions=ints(pos),
                       cos_sin=up(cs), q_weight=up(w), k_weight=up(w), eps=1e-5, norm=norm, k_back=kb)
    for src, out in ((q, qo), (k, ko)):
        want = AO.norm_rope32(src.float().cpu().numpy(), w, 1e-5, pos, cs, norm=norm)
        assert torch.equal(out.cpu(), torch.tensor(want).to(x.dtype))
    assert torch.equal(qa, qo)
    few = slice(0, 40)
    want = AO.kv_values(*AO.kv_blocks(AO.norm_rope32(k[few].float().cpu().numpy(), w, 1e-5, pos[few], cs, norm=norm)))
    assert torch.equal(kb[few].cpu(), torch.tensor(want.astype(np.float32)).to(x.dtype))
    assert qg.qg_device_status() == 0


@pytest.mark.parametrize("D,heads,new,act", [(256, 4, 3, "f32"), (256, 2, 4, "f32"), (256, 16, 1, "bf16"), (128, 12, 1, "f32")])
def test_lists_of_requests_that_leave_room_for_fewer_rows(D, heads, new, act):
    """1024 requests' lengths in shared memory: a shallower ring, or a tile of fewer rows."""
    rng = np.random.default_rng(D + new)
    held, fresh = rng.integers(0, 6, 1024), rng.integers(0, new + 1, 1024)
    held[500], fresh[3] = 200, new
    c = Case(D, D, heads, 1, held.tolist(), fresh.tolist(), page=16, act=act)
    c.check(c.run())
