"""GPU parity of the attention path: page tables, head norm and rotation, cache append,
attention over the 4-bit cache, each against the fp64 oracle.

Tolerances (derived from the arithmetic, before any run):
* pages: integers, equal.   Cache bytes and rotated heads in fp32: equal to the definition's
  fp32 operations (the order of every operation is part of the definition).
* heads against fp64: 12 roundings of 2^-24 on a value and its partner, the root's at half
  weight: 2^-20 of |y| + |partner|; bf16 adds 2^-8.
* attention: a score is a sum of |q| |d| |code| terms (code - 8 enters as code minus 8, 23
  at most) whose tensor products truncate at most 8 times (2^-23 each) and whose queries carry
  2^-21: |ds| <= 2^-19 * scale * sum |q| 23 |d|, plus 2^-20 for the exponent's argument.  A
  probability is off by that factor and 2^-20, an output by twice that of sum p |v|; and, since
  probabilities enter the product as fp16 terms on a grid of 2^-24 with the row's largest at 2^7
  or more, by 2^-32 of sum |v|.
  One-term probabilities (bf16) are off by 2^-11 each, the output's rounding adds 2^-8 |out|.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attention_oracle as AO

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


def dev():
    return torch.device("cuda:0")


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=dev())


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ------------------------------------------------------------------------------------ pages

def run_pages(held, fresh, free, table, page, n_tok, begin=None, in_place=False):
    n = len(held)
    t = torch.tensor(np.asarray(table).reshape(n, -1), dtype=torch.int32, device=dev())
    seq, cu = ints([-7] * n), ints([-7] * (n + 1))
    slots = torch.full((n_tok,), -7, dtype=torch.int64, device=dev())
    pos = torch.full((n_tok,), -7, dtype=torch.int32, device=dev())
    b = None if begin is None else ints([begin])
    end = b if in_place else ints([-7])
    qg.qg_cache_pages(ints(held), ints(fresh), ints(free), t, seq, cu, slots, pos, page, free_begin=b, free_end=end)
    return [host(x) for x in (t, seq, cu, slots, pos, end)]


@pytest.mark.parametrize("n_req,most_held,most_new,page", [(1, 0, 1, 16), (1, 40, 3, 16), (5, 100, 4, 48), (33, 1000, 4, 64),
                                                           (700, 300, 2, 32), (3, 0, 5000, 16), (64, 50, 700, 128),
                                                           (2000, 64, 3, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_match_oracle(n_req, most_held, most_new, page, in_place):
    rng = np.random.default_rng(n_req + page)
    held = rng.integers(0, most_held + 1, n_req)
    fresh = rng.integers(0, most_new + 1, n_req)
    if n_req > 2:
        held[1] = fresh[1] = 0                               # a request with nothing
        held[0] = page * 2                                   # new tokens begin a page
    n_tok = int(fresh.sum()) + 3                             # padding at the end
    width = int(((held + fresh + page - 1) // page).max()) + 1
    free = rng.permutation(int(((held + fresh + page - 1) // page).sum()) + 20)
    table = np.full((n_req, width), -1)
    at = 0
    for r in range(n_req):
        k = -(-int(held[r]) // page)
        table[r, :k] = 10000 + np.arange(at, at + k)
        at += k
    want = AO.cache_pages(held.tolist(), fresh.tolist(), free, 2, table, page, n_tok)
    got = run_pages(held, fresh, free, table, page, n_tok, begin=2, in_place=in_place)
    for w, g in zip(want, got):
        assert np.array_equal(np.asarray(w).reshape(-1), g.reshape(-1))
    assert qg.qg_device_status() == 0


def test_pages_errors_are_reported_and_harmless():
    t, seq, cu, slots, pos, end = run_pages([0, 0], [20, 20], [5, 6, 7], [[-1, -1]] * 2, 16, 40)
    assert qg.qg_device_status() == qg.QG_DEVICE_NO_PAGES
    assert t.tolist() == [[5, 6], [7, -1]] and slots[36:].tolist() == [-1] * 4 and slots[35] == 7 * 16 + 15 and end[0] == 3
    t, seq, cu, slots, pos, end = run_pages([0], [40], [5, 6, 7], [[-1, -1]], 16, 40)      # a row of two pages for three
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE and t.tolist() == [[5, 6]] and (slots[32:] == -1).all()
    t, seq, cu, slots, pos, end = run_pages([0, 0], [5, 5], [5, 6], [[-1]] * 2, 16, 7)      # more new tokens than slots
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH and cu.tolist() == [0, 5, 7]
    t, seq, cu, slots, pos, end = run_pages([-3, 1], [5, 1], [5, 6], [[-1], [4]], 16, 6)
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH and slots[0] == 4 * 16 + 1 and cu.tolist() == [0, 0, 1]
    run_pages([16], [1], [5], [[-1, -1]], 16, 1)             # a held page that the table lacks is not read
    assert qg.qg_device_status() == 0
    run_pages([3], [1], [5], [[-1]], 16, 1)                  # ... unless the new token falls on it
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE


def test_pages_no_requests():
    cu, slots, pos = ints([-7]), torch.full((4,), -7, dtype=torch.int64, device=dev()), ints([-7] * 4)
    lib = qg.load_library()
    assert lib.qg_cache_pages(None, None, 0, 16, None, 0, None, None, None, 0, None, cu.data_ptr(), slots.data_ptr(),
                              pos.data_ptr(), 4, None) == 0
    torch.cuda.synchronize()
    assert cu.item() == 0 and (slots == -1).all() and (pos == -1).all()


# ------------------------------------------------------------------------------------ heads

def heads_input(rng, n, hq, hk, D, act, hv=0):
    x = (rng.standard_normal((n, hq + hk + hv, D)) * rng.uniform(0.05, 20, (n, hq + hk + hv, 1))).astype(np.float32)
    return torch.tensor(x, device=dev()).to(DT[act])


def rotation(rng, n_pos, rot):
    a = rng.uniform(0, 6.28, (n_pos, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


HEAD_CASES = [  # n, hq, hk, D, rot, act, interleaved, unit, norm, weights
    (1, 1, 1, 64, 64, "f32", False, False, True, True), (3, 6, 2, 128, 64, "f32", True, True, True, True),
    (4, 48, 16, 128, 128, "f32", False, False, True, True), (5, 7, 3, 256, 256, "bf16", False, True, True, True),
    (2, 5, 1, 64, 16, "bf16", True, False, True, False), (2, 4, 4, 128, 0, "f32", False, False, True, True),
    (3, 4, 1, 256, 64, "f32", True, False, False, False), (6, 0, 3, 128, 128, "f32", False, False, True, True),
    (6, 3, 0, 128, 32, "bf16", False, False, True, True), (1700, 11, 5, 128, 128, "f32", False, False, True, True),
    (1300, 13, 3, 64, 32, "bf16", False, True, True, True), (900, 21, 3, 256, 128, "f32", True, False, True, True),
    (2100, 9, 2, 128, 64, "bf16", False, False, True, True), (800, 30, 2, 256, 256, "bf16", False, False, True, True)]


@pytest.mark.parametrize("n,hq,hk,D,rot,act,inter,unit,norm,weights", HEAD_CASES)
def test_norm_rope_matches_oracle(n, hq, hk, D, rot, act, inter, unit, norm, weights):
    rng = np.random.default_rng(n + D)
    x = heads_input(rng, n, hq, hk, D, act, hv=1)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    qw, kw = [(rng.standard_normal(D) * 0.3 + (0 if unit else 1)).astype(np.float32) if weights else None for _ in range(2)]
    cs = rotation(rng, 50, rot) if rot else None
    pos = rng.integers(0, 50, n)
    qo, ko = torch.full_like(q, 7).contiguous(), torch.full_like(k, 7).contiguous()
    up = lambda w: None if w is None else torch.tensor(w, device=dev())  # noqa: E731
    qg.qg_qk_norm_rope(q, k, qo, ko, ints(pos) if rot else None, up(cs), up(qw), up(kw), 1e-5, norm, unit, inter)
    for src, out, w in ((q, qo, qw), (k, ko, kw)):
        xh = src.float().cpu().numpy()
        want32 = AO.norm_rope32(xh, w, 1e-5, pos, cs, unit, inter, norm)
        if act == "f32":
            assert np.array_equal(out.cpu().numpy(), want32)
        else:
            assert torch.equal(out.cpu(), torch.tensor(want32).bfloat16())
        want = AO.norm_rope(xh, w, 1e-5, pos, cs, unit, inter, norm)
        flat = AO.norm_rope(xh, w, 1e-5, None, None, unit, inter, norm)
        size = np.abs(want) + np.abs(flat).max(-1, keepdims=True)
        assert np.all(np.abs(host(out) - want) <= (2.0 ** -20 if act == "f32" else 2.0 ** -8 + 2.0 ** -20) * size)
    assert qg.qg_device_status() == 0


def test_norm_rope_in_place_and_padding():
    rng = np.random.default_rng(1)
    x = heads_input(rng, 6, 4, 2, 128, "f32")
    q, k = x[:, :4], x[:, 4:]
    cs = rotation(rng, 10, 128)
    pos = np.array([3, -1, 9, 10, 0, -5])
    q0, k0 = q.cpu().numpy().copy(), k.cpu().numpy().copy()
    qg.qg_qk_norm_rope(q, k, q, k, ints(pos), torch.tensor(cs, device=dev()))
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH          # position 10 of 10
    good = [0, 2, 4]
    for got, src in ((q, q0), (k, k0)):
        want = AO.norm_rope32(src[good], None, 1e-6, pos[good], cs)
        assert np.array_equal(got.cpu().numpy()[good], want)
        assert (got.cpu().numpy()[[1, 3, 5]] == 0).all()


def test_norm_rope_extreme_rows():
    """Zero rows, huge and tiny rows, a NaN and an infinity: as the definition's operations give."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 1, 128)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e25
    x[2] *= 1e-30
    x[3, 0, 5] = np.nan
    x[4, 0, 6] = np.inf
    t = torch.tensor(x, device=dev())
    out, k = torch.empty_like(t), torch.empty_like(t)
    qg.qg_qk_norm_rope(t, t, out, k)
    with np.errstate(all="ignore"):
        want = AO.norm_rope32(x, None, 1e-6, None, None)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


# ------------------------------------------------------------------------------------ append

APPEND_CASES = [  # n, hq, hk, D, page, rot, act, inter
    (1, 3, 1, 128, 16, 128, "f32", False), (4, 48, 16, 128, 64, 128, "f32", False), (19, 4, 2, 64, 48, 32, "bf16", True),
    (33, 2, 3, 256, 32, 256, "f32", False), (7, 0, 2, 128, 16, 0, "f32", False), (500, 24, 8, 128, 32, 64, "f32", True),
    (600, 20, 5, 256, 16, 64, "bf16", False), (700, 30, 3, 64, 128, 64, "f32", False), (1000, 16, 3, 128, 64, 128, "bf16", False)]


@pytest.mark.parametrize("n,hq,hk,D,page,rot,act,inter", APPEND_CASES)
def test_append_matches_oracle(n, hq, hk, D, page, rot, act, inter):
    rng = np.random.default_rng(n * 3 + D)
    x = heads_input(rng, n, hq, hk, D, act, hv=hk)
    if n >= 4:                                               # blocks of zeros, ties, values that spoil a block
        x[0, -1] = 0
        x[1, -1, :32] = 0.5
        x[1, -1, 3], x[1, -1, 9] = 2.0, -2.0
        x[2, -1, 40] = float("nan")
        x[3, -1, 41] = float("inf")
        x[3, -1, 1] = 1e6
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    w = rng.standard_normal(D).astype(np.float32)
    cs = rotation(rng, n + 4, rot) if rot else None
    pos = np.arange(n) + 3
    n_pages = -(-n // page) + 2
    slots = rng.permutation(n_pages * page)[:n].astype(np.int64)
    if n > 6:
        slots[6] = -1                                        # padding: nothing stored
    start = rng.integers(0, 256, AO.pool_bytes(n_pages, page, hk, D)).astype(np.uint8)
    pool = torch.tensor(start, device=dev())
    cache = qg.qg_cache(pool, n_pages, page, hk, D)
    qo = torch.zeros(n, hq, D, dtype=x.dtype, device=dev())
    kb, vb = [torch.zeros(n, hk, D, dtype=x.dtype, device=dev()) for _ in range(2)]
    up = lambda a: None if a is None else torch.tensor(a, device=dev())  # noqa: E731
    qg.qg_cache_append(cache, k, v, up(slots), q=q if hq else None, q_out=qo if hq else None, positions=ints(pos), cos_sin=up(cs),
                       q_weight=up(w), k_weight=up(w), interleaved=inter, k_back=kb, v_back=vb)
    assert qg.qg_device_status() == 0
    kf = AO.norm_rope32(k.float().cpu().numpy(), w, 1e-6, pos, cs, False, inter)
    vf = v.float().cpu().numpy()
    if hq:
        qf = AO.norm_rope32(q.float().cpu().numpy(), w, 1e-6, pos, cs, False, inter)
        assert torch.equal(qo.cpu(), torch.tensor(qf).to(x.dtype))
    for back, f in ((kb, kf), (vb, vf)):
        want = torch.tensor(AO.kv_values(*AO.kv_blocks(f)).astype(np.float32)).to(x.dtype).float().numpy()
        assert np.array_equal(back.float().cpu().numpy(), want, equal_nan=True)
    want = start.copy()
    few = range(n) if n <= 40 else rng.permutation(n)[:25]
    for i in few:
        if slots[i] >= 0:
            for h in range(hk):
                AO.kv_store(want, slots[i], h, page, hk, D, kf[i, h], vf[i, h])
    got = pool.cpu().numpy()
    if n <= 40:
        assert np.array_equal(got, want)                     # nothing but the tokens' own nibbles and scales changed
    else:
        keys = [s for s in slots[list(few)] if s >= 0]
        for h in range(hk):
            for a, b in zip(AO.kv_load(got, keys, h, page, hk, D), AO.kv_load(want, keys, h, page, hk, D)):
                assert np.array_equal(a, b, equal_nan=True)


def test_append_bad_slots_are_reported_and_not_stored():
    rng = np.random.default_rng(9)
    x = heads_input(rng, 4, 0, 2, 128, "f32", hv=2)
    pool = torch.zeros(AO.pool_bytes(2, 16, 2, 128), dtype=torch.uint8, device=dev())
    cache = qg.qg_cache(pool, 2, 16, 2, 128)
    slots = torch.tensor([32, -2, 1 << 40, -1], device=dev())
    qg.qg_cache_append(cache, x[:, :2], x[:, 2:], slots, norm=False)
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE
    assert int(pool.max()) == 0


# ------------------------------------------------------------------------------------ attention

class Case:
    """A filled cache with its requests, and the oracle's answer."""

    def __init__(self, seed, D, heads, kv, held, fresh, page=16, act="f32", window=0, tree=False, scale=None, garbage=True,
                 q_scale=1.0, extra_pages=2, v_scale=None):
        rng = self.rng = np.random.default_rng(seed)
        self.D, self.heads, self.kv, self.page, self.act, self.window = D, heads, kv, page, act, window
        self.scale = D ** -0.5 if scale is None else scale
        self.held, self.fresh = list(held), list(fresh)
        n = len(held)
        counts = [-(-(h + f) // page) for h, f in zip(held, fresh)]
        self.n_pages = sum(counts) + extra_pages
        start = rng.integers(0, 256, AO.pool_bytes(self.n_pages, page, kv, D)).astype(np.uint8)
        if garbage:                                          # whatever is not written reads as NaN
            start[:] = 0xFF
        self.pool = torch.tensor(start, device=dev())
        ids = rng.permutation(self.n_pages)
        self.table = np.full((n, max(max(counts, default=0), 1) + 1), -1)
        at = 0
        for r, c in enumerate(counts):
            self.table[r, :c] = ids[at:at + c]
            at += c
        self.seq = [h + f for h, f in zip(held, fresh)]
        self.cu = np.concatenate([[0], np.cumsum(fresh)])
        self.n_tok = int(self.cu[-1])
        self.slots = [np.array([self.table[r, i // page] * page + i % page for i in range(s)], dtype=np.int64)
                      for r, s in enumerate(self.seq)]
        total = sum(self.seq)
        vs = np.exp(rng.uniform(-3, 3, (total, kv, D // 32, 1))) if v_scale is None else v_scale
        self.k = rng.standard_normal((total, kv, D)).astype(np.float32)
        self.v = (rng.standard_normal((total, kv, D // 32, 32)) * vs).reshape(total, kv, D).astype(np.float32)
        self.q = torch.tensor((rng.standard_normal((self.n_tok, heads, D)) * q_scale).astype(np.float32), device=dev()).to(DT[act])
        self.bits = None
        if tree:
            j = np.concatenate([np.arange(f) for f in fresh]) if self.n_tok else np.zeros(0, int)
            self.bits = (rng.integers(0, 1 << 20, self.n_tok) & ((1 << j) - 1)) | (1 << j)
        self.append()

    def append(self):
        if sum(self.seq):
            cache = qg.qg_cache(self.pool, self.n_pages, self.page, self.kv, self.D)
            qg.qg_cache_append(cache, torch.tensor(self.k, device=dev()), torch.tensor(self.v, device=dev()),
                               torch.tensor(np.concatenate(self.slots), device=dev()), norm=False)

    def run(self, max_new=None, q=None, out=None, ws=None, lse=True, table=None, seq=None, stream=None):
        cache = qg.qg_cache(self.pool, self.n_pages, self.page, self.kv, self.D)
        out = torch.full_like(self.q, 7) if out is None else out
        self.lse = torch.full((max(self.n_tok, 1), self.heads), 7.0, device=dev())
        self.ws = ws if ws is not None else torch.zeros(qg.qg_attention_workspace_bytes(self.heads, self.kv, self.D),
                                                        dtype=torch.uint8, device=dev())
        qg.qg_attention(cache, self.q if q is None else q, ints(self.table.ravel()).view(self.table.shape) if table is None else table,
                        ints(self.seq) if seq is None else seq, ints(self.cu), out, self.ws, self.scale,
                        max_new=max(self.fresh, default=1) or 1 if max_new is None else max_new, window=self.window,
                        span_mask=None if self.bits is None else ints(self.bits), lse=self.lse if lse else None, stream=stream)
        return out

    def expect(self):
        """(out, tolerance, lse, its tolerance) of every row, fp64."""
        pool = self.pool.cpu().numpy()
        q = host(self.q)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        lse, ltol = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
        G = self.heads // self.kv
        for r, (s, f) in enumerate(zip(self.seq, self.fresh)):
            if f == 0:
                continue
            for h in range(self.kv):
                K, V = AO.kv_load(pool, self.slots[r], h, self.page, self.kv, self.D)
                d = np.abs(K).reshape(s, -1, 32).max(-1).repeat(32, -1) / 7.0          # at least |d|
                for j in range(f):
                    tok = int(self.cu[r]) + j
                    see = AO.visible(s, s, f, j, self.window, None if self.bits is None else self.bits[tok])
                    for g in range(G):
                        row = q[tok, h * G + g]
                        o, l, p = AO.attention(row, K, V, see, self.scale)
                        out[tok, h * G + g], lse[tok, h * G + g] = o, l
                        if see.any():
                            with np.errstate(invalid="ignore"):
                                ds = 2.0 ** -19 * abs(self.scale) * 23 * (d[see] @ np.abs(row)) + 2.0 ** -20
                                e = 2 * ds.max() + 2.0 ** -19 + (2.0 ** -10 if self.act == "bf16" else 0)
                                tol[tok, h * G + g] = e * (p @ np.abs(V[see])) + 2.0 ** -32 * np.abs(V[see]).sum(0) + (2.0 ** -8 * np.abs(o) if self.act == "bf16" else 0)
                                ltol[tok, h * G + g] = ds.max() + 2.0 ** -20 * max(1.0, abs(l))
        return out, tol, lse, ltol

    def check(self, got):
        want, tol, lse, ltol = self.expect()
        g = host(got)
        assert np.array_equal(np.isnan(g), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.all(np.abs(g - want)[ok] <= tol[ok]), float(np.max((np.abs(g - want) / np.maximum(tol, 1e-300))[ok]))
        gl = host(self.lse)[:self.n_tok]
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty)
        ok = ~empty & ~np.isnan(lse)
        assert np.all(np.abs(gl[ok] - lse[ok]) <= ltol[ok])
        assert int(self.ws[:qg.QG_ATTENTION_ZERO_BYTES].max()) == 0          # left as found
        assert qg.qg_device_status() == 0


LENGTHS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,new", [(1, 1, 1), (6, 2, 1), (8, 1, 1), (6, 2, 4), (16, 1, 1), (5, 1, 5), (24, 2, 2)])
def test_attention_lengths(D, act, heads, kv, new):
    """Every length around a record, a unit and a page, with 1 to 25 rows per key/value head."""
    fresh = [min(new, 1 + i % new) for i in range(len(LENGTHS))]
    c = Case(D + heads, D, heads, kv, LENGTHS, fresh, page=48, act=act)
    c.check(c.run())


@pytest.mark.parametrize("D,heads,kv,page,new,window,tree,act", [
    (128, 4, 2, 16, 4, 0, True, "f32"), (128, 4, 2, 32, 3, 20, False, "f32"), (64, 9, 3, 64, 4, 1, True, "f32"),
    (256, 6, 1, 16, 4, 37, True, "f32"), (256, 6, 1, 128, 2, 64, False, "bf16"), (128, 8, 8, 16, 4, 100, True, "bf16"),
    (128, 3, 1, 16, 20, 0, True, "f32"), (64, 2, 1, 48, 40, 33, False, "f32"), (128, 16, 2, 16, 9, 5, True, "f32")])
def test_attention_masks(D, heads, kv, page, new, window, tree, act):
    """Windows that cut inside and at the edges of units, trees that hide some or all new keys."""
    c = Case(new + page, D, heads, kv, [0, 5, 33, 200], [new, 1, new, max(1, new - 1)], page=page, act=act, window=window, tree=tree)
    if tree:
        c.bits[0] = 0                                        # a row that sees nothing: held 0, no bit
        c.bits[-1] = 0                                       # a row that sees the old keys only
    c.check(c.run())


@pytest.mark.parametrize("page", [16, 32, 48])
def test_attention_window_does_not_need_older_pages(page):
    """Pages wholly before the window may have been given away: their entries are not used."""
    c = Case(41, 128, 6, 2, [200, 77, 1000], [3, 1, 2], page=page, window=40)
    want = c.run()
    c.check(want)
    table = c.table.copy()
    for r, (s, f) in enumerate(zip(c.seq, c.fresh)):
        table[r, :max(0, s - f + 1 - c.window) // page] = -1
    assert (table != c.table).sum() > 8
    assert torch.equal(c.run(table=ints(table.ravel()).view(table.shape)), want) and qg.qg_device_status() == 0


def test_attention_split_over_the_gpu():
    """Long caches: parts joined across warps and CTAs; one request, several, uneven ones."""
    for seed, (held, fresh, heads, kv) in enumerate([([6000], [1], 4, 1), ([3000], [4], 6, 2), ([9000, 0, 40], [1, 2, 3], 8, 2),
                                                     ([700] * 5, [3] * 5, 16, 2)]):
        c = Case(100 + seed, 128, heads, kv, held, fresh, page=64)
        got = c.run()
        c.check(got)
        assert torch.equal(got, c.run(ws=c.ws)) and torch.equal(got, c.run(ws=c.ws))         # the same on every run


def test_attention_typical_error():
    """Gaussian queries, keys and values: the error in norm stays below 2^-19 (fp32's own for
    scores of this size: 2^-20 an exponential, as much again for its argument)."""
    c = Case(5, 128, 8, 2, [5000, 777], [1, 4], page=64, v_scale=1.0)
    got = host(c.run())
    want = c.expect()[0]
    assert np.linalg.norm(got - want) <= 2.0 ** -19 * np.linalg.norm(want)


def test_attention_many_requests():
    """More requests than a warp, than a CTA's threads; some without new tokens."""
    rng = np.random.default_rng(3)
    for n in (31, 33, 600, 1024):
        held, fresh = rng.integers(0, 70, n), rng.integers(0, 3, n)
        if n == 600:
            held, fresh = held % 20, fresh * (rng.random(n) < 0.1).astype(int)
        held = held if n < 1000 else held % 9
        c = Case(n, 64, 2, 1, held.tolist(), fresh.tolist(), page=16)
        c.check(c.run())


def test_attention_scores_of_every_size():
    for q_scale, scale in ((40.0, None), (1e-25, 1e24), (1e20, 1e-21), (1.0, -0.2), (1.0, 0.0), (1e-30, 1.0)):
        c = Case(7, 128, 6, 2, [90, 3], [2, 1], q_scale=q_scale, scale=scale)
        c.check(c.run())


def test_attention_values_of_every_size():
    for vs in (1e-6, 3000.0, 1e-3):
        c = Case(8, 128, 4, 2, [90, 3], [2, 1], v_scale=vs)
        c.check(c.run())


def test_attention_nan_stays_where_it_is_seen():
    """A NaN or infinite key or value spoils the rows (for a value: the block of 32) that see it
    and no others; a NaN query spoils its own row."""
    for D in (64, 128, 256):
        c = Case(11, D, 4, 2, [60, 40], [4, 4], page=16, window=30, tree=True)
        c.bits[:] = [1, 2, 4, 8] * 2                         # every new token sees itself only
        c.v[61, 1, 3] = np.nan                               # request 0's token 61: its row alone, block 0 of head 1
        c.k[64 + 42, 0, 5] = np.inf                          # request 1's token 42: its row alone, head 0
        c.v[20, 0, D - 1] = np.nan                           # outside the window of every row
        c.append()
        c.q[2, 3, 7] = float("nan")
        got = c.run()
        c.check(got)
        bad = torch.isnan(got)
        assert bad[1, 2:, :32].all() and not bad[1, :2].any() and not bad[1, 2:, 32:].any() and not bad[0].any()
        assert bad[2, 3].all() and not bad[2, :3].any()
        assert bad[6, :2].all() and not bad[6, 2:].any() and not bad[[4, 5, 7]].any()


def test_attention_strides_streams_and_early_start():
    c = Case(13, 128, 6, 2, [300, 17, 0], [2, 1, 4], page=32)
    want = c.run()
    wide = torch.zeros(c.n_tok, 10, 128, device=dev())
    wide[:, 2:8] = c.q
    out = torch.zeros(c.n_tok, 9, 128, device=dev())
    c.run(q=wide[:, 2:8], out=out[:, 1:7])
    assert torch.equal(out[:, 1:7], want) and float(out[:, 0].abs().max()) == 0 and float(out[:, 7:].abs().max()) == 0
    side = torch.cuda.Stream()
    ws = c.ws.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                            # torch's current stream is taken
        a = c.run(ws=ws)
    side.synchronize()
    b = c.run(ws=ws, stream=side.cuda_stream)
    side.synchronize()
    qg.qg_set_launch_options(qg.QG_LAUNCH_EARLY_START)
    d = [c.run(ws=c.ws) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want) and all(torch.equal(x, want) for x in d)


def test_attention_row_tiles_agree():
    """max_new only chooses the kernel: every tile gives the same rows within the tolerance."""
    c = Case(17, 128, 3, 1, [100, 2], [6, 1], page=16)
    for max_new in (1, 2, 3, 4, 5, 6, 100):
        c.check(c.run(max_new=max_new))


def test_attention_past_32_bits():
    """Pages beyond 4 GB of cache, for the append and for the attention."""
    free, _ = torch.cuda.mem_get_info()
    page, kv, D = 16, 1, 128
    n_pages = (5 << 30) // AO.pool_bytes(1, page, kv, D)
    if free < 7 << 30:
        pytest.skip("needs 7 GB")
    c = Case(19, D, 2, kv, [100], [2], page=page)
    small = c.pool.cpu().numpy()
    pool = torch.empty(AO.pool_bytes(n_pages, page, kv, D), dtype=torch.uint8, device=dev())
    cache = qg.qg_cache(pool, n_pages, page, kv, D)
    up = n_pages - c.n_pages
    slots = torch.tensor(np.concatenate(c.slots) + up * page, device=dev())
    qg.qg_cache_append(cache, torch.tensor(c.k, device=dev()), torch.tensor(c.v, device=dev()), slots, norm=False)
    assert int(slots.min()) * 18 * D // 16 > 1 << 32
    out = torch.zeros_like(c.q)
    ws = torch.zeros(qg.qg_attention_workspace_bytes(2, kv, D), dtype=torch.uint8, device=dev())
    table = ints(np.where(c.table >= 0, c.table + up, -1).ravel()).view(c.table.shape)
    qg.qg_attention(cache, c.q, table, ints(c.seq), ints(c.cu), out, ws, c.scale, max_new=2)
    assert torch.equal(out, c.run()) and small.size < pool.numel()
    c.check(c.run())


def test_attention_bad_inputs_are_reported_and_harmless():
    c = Case(23, 128, 4, 2, [40, 40], [1, 1], page=16)
    want = c.run()
    bad = c.table.copy()
    bad[0, 1] = c.n_pages                                    # a page outside the cache
    got = c.run(table=ints(bad.ravel()).view(bad.shape))
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE and torch.equal(got[1], want[1])
    bad[0, 1] = -5
    c.run(table=ints(bad.ravel()).view(bad.shape))
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE
    got = c.run(seq=ints([10 ** 9, 41]))                     # more tokens than the table's row holds: left out
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_PAGE and (got[0] == 7).all() and torch.equal(got[1], want[1])
    got = c.run(seq=ints([-4, 41]))
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH and (got[0] == 7).all() and torch.equal(got[1], want[1])
    keep, c.cu = c.cu, np.array([0, 1, 9])                   # more new tokens than rows
    got = c.run()
    assert qg.qg_device_status() == qg.QG_DEVICE_BAD_LENGTH and torch.equal(got[0], want[0]) and (got[1] == 7).all()
    c.cu = keep
    assert torch.equal(c.run(), want)


def test_attention_bounded_wait():
    """A wait that cannot end gives up, reports and returns; after the workspace is zeroed again
    the next call is right."""
    c = Case(29, 128, 4, 2, [500], [1], page=16)
    want = c.run()
    qg.qg_set_wait_limit(2000, 16)
    c.run()
    torch.cuda.synchronize()
    assert qg.qg_device_status() & qg.QG_DEVICE_WAIT_TIMEOUT
    qg.qg_set_wait_limit(0, 0)
    assert torch.equal(c.run(), want)
    assert qg.qg_device_status() == 0


# ------------------------------------------------------------------------------------ together

def test_steps_of_a_sequence():
    """Prompt, then decode and verify steps, page by page: every step's outputs against the
    oracle on the cache as it stands, in one captured graph's worth of calls."""
    rng = np.random.default_rng(31)
    D, heads, kv, page, n_req = 128, 6, 2, 16, 3
    n_pages = 40
    pool = torch.full((AO.pool_bytes(n_pages, page, kv, D),), 0xFF, dtype=torch.uint8, device=dev())
    cache = qg.qg_cache(pool, n_pages, page, kv, D)
    table = torch.full((n_req, 8), -1, dtype=torch.int32, device=dev())
    free, begin = ints(rng.permutation(n_pages)), ints([0])
    held, cs = ints([0] * n_req), torch.tensor(rotation(rng, 200, D), device=dev())
    ws = torch.zeros(qg.qg_attention_workspace_bytes(heads, kv, D), dtype=torch.uint8, device=dev())
    total = np.zeros(n_req, int)
    for fresh in ([7, 30, 1], [1, 1, 1], [4, 2, 3], [1, 0, 4], [3, 1, 20]):
        n = sum(fresh)
        qkv = torch.tensor(rng.standard_normal((n, heads + 2 * kv, D)).astype(np.float32), device=dev())
        seq, cu, slots, pos = ints([0] * n_req), ints([0] * (n_req + 1)), torch.zeros(n, dtype=torch.int64, device=dev()), ints([0] * n)
        qg.qg_cache_pages(held, ints(fresh), free, table, seq, cu, slots, pos, page, free_begin=begin, free_end=begin)
        q = torch.empty(n, heads, D, device=dev())
        qg.qg_cache_append(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], slots, q=qkv[:, :heads], q_out=q, positions=pos, cos_sin=cs)
        out = torch.empty_like(q)
        qg.qg_attention(cache, q, table, seq, cu, out, ws, D ** -0.5, max_new=max(fresh))
        total += fresh
        assert host(seq).tolist() == total.tolist()
        t, hpool = host(table), pool.cpu().numpy()
        for r in range(n_req):
            sl = [int(t[r, i // page]) * page + i % page for i in range(total[r])]
            for h in range(kv):
                K, V = AO.kv_load(hpool, sl, h, page, kv, D)
                assert np.all(np.isfinite(K))
                for j in range(fresh[r]):
                    tok = sum(fresh[:r]) + j
                    see = AO.visible(total[r], total[r], fresh[r], j)
                    for g in range(heads // kv):
                        o, _, p = AO.attention(host(q)[tok, h * 3 + g], K, V, see, D ** -0.5)
                        assert np.allclose(host(out)[tok, h * 3 + g], o, atol=1e-4)
        held = seq
    assert int(begin) == sum(-(-int(x) // page) for x in total)
    assert qg.qg_device_status() == 0
