"""The attention path's calls refuse bad arguments before anything is launched (CPU; the fake
device addresses are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest

import block_quantized_token_format_gb300 as qg

A = 1 << 20
OK, INVAL, ALIGN, UNSUP, WORK = 0, -1, -2, -3, -4


def cache(data=A, n_pages=10, page=16, heads=2, dim=128):
    qg.load_library()
    return qg.qg_cache(data, n_pages, page, heads, dim)


def test_sizes():
    assert qg.qg_cache_bytes(10, 16, 2, 128) == 10 * 16 * 2 * 144
    assert qg.qg_cache_bytes(1 << 24, 64, 16, 256) == (1 << 24) * 64 * 16 * 288      # past 32 bits
    for bad in ((0, 16, 2, 128), (10, 8, 2, 128), (10, 24, 2, 128), (10, 16, 0, 128), (10, 16, 2, 96), (-1, 16, 2, 128)):
        assert qg.qg_cache_bytes(*bad) == 0
    assert qg.qg_attention_workspace_bytes(48, 16, 128) > qg.QG_ATTENTION_ZERO_BYTES
    for bad in ((0, 1, 128), (3, 2, 128), (4, 2, 100), (4, 0, 64)):
        assert qg.qg_attention_workspace_bytes(*bad) == 0
    assert qg.QG_CACHE_MAX == 65280.0


def test_pages_refusals():
    lib = qg.load_library()
    ok = dict(held=A, fresh=A, n_req=3, page=16, free=A, n_free=5, begin=None, end=None, table=A, width=4, seq=2 * A,
              cu=3 * A, slots=A, pos=A, n_tok=7)

    def call(**kw):
        return lib.qg_cache_pages(*{**ok, **kw}.values(), None)
    for k in ("held", "fresh", "free", "table", "seq", "cu", "slots", "pos"):
        assert call(**{k: None}) == INVAL, k
        assert call(**{k: A + 2}) == ALIGN, k
    assert call(slots=A + 4) == ALIGN
    assert call(n_req=-1) == INVAL and call(n_req=16385) == UNSUP
    assert call(page=8) == INVAL and call(page=24) == INVAL
    assert call(n_free=-1) == INVAL and call(n_tok=-1) == INVAL and call(width=-1) == INVAL
    assert call(seq=A) == INVAL and call(cu=A) == INVAL          # outputs over the lengths


def heads_ok():
    return dict(act=0, q=A, qs=6 * 128, k=A, ks=2 * 128, n=4, hq=6, hk=2, D=128, qw=None, kw=None, eps=1e-6, flags=0, cs=A,
                npos=100, rot=128, pos=A, qo=A, qos=6 * 128, ko=A, kos=2 * 128)


def test_norm_rope_refusals():
    lib = qg.load_library()

    def call(**kw):
        return lib.qg_qk_norm_rope(*{**heads_ok(), **kw}.values(), None)
    for k in ("q", "k", "qo", "ko", "pos"):
        assert call(**{k: None}) == INVAL, k
    for k in ("q", "k", "qo", "ko"):
        assert call(**{k: A + 8}) == ALIGN, k
    assert call(qs=6 * 128 + 2) == ALIGN and call(qs=100) == INVAL and call(kos=2) == INVAL
    assert call(act=2) == INVAL and call(D=96) == INVAL and call(flags=8) == INVAL
    assert call(n=-1) == INVAL and call(hq=-1) == INVAL and call(hk=70000) == INVAL
    assert call(eps=-1.0) == INVAL and call(eps=float("nan")) == INVAL
    for rot in (0, 8, 24, 144):
        assert call(rot=rot) == INVAL, rot
    assert call(npos=0) == INVAL and call(cs=None) == INVAL      # rot without a table
    assert call(n=0, q=None, k=None, qo=None, ko=None) in (OK, -5)        # nothing to do (no device here)


def test_append_refusals():
    lib = qg.load_library()
    c = cache()
    ok = dict(c=c.address, act=0, q=A, qs=6 * 128, k=A, ks=256, v=A, vs=256, n=4, hq=6, qw=None, kw=None, eps=1e-6, flags=0,
              cs=A, npos=100, rot=128, pos=A, slots=A, qo=A, qos=6 * 128, kb=None, vb=None)

    def call(**kw):
        return lib.qg_cache_append(*{**ok, **kw}.values(), None)
    for k in ("c", "q", "k", "v", "slots", "qo", "pos"):
        assert call(**{k: None}) == INVAL, k
    for k in ("q", "k", "v", "qo", "kb", "vb"):
        assert call(**{k: A + 8}) == ALIGN, k
    assert call(slots=A + 4) == ALIGN and call(vs=255) == INVAL
    for bad in (dict(data=None), dict(n_pages=0), dict(page=8), dict(page=17), dict(heads=0), dict(dim=80)):
        assert call(c=(k := cache(**bad)).address) == INVAL, (bad, k)
    assert call(c=(k := cache(data=A + 8)).address) == ALIGN, k


def test_attention_refusals():
    lib = qg.load_library()
    c = cache()
    ws = qg.qg_attention_workspace_bytes(6, 2, 128)
    ok = dict(c=c.address, act=0, q=A, qs=768, n=4, hq=6, table=A, width=3, seq=A, cu=A, n_req=2, max_new=2, window=0,
              mask=None, scale=0.1, out=A, os=768, lse=None, ws=A, wsb=ws)

    def call(**kw):
        return lib.qg_attention(*{**ok, **kw}.values(), None)
    for k in ("c", "q", "table", "seq", "cu", "out"):
        assert call(**{k: None}) == INVAL, k
    for k in ("q", "out", "ws"):
        assert call(**{k: A + 8}) == ALIGN, k
    for k in ("table", "seq", "cu", "mask", "lse"):
        assert call(**{k: A + 2}) == ALIGN, k
    assert call(ws=None) == WORK and call(wsb=ws - 1) == WORK
    assert call(hq=5) == INVAL and call(hq=0) == INVAL and call(act=7) == INVAL
    assert call(qs=700) == INVAL and call(os=767) == INVAL and call(qs=770) == ALIGN
    assert call(max_new=0) == INVAL and call(window=-1) == INVAL and call(n=-1) == INVAL and call(n_req=-1) == INVAL
    assert call(scale=float("inf")) == INVAL and call(scale=float("nan")) == INVAL
    assert call(n_req=1025) == UNSUP
    assert call(n_req=0, q=None, table=None) == OK and call(n=0, q=None) == OK       # nothing to do
    big = cache(n_pages=(1 << 31) - 1, page=65536, heads=64)
    assert call(c=big.address, hq=64, qs=64 * 128, os=64 * 128, wsb=1 << 40) in (UNSUP, -5)


def test_binding_refuses_tensors_it_cannot_take():
    torch = pytest.importorskip("torch")
    qg.load_library()
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        qg.qg_qk_norm_rope(x, x, x, x)
    with pytest.raises(TypeError):
        qg.qg_qk_norm_rope(x.double(), x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        qg.qg_cache(torch.zeros(1 << 20, dtype=torch.uint8), 10, 16, 2, 128)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        qg.qg_cache_pages(i, i, i, torch.zeros(3, 2, dtype=torch.int32), i, i, torch.zeros(3, dtype=torch.int64), i, 16)


def test_cache_struct_matches_the_header():
    assert ctypes.sizeof(qg.qg_cache) == 32 and qg.qg_cache.head_dim.offset == 24
