"""The whole-prompt calls refuse bad arguments before anything is launched (CPU; the fake device
addresses are never dereferenced)."""
from __future__ import annotations

import numpy as np
import pytest

import block_quantized_token_format_gb300 as qg

A = 1 << 20
OK, INVAL, ALIGN, UNSUP, WORK = 0, -1, -2, -3, -4


def test_gemm_workspace():
    w = qg.qgemm_workspace_bytes
    assert w("q8_0", "bf16", 100, 2560, 10) >= 10 * 2560 * 2 + 10 * 4
    assert w("q8_0", "f32", 100, 2560, 10) >= 2 * 10 * 2560 * 2
    assert w("bf16", "f32", 100, 2560, 10) >= 3 * 10 * 2560 * 2
    assert w("q4_0", "f32", 100, 64, (1 << 31) - 2000) > 1 << 38        # past 32 bits
    assert w("q8_0", "bf16", 100, 2560, 0) > 0 and w("q8_0", "bf16", 100, 2560, 10, 512) >= w("q8_0", "bf16", 100, 2560, 10)
    for bad in ((0, 2560, 10, 0), (100, 33, 10, 0), (100, 0, 10, 0), (100, 2560, -1, 0), (100, 2560, 10, -1), (100, 2560, 10, 65537),
                (100, 2560, 1 << 31, 0)):
        assert w("q8_0", "bf16", *bad) == 0
    assert w("q8_0", 2, 100, 2560, 10) == 0 and w(7, "f32", 100, 2560, 10) == 0
    assert qg._act("torch.bfloat16") == qg.QG_ACT_BF16 and qg._act("f32") == qg.QG_ACT_F32


def test_gemm_refusals():
    lib = qg.load_library()
    ok = dict(fmt=0, W=A, n_out=100, n_in=64, act=0, x=2 * A, xs=64, ntok=5, bias=None, f=0, res=None, rs=0, y=3 * A, ys=100, ws=4 * A, wb=1 << 30)

    def call(**kw):
        return lib.qgemm(*{**ok, **kw}.values(), None)
    for k in ("W", "x", "y"):
        assert call(**{k: None}) == INVAL, k
    assert call(ws=None) == WORK and call(wb=100) == WORK and call(ws=4 * A + 8) == ALIGN
    assert call(fmt=9) == INVAL and call(act=2) == INVAL and call(n_out=0) == INVAL and call(n_in=48) == INVAL and call(ntok=-1) == INVAL
    assert call(f=5) == INVAL and call(f=-1) == INVAL and call(f=4, n_out=101, ys=101) == INVAL
    assert call(xs=63) == INVAL and call(ys=99) == INVAL and call(res=5 * A, rs=99) == INVAL and call(f=4, ys=49) == INVAL
    assert call(xs=66) == ALIGN and call(x=2 * A + 8) == ALIGN and call(W=A + 8) == ALIGN and call(y=3 * A + 2) == ALIGN
    assert call(act=1, xs=68) == ALIGN and call(act=1, y=3 * A + 1) == ALIGN and call(bias=A + 2) == ALIGN and call(res=5 * A + 2, rs=100) == ALIGN
    assert call(y=2 * A) == INVAL                                    # the outputs over the tokens
    assert call(res=3 * A, rs=104) == INVAL                          # over a residual of another stride
    assert call(xs=1 << 40) == INVAL and call(ys=1 << 40) == INVAL
    assert call(ntok=0, W=None, x=None, y=None) == OK                # nothing to do


def test_experts_refusals():
    lib = qg.load_library()
    ok = dict(fmt=0, W=A, n_exp=8, n_out=100, n_in=64, act=0, x=2 * A, xs=64, n_x=5, off=5 * A, rows=None, slots=5, f=0, y=3 * A, ys=100, ws=4 * A,
              wb=1 << 30)

    def call(**kw):
        return lib.qgemm_experts(*{**ok, **kw}.values(), None)
    for k in ("W", "x", "y", "off"):
        assert call(**{k: None}) == INVAL, k
    assert call(n_exp=0) == INVAL and call(n_exp=70000) == INVAL and call(n_exp=60000, n_out=60000, ys=60000) == INVAL
    assert call(n_x=4) == INVAL and call(n_x=0, rows=6 * A) == INVAL and call(slots=-1) == INVAL
    assert call(off=5 * A + 2) == ALIGN and call(rows=6 * A + 2) == ALIGN
    assert call(wb=16) == WORK and call(slots=0, off=None) == OK


def test_attention_refusals():
    lib = qg.load_library()
    ok = dict(act=1, q=A, qs=6 * 128, k=2 * A, ks=2 * 128, v=3 * A, vs=2 * 128, n=10, hq=6, hk=2, D=128, cu=4 * A, n_seq=2, longest=7, window=0, scale=0.1,
              out=5 * A, os=6 * 128, lse=None, ws=6 * A, wb=1 << 30)

    def call(**kw):
        return lib.qg_prompt_attention(*{**ok, **kw}.values(), None)
    for k in ("q", "k", "v", "out", "cu"):
        assert call(**{k: None}) == INVAL, k
    for k in ("q", "k", "v", "out"):
        assert call(**{k: ok[k] + 8}) == ALIGN, k
    assert call(qs=6 * 128 + 2) == ALIGN and call(qs=100) == INVAL and call(ks=100) == INVAL and call(vs=2) == INVAL and call(os=5 * 128) == INVAL
    assert call(act=2) == INVAL and call(D=96) == INVAL and call(hq=7) == INVAL and call(hk=0) == INVAL and call(n=-1) == INVAL
    assert call(n_seq=-1) == INVAL and call(longest=0) == INVAL and call(window=-1) == INVAL and call(scale=float("nan")) == INVAL
    assert call(n_seq=16385) == UNSUP and call(hq=129, hk=1, qs=129 * 128, os=129 * 128) == UNSUP
    assert call(out=A) == INVAL and call(out=2 * A) == INVAL and call(cu=4 * A + 2) == ALIGN and call(lse=A + 2) == ALIGN
    assert call(ws=None) == WORK and call(wb=8) == WORK and call(act=0, wb=256) == WORK and call(ws=6 * A + 4) == ALIGN
    assert call(n=0, q=None, cu=None) == OK and call(n_seq=0, cu=None) == OK
    size = qg.qg_prompt_attention_workspace_bytes
    assert size("bf16", 10, 6, 2, 128) >= 16 and size("f32", 10, 6, 2, 128) >= 10 * (6 + 2 + 2) * 128 * 4
    for bad in ((10, 7, 2, 128), (10, 6, 0, 128), (10, 6, 2, 96), (-1, 6, 2, 128)):
        assert size("bf16", *bad) == 0


def test_binding_refuses_without_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(KeyError):
        qg.qgemm("q8_0", A, 100, 64, x, x, None, activation="relu")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        qg.qgemm("q8_0", A, 100, 64, x.half(), x, None)
    with pytest.raises(ValueError, match="x: a CUDA"):
        qg.qgemm("q8_0", A, 100, 64, x, x, None)
    with pytest.raises(ValueError, match="q: a CUDA"):
        qg.qg_prompt_attention(torch.zeros(4, 2, 64), None, None, None, None, None, 1.0, 4)
    with pytest.raises(TypeError):
        qg.qgemm_experts("q8_0", A, 8, 100, 64, np.zeros((4, 64), np.float32), None, None, None)


def test_tile_description_refuses():
    for bad in (("q8_0", "bf16", 0, 64, 1), ("q8_0", "bf16", 8, 33, 1), ("q8_0", "bf16", 8, 64, 0), ("q8_0", "bf16", 8, 64, 1, -1),
                ("q8_0", "bf16", 8, 64, 1, 70000), ("q8_0", 2, 8, 64, 1)):
        with pytest.raises(qg.QGError):
            qg.qg_describe_gemm_tile(*bad)
