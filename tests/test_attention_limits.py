"""Refusals of the attention path's calls at the ends of their ranges (CPU; every call here is
refused on the host, the fake device addresses are never dereferenced)."""
from __future__ import annotations

from test_attention_abi import A, INVAL, cache, heads_ok

import block_quantized_token_format_gb300 as qg


def test_in_place_at_another_stride_is_refused():
    """Rows written over rows that other warps have yet to read."""
    lib = qg.load_library()

    def rope(**kw):
        return lib.qg_qk_norm_rope(*{**heads_ok(), **kw}.values(), None)
    B = A + (1 << 16)
    assert rope(ko=B, qos=800) == INVAL and rope(qo=B, kos=512) == INVAL and rope(n=2, ko=B, qs=1024) == INVAL

    c = cache()
    ok = dict(c=c.address, act=0, q=A, qs=6 * 128, k=2 * A, ks=512, v=3 * A, vs=512, n=4, hq=6, qw=None, kw=None, eps=1e-6, flags=0,
              cs=A, npos=100, rot=128, pos=A, slots=A, qo=A, qos=6 * 128, kb=None, vb=None)

    def append(**kw):
        return lib.qg_cache_append(*{**ok, **kw}.values(), None)
    assert append(qos=800) == INVAL and append(qs=1024) == INVAL
    assert append(kb=2 * A) == INVAL and append(vb=3 * A) == INVAL and append(kb=2 * A, n=2) == INVAL
