"""Plain fp64 implementation of the whole-prompt calls: products with an epilogue, products
grouped by expert, causal attention of packed prompts.  Test infrastructure, written from the
formulas in ``include/qgemv.h``; no sizes, tiles or orders of the kernels appear here.
"""
from __future__ import annotations

import math

import numpy as np

from .qgemv_oracle import dequantize, fmt_id, row_slice

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(v, f):
    """The epilogue's function of fp64 values; "swiglu" pairs neighbouring columns."""
    v = np.asarray(v, np.float64)
    if f == "silu":
        return v / (1.0 + np.exp(-v))
    if f == "gelu":
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    if f == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if f == "swiglu":
        g, u = v[..., 0::2], v[..., 1::2]
        return g / (1.0 + np.exp(-g)) * u
    assert f in (None, "none")
    return v


def gemm(fmt, canonical, n_out, n_in, x, bias=None, f=None, residual=None):
    """``f(W x + bias) + residual`` for the rows of ``x``."""
    v = np.asarray(x, np.float64) @ dequantize(fmt_id(fmt), canonical, n_out, n_in).T
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    v = activation(v, f)
    return v if residual is None else v + np.asarray(residual, np.float64)


def gemm_abs(fmt, canonical, n_out, n_in, x):
    """``sum_i |W[o, i] x[t, i]|``, what the products' errors are measured by."""
    return np.abs(np.asarray(x, np.float64)) @ np.abs(dequantize(fmt_id(fmt), canonical, n_out, n_in)).T


def gemm_experts(fmt, canonical, n_experts, n_out, n_in, x, offsets, rows=None, f=None, product=gemm):
    """``{slot: outputs}`` of the slots ``offsets[e] .. offsets[e + 1]`` of every expert e."""
    x, got = np.asarray(x, np.float64), {}
    for e in range(n_experts):
        slots = list(range(int(offsets[e]), int(offsets[e + 1])))
        if not slots:
            continue
        at = slots if rows is None else [int(rows[s]) for s in slots]
        one = row_slice(fmt_id(fmt), canonical, n_experts * n_out, n_in, e * n_out, (e + 1) * n_out)
        y = product(fmt, one, n_out, n_in, x[at])
        for s, v in zip(slots, y if f is None else activation(y, f)):
            got[s] = v
    return got


def prompt_attention(q, k, v, cu_seq, scale, window=0):
    """Packed prompts ``q [n, heads, D]``, ``k``, ``v [n, kv_heads, D]`` -> (out, lse, sum of p |v|),
    rows outside the prompts NaN.  Keys and values that a row does not see take no part."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, heads, D = q.shape
    group = heads // k.shape[1]
    out, lse, spread = np.full((n, heads, D), np.nan), np.full((n, heads), np.nan), np.full((n, heads, D), np.nan)
    for a, b in zip(cu_seq[:-1], cu_seq[1:]):
        for i in range(a, b):
            lo = max(a, i - window + 1) if window else a
            for h in range(heads):
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k[lo:i + 1, h // group] @ q[i, h])
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    p = p / total
                    out[i, h] = p @ v[lo:i + 1, h // group]
                    spread[i, h] = p @ np.abs(v[lo:i + 1, h // group])
                    lse[i, h] = m + np.log(total)
    return out, lse, spread
