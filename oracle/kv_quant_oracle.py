"""fp64 oracle of the 8-bit drafter KV cache: append, read and decode attention.

Plain numpy on the definitions in include/peagle.h (peagle_kv_quant and the calls after it);
no code of the CUDA path.  A cache is a pair of arrays: ``codes``, the e4m3 values
[layers, batch, heads, capacity, head_dim] as float64, and ``scale`` [layers, batch, heads,
capacity / block]; the value of a slot is its code times its block's scale.
"""
from __future__ import annotations

import numpy as np

TOP = 448.0  # the largest e4m3 value
E_MIN, E_MAX = -40, 120  # exponents of the scales that append writes


def e4m3_round(x):
    """The nearest e4m3 value, ties to the even one; |x| <= 448.  Three bits follow the leading
    one; below 2^-6 the spacing stays 2^-9."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.round(x / step) * step


def block_scale(amax):
    """The smallest power of two s (exponent E_MIN .. E_MAX) with amax <= 448 s; 1 for zero."""
    amax = np.asarray(amax, np.float64)
    e = np.full(amax.shape, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = np.where(amax > TOP * 2.0 ** k, k + 1, e)
    return np.where(amax > 0, np.ldexp(1.0, e), 1.0)


def append(codes, scale, block, lens, n, rows):
    """Rows [layers, batch, n_max, heads, head_dim] into slots lens[b] .. lens[b] + n[b] - 1;
    returns new (codes, scale)."""
    codes, scale = codes.copy(), scale.copy()
    for b, (at, m) in enumerate(zip(lens, n)):
        at, end = int(at), int(at) + int(m)
        if m <= 0:
            continue
        for i in range(at // block, (end - 1) // block + 1):
            lo, hi = i * block, min((i + 1) * block, end)
            old = max(min(at, hi), lo)
            x = np.concatenate([
                codes[:, b, :, lo:old] * scale[:, b, :, i, None, None],
                np.swapaxes(rows[:, b, max(lo, at) - at:hi - at], 1, 2).astype(np.float64)], 2)
            fine = np.isfinite(x)
            s = block_scale(np.where(fine, np.abs(x), 0.0).max((2, 3)))
            q = e4m3_round(np.where(fine, x, 0.0) / s[..., None, None])
            codes[:, b, :, lo:hi] = np.where(fine, q, np.nan)
            scale[:, b, :, i] = s
    return codes, scale


def values(codes, scale, block):
    return codes * np.repeat(scale, block, -1)[..., None]


def span(length, j, causal, window):
    """Slots [begin, end) that draft row j of a request of this length sees."""
    end = length + j + 1 if causal else length
    return (max(0, length + j - window + 1) if window else 0), end


def attention(q, k, v, lens, K, causal=True, window=0, scale=None):
    """q [batch * K, n_q_heads, head_dim]; k, v [batch, n_kv_heads, capacity, head_dim] values.
    Returns (out, lse, absolute): sum_t p_t v_t, log sum exp, and sum_t p_t |v_t|."""
    BK, nq, hd = q.shape
    G = nq // k.shape[1]
    scale = hd ** -0.5 if scale is None else scale
    out, absolute = np.zeros((BK, nq, hd)), np.zeros((BK, nq, hd))
    lse = np.full((BK, nq), -np.inf)
    for r in range(BK):
        b, j = divmod(r, K)
        begin, end = span(int(lens[b]), j, causal, window)
        if end <= begin:
            continue
        for h in range(nq):
            kk, vv = k[b, h // G, begin:end], v[b, h // G, begin:end]
            x = scale * (kk @ q[r, h])
            m = x.max()
            p = np.exp(x - m)
            lse[r, h] = m + np.log(p.sum())
            p = p / p.sum()
            out[r, h], absolute[r, h] = p @ vv, p @ np.abs(vv)
    return out, lse, absolute
