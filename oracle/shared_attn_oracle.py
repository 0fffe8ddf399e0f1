"""fp64 oracle of decode attention over a shared prefix and each request's own slots.

Plain numpy on the definition in include/peagle.h (peagle_decode_attention_shared); no code of
the CUDA path.
"""
from __future__ import annotations

import numpy as np


def attention(q, pk, pv, prefix, k, v, lens, K, causal=True, scale=None):
    """q [batch * K, nq, hd]; pk, pv [nkv, >= prefix, hd]; k, v [batch, nkv, cap, hd].  Returns out, the
    log-sum-exp [batch * K, nq], and each row's sum of |weight x value| [batch * K, nq, hd] (for the
    bounds of roundings)."""
    rows, nq, hd = q.shape
    nkv = pk.shape[0]
    G = nq // nkv
    scale = hd ** -0.5 if scale is None else scale
    out, size = np.zeros((2, rows, nq, hd))
    lse = np.full((rows, nq), -np.inf)
    for row in range(rows):
        b, j = divmod(row, K)
        n = int(lens[b]) + (j + 1 if causal else 0)
        for h in range(nq):
            g = h // G
            kk = np.concatenate([pk[g, :prefix], k[b, g, :n]])
            vv = np.concatenate([pv[g, :prefix], v[b, g, :n]])
            if not len(kk):
                continue
            x = scale * (kk @ q[row, h])
            m = x.max()
            w = np.exp(x - m)
            lse[row, h] = m + np.log(w.sum())
            out[row, h] = w @ vv / w.sum()
            size[row, h] = w @ np.abs(vv) / w.sum()
    return out, lse, size
