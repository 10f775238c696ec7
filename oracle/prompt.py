"""CPU oracle of attention over packed prompts, in float64.

For each sequence, one query row and head at a time, straight from the
definition: scores against the visible keys only (masked positions are never
read), a two-pass softmax, the weighted sum of the values.
"""
from __future__ import annotations

import math

import numpy as np


def prompt_attention(q, k, v, cu_q, cu_k, softmax_scale: float, causal: bool):
    """(out [total_q, Hq, D], lse [total_q, Hq]) as float64; rows that no
    sequence names are NaN.  q, k, v: torch CPU tensors [rows, heads, D];
    cu_q, cu_k: integer sequences."""
    q, k, v = (x.double().numpy() for x in (q, k, v))
    Hq, Hkv = q.shape[1], k.shape[1]
    out = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for s in range(len(cu_q) - 1):
        q0, lq, k0, lk = int(cu_q[s]), int(cu_q[s + 1] - cu_q[s]), int(cu_k[s]), int(cu_k[s + 1] - cu_k[s])
        for i in range(lq):
            vis = max(0, min(lk, i + 1 + lk - lq)) if causal else lk
            for h in range(Hq):
                g = h // (Hq // Hkv)
                if vis == 0:
                    out[q0 + i, h], lse[q0 + i, h] = 0.0, -math.inf
                    continue
                x = softmax_scale * (k[k0:k0 + vis, g] @ q[q0 + i, h])
                m = x.max()
                p = np.exp(x - m)
                out[q0 + i, h] = (p @ v[k0:k0 + vis, g]) / p.sum()
                lse[q0 + i, h] = m + math.log(p.sum())
    return out, lse
