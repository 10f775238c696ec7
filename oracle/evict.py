"""CPU oracles of the accumulated attention weight and of the eviction by it.

Both walk the definition entry by entry on the cache of a Workload (CPU
tensors): `attention_mass` decodes K through the same table walk as the dense
oracle and sums float64 weights, `evict` orders slots by (always kept, mass,
lower slot) and moves bytes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_attention_quantized_gb300 import workloads as W


def k_rows(w, b: int, g: int) -> np.ndarray:
    """The K rows of request b and kv head g as float64 [L, Dk], dequantized."""
    L = int(w.context_lens[b])
    bits = W.BITS[w.kv_dtype]
    rb = w.Dk * bits // 8
    block = w.Hkv * w.bs * rb + (w.Hkv * w.bs * 4 if w.k_scale_mode == "token" else 0)
    pool = w.k_pool.contiguous().view(torch.uint8).reshape(w.num_blocks, -1)
    assert pool.shape[1] == block
    out = np.zeros((L, w.Dk))
    for t in range(L):
        blk, slot = int(w.block_table[b, t // w.bs]), t % w.bs
        at = (g * w.bs + slot) * rb
        raw = pool[blk, at:at + rb]
        if w.kv_dtype in ("f16", "bf16"):
            x = raw.clone().view(W.TORCH_FLOAT[w.kv_dtype]).double().numpy()
        elif w.kv_dtype == "e4m3":
            x = raw.clone().view(torch.float8_e4m3fn).double().numpy()
        elif w.kv_dtype == "int8":
            x = raw.clone().view(torch.int8).double().numpy()
        else:
            u = raw.to(torch.int16)
            x = torch.stack((((u & 15) ^ 8) - 8, ((u >> 4) ^ 8) - 8), -1).reshape(-1).double().numpy()
        if w.k_scale_mode == "tensor":
            x = x * float(w.k_scale[0])
        elif w.k_scale_mode == "channel":
            x = x * w.k_scale[g].double().numpy()
        elif w.k_scale_mode == "token":
            at = w.Hkv * w.bs * rb + (g * w.bs + slot) * 4
            x = x * float(pool[blk, at:at + 4].clone().view(torch.float32)[0])
        out[t] = x
    return out


def attention_mass(w, lse, mass, decay: float = 1.0):
    """(mass after the call, the largest |score| met) for CPU tensors lse
    [B, n, Hq] and mass [B, Hkv, max_context_len]."""
    out = mass.double().numpy().copy()
    q, lse = w.q.double().numpy(), lse.double().numpy()
    G, top = w.Hq // w.Hkv, 0.0
    for b in range(w.B):
        L = int(w.context_lens[b])
        for g in range(w.Hkv):
            k = k_rows(w, b, g)
            add = np.zeros(L)
            for j in range(w.n):
                vis = max(0, L - (w.n - 1 - j)) if w.causal else L
                for h in range(g * G, (g + 1) * G):
                    if lse[b, j, h] == -math.inf or vis == 0:
                        continue
                    x = w.softmax_scale * (k[:vis] @ q[b, j, h])
                    top = max(top, float(np.abs(x).max()))
                    add[:vis] += np.exp(x - lse[b, j, h])
            out[b, g, :L] = add if decay == 0.0 else decay * out[b, g, :L] + add
    return out, top


def evict(w, budget: int, sinks: int, recent: int, mass, positions, history):
    """What pa_evict leaves, on CPU copies: a dict of k_pool, v_pool, mass,
    positions, history, lens."""
    kp = w.k_pool.clone()
    vp = None if w.v_pool is None else w.v_pool.clone()
    mo, po, ho = mass.clone(), positions.clone(), history.clone()
    lens = w.context_lens.clone()
    bits = W.BITS[w.kv_dtype]
    planes = [(kp, w.Dk * bits // 8, w.k_scale_mode)]
    if vp is not None:
        planes.append((vp, w.Dv * bits // 8, w.v_scale_mode))
    for b in range(w.B):
        L, (base, dropped) = int(w.context_lens[b]), (int(x) for x in history[b])
        left = min(L, budget)
        lens[b] = left
        ho[b, 0], ho[b, 1] = left, dropped + L - left
        for g in range(w.Hkv):
            pos = [int(positions[b, g, s]) if s < base else dropped + s for s in range(L)]

            def rank(s):
                always = pos[s] < sinks or pos[s] >= L + dropped - recent
                m = float(mass[b, g, s])
                return (0 if always else 1, 0.0 if always else (math.inf if math.isnan(m) else -m),
                        1 if (not always and math.isnan(m)) else 0, s)

            kept = sorted(sorted(range(L), key=rank)[:left])
            stay = [s for s in kept if s < left]
            move = [s for s in kept if s >= left]
            free = [s for s in range(left) if s not in set(stay)]
            for s in stay:
                po[b, g, s] = pos[s]
            mo[b, g, left:L] = 0.0
            for s, d in zip(move, free):
                mo[b, g, d], po[b, g, d] = mass[b, g, s], pos[s]
                for pool, rb, mode in planes:
                    flat = pool.view(torch.uint8).reshape(w.num_blocks, -1)
                    bs_, bd = int(w.block_table[b, s // w.bs]), int(w.block_table[b, d // w.bs])
                    i, j = (g * w.bs + s % w.bs), (g * w.bs + d % w.bs)
                    flat[bd, j * rb:(j + 1) * rb] = flat[bs_, i * rb:(i + 1) * rb].clone()
                    if mode == "token":
                        o = w.Hkv * w.bs * rb
                        flat[bd, o + 4 * j:o + 4 * j + 4] = flat[bs_, o + 4 * i:o + 4 * i + 4].clone()
    return dict(k_pool=kp, v_pool=vp, mass=mo, positions=po, history=ho, lens=lens)
