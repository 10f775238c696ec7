"""Pins of the oracles of prompt attention, accumulated weight and eviction
(oracle/prompt.py, oracle/evict.py) against other routes to the same numbers.
No GPU."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import evict as OE
from oracle import prompt as OP
from paged_attention_quantized_gb300 import workloads as W


def qkv(lq, lk, Hq, Hkv, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    f = lambda n, h: torch.randn(n, h, D, generator=g, dtype=torch.float64)
    cu = lambda l: np.concatenate([[0], np.cumsum(l)]).tolist()
    return f(sum(lq), Hq), f(sum(lk), Hkv), f(sum(lk), Hkv), cu(lq), cu(lk)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_is_torch_attention_per_sequence(causal):
    q, k, v, cq, ck = qkv([5, 1, 8], [5, 4, 11], 6, 2, 16)
    out, lse = OP.prompt_attention(q, k, v, cq, ck, 0.3, causal)
    for s in range(3):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        mask = torch.ones(b - a, d - c, dtype=torch.bool)
        if causal:
            mask = mask.tril((d - c) - (b - a))
        kk, vv = (x[c:d].repeat_interleave(3, 1).transpose(0, 1) for x in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(q[a:b].transpose(0, 1), kk, vv, attn_mask=mask, scale=0.3)
        assert np.abs(out[a:b] - ref.transpose(0, 1).numpy()).max() <= 1e-12
        z = (q[a:b].transpose(0, 1) @ kk.transpose(1, 2) * 0.3).masked_fill(~mask, -math.inf)
        assert np.abs(lse[a:b] - torch.logsumexp(z, -1).T.numpy()).max() <= 1e-12


def test_prompt_last_row_is_the_decode_oracle():
    # the last token of a prompt sees what a decode row sees in a cache of the same keys
    w = W.make("bf16", context_lens=[37], Hq=4, Hkv=2, D=64)
    ref, rl = oracle.attention(w)
    rows = lambda pool: torch.stack([pool.view(torch.bfloat16).reshape(w.num_blocks, 2, w.bs, 64)[
        int(w.block_table[0, t // w.bs]), :, t % w.bs] for t in range(37)])
    q = torch.zeros(37, 4, 64, dtype=torch.bfloat16)
    q[-1] = w.q[0, 0]
    out, lse = OP.prompt_attention(q, rows(w.k_pool), rows(w.v_pool), [0, 37], [0, 37], w.softmax_scale, True)
    assert np.abs(out[-1] - ref.reshape(4, 64)).max() <= 1e-12
    assert np.abs(lse[-1] - rl.reshape(4)).max() <= 1e-12


def test_prompt_empty_rows_and_unnamed_rows():
    q, k, v, cq, ck = qkv([4, 2], [2, 0], 2, 1, 8)
    out, lse = OP.prompt_attention(q, k, v, cq, ck, 1.0, True)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all()     # lk < lq: the first rows see nothing
    assert np.isfinite(lse[2:4]).all() and np.isneginf(lse[4:]).all()
    out, lse = OP.prompt_attention(q, k, v, [0, 3], [0, 2], 1.0, True)
    assert np.isnan(out[3:]).all() and np.isnan(lse[3:]).all()


def test_prompt_hidden_keys_do_not_matter():
    q, k, v, cq, ck = qkv([6], [6], 2, 1, 8)
    want, _ = OP.prompt_attention(q, k, v, cq, ck, 1.0, True)
    k[4], v[4] = math.nan, math.inf
    out, _ = OP.prompt_attention(q, k, v, cq, ck, 1.0, True)
    assert np.array_equal(out[:4], want[:4]) and np.isnan(out[4:]).all()


ENC = [("bf16", dict(D=64)), ("e4m3", dict(D=64, n=3, poison=True)), ("int8", dict(D=64)), ("int4", dict(D=128)),
       ("tiny", {})]


@pytest.mark.parametrize("name,kw", ENC, ids=lambda x: str(x))
def test_mass_is_the_column_sum_of_the_softmax(name, kw):
    w = W.make(name, context_lens=[9, 40], Hq=4, Hkv=2, **kw)
    if w.k_scale_mode == "channel":
        w.q = (w.q.float() / 1e5).to(w.q.dtype)
    _, lse = oracle.attention(w)
    lse = torch.from_numpy(lse.reshape(2, w.n, 4))
    mass = torch.rand(2, 2, w.max_context_len)
    got, _ = OE.attention_mass(w, lse, mass, 0.5)
    added = got - 0.5 * mass.double().numpy()
    for b, L in enumerate((9, 40)):
        # weights of a row add up to one: G * n rows a kv head
        assert np.abs(added[b, :, :L].sum(-1) - 2 * w.n).max() <= 1e-9
        assert np.array_equal(got[b, :, L:], mass[b, :, L:].double().numpy())
    # the decoded K rows give the dense oracle's log-sum-exps
    for b in range(2):
        for h in range(4):
            k = OE.k_rows(w, b, h // 2)
            x = w.softmax_scale * (k @ w.q[b, w.n - 1, h].double().numpy())
            m = x.max()
            assert abs(m + math.log(np.exp(x - m).sum()) - float(lse[b, w.n - 1, h])) <= 1e-9 * max(1.0, abs(m))


def test_mass_decay_zero_ignores_the_old_total_and_empty_rows_add_nothing():
    w = W.make("bf16", context_lens=[2, 5], Hq=2, Hkv=1, D=64, n=3)
    w.causal = True
    _, lse = oracle.attention(w)
    lse = torch.from_numpy(lse.reshape(2, 3, 2))
    nan = torch.full((2, 1, 5), math.nan)
    got, _ = OE.attention_mass(w, lse, nan, 0.0)
    assert abs(got[0, 0, :2].sum() - 4) <= 1e-9 and np.isnan(got[0, 0, 2:]).all()   # two of three rows see anything
    assert abs(got[1, 0].sum() - 6) <= 1e-9
    got, _ = OE.attention_mass(w, torch.full_like(lse, -math.inf), torch.ones(2, 1, 5))
    assert (got == 1).all()


def evict_state(w, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(w.B, w.Hkv, w.max_context_len, generator=g),
            torch.zeros(w.B, w.Hkv, w.max_context_len, dtype=torch.int32), torch.zeros(w.B, 2, dtype=torch.int32))


def rows_of(w, pool, b, g, n):
    rb = w.Dk * W.BITS[w.kv_dtype] // 8
    flat = pool.view(torch.uint8).reshape(w.num_blocks, -1)
    return [bytes(flat[int(w.block_table[b, s // w.bs]),
                       (g * w.bs + s % w.bs) * rb:(g * w.bs + s % w.bs + 1) * rb].tolist()) for s in range(n)]


def test_evict_keeps_the_largest_and_every_kept_token_once():
    w = W.make("bf16", context_lens=[50, 20, 33], Hq=4, Hkv=2, D=64)
    mass, positions, history = evict_state(w)
    e = OE.evict(w, 20, 2, 5, mass, positions, history)
    assert e["lens"].tolist() == [20, 20, 20] and e["history"].tolist() == [[20, 30], [20, 0], [20, 13]]
    for b, L in enumerate((50, 20, 33)):
        for g in range(2):
            old = rows_of(w, w.k_pool, b, g, L)
            new = rows_of(w, e["k_pool"], b, g, 20)
            pos = e["positions"][b, g, :20].tolist()
            assert len(set(pos)) == 20 and {0, 1} <= set(pos) and set(range(L - 5, L)) <= set(pos)
            assert [old[p] for p in pos] == new
            assert e["mass"][b, g, :20].tolist() == [float(mass[b, g, p]) for p in pos]
            out = set(range(L)) - set(pos)
            mid = [p for p in pos if 2 <= p < L - 5]
            if out and mid:
                assert max(float(mass[b, g, p]) for p in out) <= min(float(mass[b, g, p]) for p in mid)
            # a kept token below the new end stays where it is
            assert all(pos[s] == s for s in range(20) if s in pos and s < 20)
    # nothing else of the pool changes
    changed = (e["k_pool"].view(torch.uint8) != w.k_pool.view(torch.uint8)).reshape(w.num_blocks, -1).any(1)
    allowed = {int(w.block_table[b, s // w.bs]) for b in range(3) for s in range(20)}
    assert set(torch.nonzero(changed)[:, 0].tolist()) <= allowed


def test_evict_uses_recorded_positions():
    w = W.make("bf16", context_lens=[30], Hq=2, Hkv=1, D=64)
    mass, positions, history = evict_state(w, 1)
    history[0] = torch.tensor([24, 100])              # 24 recorded slots, 100 tokens dropped before
    positions[0, 0, :24] = torch.randperm(124)[:24].to(torch.int32)
    positions[0, 0, 7] = 0                            # the sink sits in slot 7
    mass[0, 0, 7] = -1.0
    e = OE.evict(w, 10, 1, 4, mass, positions, history)
    pos = e["positions"][0, 0, :10].tolist()
    assert pos[7] == 0 and {126, 127, 128, 129} <= set(pos)
    assert e["history"].tolist() == [[10, 120]]


def test_evict_twice_is_evict_once():
    w = W.make("int8", context_lens=[40], Hq=2, Hkv=1, D=64)
    st = evict_state(w, 2)
    e = OE.evict(w, 16, 1, 3, *st)
    again = OE.evict(dataclasses.replace(w, k_pool=e["k_pool"], v_pool=e["v_pool"]), 16, 1, 3, *st)
    assert torch.equal(again["k_pool"], e["k_pool"]) and torch.equal(again["positions"], e["positions"])


def test_planted_mistakes_are_seen():
    # an off-by-one horizon, a dropped head, and a stable compaction differ from the definition
    q, k, v, cq, ck = qkv([6], [6], 2, 1, 8)
    a, _ = OP.prompt_attention(q, k, v, cq, ck, 1.0, True)
    b, _ = OP.prompt_attention(q, k[:-1], v[:-1], cq, [0, 5], 1.0, True)
    assert np.abs(a - b).max() > 1e-3
    w = W.make("bf16", context_lens=[30], Hq=2, Hkv=1, D=64)
    st = evict_state(w, 3)
    e = OE.evict(w, 10, 0, 2, *st)
    assert e["positions"][0, 0, :10].tolist() != sorted(e["positions"][0, 0, :10].tolist())
