"""pa_evict on the GPU against the oracle (oracle/evict.py): pools, mass,
positions, history and lengths are compared byte for byte, since an eviction
computes nothing -- it orders and moves."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from oracle import evict as OE
import paged_attention_quantized_gb300 as pa
from paged_attention_quantized_gb300 import build as pabuild
from paged_attention_quantized_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    pabuild.build()


def state_of(w, seed=0, base=0, dropped=0, ties=False):
    """(mass, positions, history) on the CPU: a long-tailed mass, and for base
    > 0 distinct positions below base + dropped in no order."""
    g = torch.Generator().manual_seed(seed)
    mass = torch.exp(1.5 * torch.randn(w.B, w.Hkv, w.max_context_len, generator=g))
    if ties:
        mass = torch.floor(mass)
    positions = torch.full((w.B, w.Hkv, w.max_context_len), -7, dtype=torch.int32)
    history = torch.zeros(w.B, 2, dtype=torch.int32)
    for b in range(w.B):
        n = min(base, int(w.context_lens[b]))
        history[b, 0], history[b, 1] = n, dropped
        for h in range(w.Hkv):
            positions[b, h, :n] = torch.randperm(n + dropped, generator=g)[:n].to(torch.int32)
    return mass, positions, history


def run(w, budget, sinks, recent, mass, positions, history, in_place=False, graph=False, stream=None):
    """(pools and outputs on the CPU, error bits) of one call; w and the state are CPU objects."""
    d = w.to("cuda")
    p = pa.problem(d)
    m, ps, h = mass.cuda(), positions.cuda(), history.cuda()
    if in_place:
        mo, po, ho, lo = m, ps, h, d.context_lens
    else:
        mo, po, ho, lo = m.clone(), ps.clone(), h.clone(), d.context_lens.clone()
    ws = torch.full((pa.evict_workspace_bytes(p, budget),), 0xA5, dtype=torch.uint8, device="cuda")

    def call():
        pa.evict(d, p, budget, m, ps, h, mo, po, ho, lo, ws, sinks=sinks, recent=recent, stream=stream)

    torch.cuda.synchronize()
    if graph:
        gr, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(st):
            with torch.cuda.graph(gr, stream=st):
                call()
        gr.replay()
        gr.replay()
    else:
        call()
    torch.cuda.synchronize()
    bits = pa.binding().pa_get_error(ws.data_ptr(), pa.stream_handle())
    out = dict(k_pool=d.k_pool.cpu(), v_pool=None if d.v_pool is None else d.v_pool.cpu(), mass=mo.cpu(),
               positions=po.cpu(), history=ho.cpu(), lens=lo.cpu())
    return out, bits


def same(got, want):
    for k, x in want.items():
        if x is None:
            assert got[k] is None
        elif k.endswith("pool"):
            assert torch.equal(got[k].view(torch.uint8), x.view(torch.uint8)), k
        elif k == "mass":
            assert torch.equal(got[k].view(torch.int32), x.view(torch.int32)), k
        else:
            assert torch.equal(got[k], x), k


CASES = [
    # workload, its sizes, budget, sinks, recent, base, dropped
    ("tiny", dict(), 16, 1, 4, 0, 0),
    ("tiny", dict(context_lens=[1, 0, 2]), 1, 1, 0, 0, 0),
    ("bf16", dict(context_lens=[5, 64, 65, 200, 640], Hq=8, Hkv=2), 64, 4, 16, 0, 0),
    ("bf16", dict(context_lens=[129, 130, 131], Hq=8, Hkv=4), 128, 2, 30, 128, 900),
    ("e4m3", dict(context_lens=[700, 33, 1000], Hq=8, Hkv=2, n=1), 100, 0, 100, 0, 0),
    ("int8", dict(context_lens=[300, 299], Hq=4, Hkv=1), 299, 0, 0, 17, 3),
    ("int4", dict(context_lens=[300, 80], Hq=4, Hkv=2), 79, 3, 7, 40, 5),
    ("latent", dict(context_lens=[200, 65, 130], Hq=16), 64, 1, 2, 0, 0),
]


@pytest.mark.parametrize("name,kw,budget,sinks,recent,base,dropped", CASES, ids=lambda x: str(x))
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_oracle(name, kw, budget, sinks, recent, base, dropped, in_place):
    w = W.make(name, **kw)
    st = state_of(w, 1, base, dropped)
    want = OE.evict(w, budget, sinks, recent, *st)
    got, bits = run(w, budget, sinks, recent, *st, in_place=in_place)
    assert bits == 0
    same(got, want)


def test_equal_masses_keep_the_lower_slot():
    w = W.make("bf16", context_lens=[400, 401], Hq=4, Hkv=2)
    for mass in (torch.zeros(2, 2, 401), torch.full((2, 2, 401), math.inf), -torch.zeros(2, 2, 401)):
        _, positions, history = state_of(w)
        got, _ = run(w, 100, 0, 10, mass, positions, history)
        same(got, OE.evict(w, 100, 0, 10, mass, positions, history))
    st = state_of(w, 3, ties=True)
    got, _ = run(w, 100, 4, 10, *st)
    same(got, OE.evict(w, 100, 4, 10, *st))


def test_special_masses_are_ordered():
    # NaN below -inf below finite below +inf; +0 and -0 tie
    w = W.make("bf16", context_lens=[40], Hq=2, Hkv=1)
    mass = torch.linspace(-3, 3, 40).reshape(1, 1, 40).clone()
    mass[0, 0, 5], mass[0, 0, 6], mass[0, 0, 7], mass[0, 0, 8] = math.nan, math.inf, -math.inf, -math.nan
    mass[0, 0, 20], mass[0, 0, 21] = 0.0, -0.0
    _, positions, history = state_of(w)
    for budget in (1, 2, 19, 20, 21, 36, 37, 38, 39, 40):
        want = OE.evict(w, budget, 0, 0, mass, positions, history)
        got, _ = run(w, budget, 0, 0, mass, positions, history)
        same(got, want)


@pytest.mark.parametrize("L", [4097, 16385, 32769, 70001])
def test_long_rows(L):
    # each way of holding the keys; checked against torch's stable sort
    w = W.make("bf16", context_lens=[L, L // 2], Hq=2, Hkv=1, D=64)
    mass, positions, history = state_of(w, 5, ties=True)
    budget, sinks, recent = L // 3, 4, 100
    got, bits = run(w, budget, sinks, recent, mass, positions, history)
    assert bits == 0
    for b, n in enumerate((L, L // 2)):
        key = mass[b, 0, :n].clone()
        key[:sinks] = math.inf
        key[n - recent:] = math.inf
        kept = torch.sort(torch.argsort(-key, stable=True)[:budget]).values
        stay, come = kept[kept < budget], kept[kept >= budget]
        free = torch.ones(budget, dtype=torch.bool)
        free[stay] = False
        pos = torch.empty(budget, dtype=torch.int32)
        pos[stay] = stay.int()
        pos[free] = come.int()
        assert torch.equal(got["positions"][b, 0, :budget], pos)
        assert torch.equal(got["mass"][b, 0, :budget], mass[b, 0, pos.long()])
        assert not got["mass"][b, 0, budget:n].any() and got["lens"][b] == budget
        rows = lambda pool, s: pool.view(torch.int16)[w.block_table[b, s // w.bs].long(), 0, s % w.bs]
        for new, old in ((got["k_pool"], w.k_pool), (got["v_pool"], w.v_pool)):
            new, old = (x.reshape(w.num_blocks, 1, w.bs, -1) for x in (new, old))
            s = torch.arange(budget)
            assert torch.equal(rows(new, s), rows(old, pos.long()))
    got2, _ = run(w, budget, sinks, recent, mass, positions, history)
    same(got2, got)


def test_replayed_graph_moves_the_same_rows():
    w = W.make("e4m3", context_lens=[300, 20, 777], Hq=8, Hkv=2, n=1)
    st = state_of(w, 2)
    got, bits = run(w, 128, 4, 16, *st, graph=True)
    assert bits == 0
    same(got, OE.evict(w, 128, 4, 16, *st))


def test_again_and_again():
    # a generation: 9 new tokens, evict to 40, eight times over, state in place
    w = W.make("bf16", context_lens=[49, 49], Hq=4, Hkv=2, D=64)
    mass, positions, history = state_of(w)
    d, h = w.to("cuda"), w
    p = pa.problem(d)
    m, ps, hi = mass.cuda(), positions.cuda(), history.cuda()
    ws = torch.empty(pa.evict_workspace_bytes(p, 40), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(9)
    for step in range(8):
        want = OE.evict(h, 40, 2, 6, mass, positions, history)
        pa.evict(d, p, 40, m, ps, hi, m, ps, hi, d.context_lens, ws, sinks=2, recent=6)
        torch.cuda.synchronize()
        same(dict(k_pool=d.k_pool.cpu(), v_pool=d.v_pool.cpu(), mass=m.cpu(), positions=ps.cpu(), history=hi.cpu(),
                  lens=d.context_lens.cpu()), want)
        seen = 49 + 9 * step
        kept = want["positions"][:, :, :40]
        for pos in [0, 1] + list(range(seen - 6, seen)):    # the sinks and the newest are always there
            assert bool((kept == pos).any(-1).all()), (step, pos)
        mass, positions, history = want["mass"], want["positions"], want["history"]
        mass[:, :, 40:49] = torch.rand(2, 2, 9, generator=g)
        m.copy_(mass)
        h = dataclasses.replace(h, k_pool=want["k_pool"], v_pool=want["v_pool"],
                                context_lens=torch.tensor([49, 49], dtype=torch.int32))
        d.context_lens.fill_(49)


def test_broken_requests_are_left_alone():
    w = W.make("bf16", context_lens=[100, 100, 100, 100], Hq=4, Hkv=2)
    b = pa.binding()
    mass, positions, history = state_of(w, 4)
    table, lens = w.block_table.clone(), w.context_lens.clone()
    table[1, 3] = w.num_blocks                # a visible block id past the pool
    lens[2] = w.max_context_len + 1           # a length past the bound
    history[3, 0] = 101                       # more recorded positions than tokens
    bad = dataclasses.replace(w, block_table=table, context_lens=lens)
    got, bits = run(bad, 50, 0, 8, mass, positions, history)
    assert bits == b.PA_DEV_ERR_BLOCK_ID | b.PA_DEV_ERR_CONTEXT_LEN
    ok = dataclasses.replace(w, B=1, block_table=w.block_table[:1], context_lens=w.context_lens[:1])
    want = OE.evict(ok, 50, 0, 8, mass[:1], positions[:1], history[:1])
    assert torch.equal(got["k_pool"].view(torch.uint8), want["k_pool"].view(torch.uint8))
    assert torch.equal(got["v_pool"].view(torch.uint8), want["v_pool"].view(torch.uint8))
    assert torch.equal(got["mass"][:1], want["mass"]) and torch.equal(got["mass"][1:], mass[1:])
    assert torch.equal(got["positions"][1:], positions[1:]) and torch.equal(got["history"][1:], history[1:])
    assert got["lens"].tolist() == [50, 100, w.max_context_len + 1, 100]


def test_two_streams_and_their_workspaces():
    ws_ = [W.make("bf16", context_lens=[300, 200], Hq=8, Hkv=4, seed=s) for s in (1, 2)]
    sts = [state_of(w, i) for i, w in enumerate(ws_)]
    wants = [OE.evict(w, 90, 1, 9, *st) for w, st in zip(ws_, sts)]
    streams = [torch.cuda.Stream() for _ in ws_]
    for _ in range(3):
        devs, outs = [], []
        for w, st, s in zip(ws_, sts, streams):
            d = w.to("cuda")
            p = pa.problem(d)
            t = [x.cuda() for x in st]
            o = [x.clone() for x in t] + [d.context_lens.clone()]
            k = torch.empty(pa.evict_workspace_bytes(p, 90), dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            devs.append((d, p, t, o, k))
        for (d, p, t, o, k), s in zip(devs, streams):
            pa.evict(d, p, 90, *t, *o, k, sinks=1, recent=9, stream=s)
        torch.cuda.synchronize()
        for (d, p, t, o, k), want in zip(devs, wants):
            same(dict(k_pool=d.k_pool.cpu(), v_pool=d.v_pool.cpu(), mass=o[0].cpu(), positions=o[1].cpu(),
                      history=o[2].cpu(), lens=o[3].cpu()), want)


def test_wrong_tensors_are_refused():
    w = W.make("tiny", device="cuda")
    p = pa.problem(w)
    m = torch.zeros(w.B, w.Hkv, w.max_context_len, device="cuda")
    ps, h = m.int(), torch.zeros(w.B, 2, dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.evict_workspace_bytes(p, 8), dtype=torch.uint8, device="cuda")
    good = [m, ps, h, m.clone(), ps.clone(), h.clone(), w.context_lens.clone(), ws]
    for i, bad in ((0, m.double()), (0, m[:, :, :-1]), (1, m), (2, h[:1]), (3, m.cpu()), (6, h[:, 0])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.evict(w, p, 8, *args)
    with pytest.raises(pa.binding().PaError):
        pa.evict(w, p, 8, *good, sinks=5, recent=4)
