"""The calls of a request's life as a user makes them, on one stream: attention
over the prompts, insert of their K and V into the paged cache, a decode step
with its log-sum-exps, the weight every token received, eviction by it, and
the next decode step over what is left."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import evict as OE
from oracle import prompt as OP
import paged_attention_quantized_gb300 as pa
from paged_attention_quantized_gb300 import build as pabuild
from paged_attention_quantized_gb300 import workloads as W
from tests.gpu_check import TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    pabuild.build()


@pytest.mark.parametrize("recipe,D", [("bf16", 128), ("e4m3", 256)])
def test_prompt_insert_attend_weigh_evict_attend(recipe, D):
    prompts, Hq, Hkv, budget, sinks, recent = [150, 33, 90], 8, 2, 64, 2, 16
    # room for the prompt and one new token
    w = W.make(recipe, device="cuda", context_lens=[x + 1 for x in prompts], Hq=Hq, Hkv=Hkv, D=D, n=1)
    g = torch.Generator().manual_seed(1)
    T = sum(prompts)
    cpu = [torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
    q, k, v = (x.cuda() for x in cpu)
    cu = torch.tensor([0] + prompts).cumsum(0).to(torch.int32)
    # 1. the prompts themselves
    pp = pa.prompt_problem(num_seqs=3, total_q=T, total_k=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D)
    out = torch.empty_like(q)
    pa.prompt_attention(pp, q, k, v, cu.cuda(), cu.cuda(), out)
    # 2. their keys and values into the cache, request by request, then the first new token
    final = w.context_lens.clone()
    new = [torch.randn(3, 1, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    for b, n in enumerate(prompts):
        one = dataclasses.replace(w, B=1, n=n, block_table=w.block_table[b:b + 1].contiguous(),
                        context_lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        a, e = int(cu[b]), int(cu[b + 1])
        pa.insert(one, pa.problem(one), k[a:e].contiguous(), v[a:e].contiguous())
    pa.insert(w, pa.problem(w), *new)
    # 3. a decode step
    p = pa.problem(w)
    dec, lse, ws = pa.alloc(w, p)
    pa.run(w, p, dec, ws, lse)
    # 4. who was looked at, 5. keep the budget
    mass = torch.zeros(3, Hkv, w.max_context_len, device="cuda")
    pa.attention_mass(w, p, lse, mass)
    positions = torch.zeros(3, Hkv, w.max_context_len, dtype=torch.int32, device="cuda")
    history = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    before = w.to("cpu")
    mass_cpu, lse_cpu = mass.cpu(), lse.cpu()
    ews = torch.empty(pa.evict_workspace_bytes(p, budget), dtype=torch.uint8, device="cuda")
    pa.evict(w, p, budget, mass, positions, history, mass, positions, history, w.context_lens, ews, sinks=sinks,
             recent=recent)
    # 6. the next step over what is left
    dec2, lse2, ws2 = pa.alloc(w, p)
    pa.run(w, p, dec2, ws2, lse2)
    torch.cuda.synchronize()
    b = pa.binding()
    assert all(b.pa_get_error(x.data_ptr(), pa.stream_handle()) == 0 for x in (ws, ews, ws2))

    # each step against its oracle on the bytes it was given
    ref, _ = OP.prompt_attention(*cpu, cu.tolist(), cu.tolist(), 1 / math.sqrt(D), True)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= TOL["bf16"] * 2   # values up to 4.5: two half steps of bf16
    tol = TOL[w.out_dtype]
    ref, rl = oracle.attention(before)
    assert np.abs(dec.double().cpu().numpy().reshape(ref.shape) - ref).max() <= tol
    want, _ = OE.attention_mass(before, lse_cpu, torch.zeros_like(mass_cpu))
    assert np.abs(mass_cpu.double().numpy() - want).max() <= 1e-5               # weights of at most 4 rows
    ev = OE.evict(before, budget, sinks, recent, mass_cpu, torch.zeros_like(positions.cpu()),
                  torch.zeros(3, 2, dtype=torch.int32))
    after = w.to("cpu")
    assert torch.equal(after.k_pool.view(torch.uint8), ev["k_pool"].view(torch.uint8))
    assert torch.equal(after.v_pool.view(torch.uint8), ev["v_pool"].view(torch.uint8))
    assert torch.equal(after.context_lens, ev["lens"]) and after.context_lens.tolist() == [64, 34, 64]
    ref, _ = oracle.attention(after)
    assert np.abs(dec2.double().cpu().numpy().reshape(ref.shape) - ref).max() <= tol
    # the kept tokens are the attention's own: without the evicted ones' small weights the
    # answer moves by at most the weight that left times the spread of the values
    lost = 1 - np.array([[ev["mass"][i, h].sum() / mass_cpu[i, h].sum() for h in range(Hkv)] for i in range(3)])
    assert lost.min() >= -1e-4 and lost.max() < 0.8
