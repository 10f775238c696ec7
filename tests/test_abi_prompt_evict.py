"""Refusals of pa_prompt_attention, pa_attention_mass and pa_evict, and what
they size, on the host: nothing here launches a kernel."""
import ctypes

import pytest

from paged_attention_quantized_gb300 import build as pabuild


@pytest.fixture(scope="module")
def B():
    pabuild.build()
    from paged_attention_quantized_gb300 import _binding
    return _binding


def prompt(B, **kw):
    base = dict(num_seqs=2, total_q=100, total_k=100, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=B.PA_BF16,
                out_dtype=B.PA_BF16, causal=1, q_stride=0, k_stride=0, v_stride=0, softmax_scale=0.1)
    base.update(kw)
    return B.PromptProblem(**base)


PTR = dict(q=1 << 20, k=2 << 20, v=3 << 20, cq=4 << 20, ck=5 << 20, out=6 << 20, lse=7 << 20, err=None)


def prompt_status(B, p, **ptr):
    d = dict(PTR, **ptr)
    return B.raw_status("pa_prompt_attention", ctypes.byref(p), d["q"], d["k"], d["v"], d["cq"], d["ck"], d["out"],
                        d["lse"], d["err"], None)


@pytest.mark.parametrize("p,ptr,want", [
    (dict(num_seqs=-1), {}, "INVALID_ARG"), (dict(total_q=-1), {}, "INVALID_ARG"), (dict(total_k=-1), {}, "INVALID_ARG"),
    (dict(num_q_heads=9), {}, "INVALID_ARG"), (dict(num_kv_heads=0), {}, "INVALID_ARG"),
    (dict(dtype=0), {}, "INVALID_ARG"), (dict(dtype=3), {}, "INVALID_ARG"), (dict(out_dtype=4), {}, "INVALID_ARG"),
    (dict(causal=2), {}, "INVALID_ARG"), (dict(softmax_scale=0.0), {}, "INVALID_ARG"),
    (dict(softmax_scale=-1.0), {}, "INVALID_ARG"), (dict(softmax_scale=float("nan")), {}, "INVALID_ARG"),
    (dict(softmax_scale=float("inf")), {}, "INVALID_ARG"), (dict(q_stride=1023), {}, "INVALID_ARG"),
    (dict(k_stride=-8), {}, "INVALID_ARG"), (dict(v_stride=255), {}, "INVALID_ARG"),
    (dict(head_dim=96), {}, "UNSUPPORTED"), (dict(head_dim=512), {}, "UNSUPPORTED"),
    (dict(num_q_heads=258), {}, "UNSUPPORTED"), (dict(num_seqs=65536), {}, "UNSUPPORTED"),
    (dict(q_stride=1028), {}, "UNSUPPORTED"), (dict(k_stride=260), {}, "UNSUPPORTED"),
    ({}, dict(q=None), "INVALID_ARG"), ({}, dict(k=None), "INVALID_ARG"), ({}, dict(v=None), "INVALID_ARG"),
    ({}, dict(cq=None), "INVALID_ARG"), ({}, dict(ck=None), "INVALID_ARG"), ({}, dict(out=None), "INVALID_ARG"),
    ({}, dict(q=(1 << 20) + 8), "INVALID_ARG"), ({}, dict(k=(1 << 20) + 2), "INVALID_ARG"),
    ({}, dict(v=(1 << 20) + 4), "INVALID_ARG"), ({}, dict(out=(1 << 20) + 8), "INVALID_ARG"),
    ({}, dict(lse=(1 << 20) + 2), "INVALID_ARG"), ({}, dict(err=(1 << 20) + 1), "INVALID_ARG"),
])
def test_prompt_refusals(B, p, ptr, want):
    assert prompt_status(B, prompt(B, **p), **ptr) == getattr(B, "PA_ERR_" + want)


def test_prompt_without_rows_is_a_no_op(B):
    none = dict.fromkeys(PTR)
    assert prompt_status(B, prompt(B, num_seqs=0), **none) == B.PA_OK
    assert prompt_status(B, prompt(B, total_q=0), **none) == B.PA_OK
    assert B.raw_status("pa_prompt_attention", None, *[None] * 9) == B.PA_ERR_INVALID_ARG


def prob(B, **kw):
    base = dict(batch=4, next_n=1, num_q_heads=32, num_kv_heads=8, head_dim_k=128, head_dim_v=128, block_size=16,
                num_blocks=1000, max_blocks_per_seq=64, max_context_len=1024, q_dtype=B.PA_BF16, kv_dtype=B.PA_BF16,
                out_dtype=B.PA_BF16, k_scale_mode=0, v_scale_mode=0, causal=0, v_is_k_prefix=0, num_sms=152,
                grid_ctas=0, softmax_scale=0.088)
    base.update(kw)
    return B.Problem(**base)


MPTR = dict(q=1 << 20, kp=2 << 20, table=3 << 20, lens=4 << 20, ks=5 << 20, lse=6 << 20, mass=7 << 20, err=None)


def mass_status(B, p, decay=1.0, **ptr):
    d = dict(MPTR, **ptr)
    return B.raw_status("pa_attention_mass", ctypes.byref(p), ctypes.c_float(decay), *[d[k] for k in MPTR], None)


@pytest.mark.parametrize("p,ptr,want", [
    (dict(batch=-1), {}, "INVALID_ARG"), (dict(next_n=0), {}, "INVALID_ARG"), (dict(num_q_heads=30), {}, "INVALID_ARG"),
    (dict(q_dtype=0), {}, "INVALID_ARG"), (dict(kv_dtype=0), {}, "INVALID_ARG"), (dict(kv_dtype=6), {}, "INVALID_ARG"),
    (dict(k_scale_mode=4), {}, "INVALID_ARG"), (dict(causal=2), {}, "INVALID_ARG"),
    (dict(softmax_scale=float("inf")), {}, "INVALID_ARG"), (dict(max_context_len=-1), {}, "INVALID_ARG"),
    (dict(head_dim_k=96), {}, "UNSUPPORTED"), (dict(head_dim_k=576, v_is_k_prefix=1), {}, "UNSUPPORTED"),
    (dict(kv_dtype=5, head_dim_k=64), {}, "UNSUPPORTED"), (dict(block_size=8), {}, "UNSUPPORTED"),
    (dict(batch=4097), {}, "UNSUPPORTED"), (dict(k_scale_mode=2), {}, "UNSUPPORTED"),
    (dict(kv_dtype=4, k_scale_mode=3), {}, "UNSUPPORTED"), (dict(next_n=1 << 19), {}, "UNSUPPORTED"),
    (dict(max_context_len=1 << 29), {}, "UNSUPPORTED"),
    ({}, dict(q=None), "INVALID_ARG"), ({}, dict(kp=None), "INVALID_ARG"), ({}, dict(table=None), "INVALID_ARG"),
    ({}, dict(lens=None), "INVALID_ARG"), ({}, dict(lse=None), "INVALID_ARG"), ({}, dict(mass=None), "INVALID_ARG"),
    (dict(kv_dtype=3, k_scale_mode=1), dict(ks=None), "INVALID_ARG"),
    ({}, dict(q=(1 << 20) + 8), "INVALID_ARG"), ({}, dict(kp=(1 << 20) + 8), "INVALID_ARG"),
    ({}, dict(mass=(1 << 20) + 2), "INVALID_ARG"),
])
def test_mass_refusals(B, p, ptr, want):
    assert mass_status(B, prob(B, **p), **ptr) == getattr(B, "PA_ERR_" + want)


def test_mass_decay_and_empty_calls(B):
    assert mass_status(B, prob(B), decay=float("nan")) == B.PA_ERR_INVALID_ARG
    none = dict.fromkeys(MPTR)
    assert mass_status(B, prob(B, batch=0), **none) == B.PA_OK
    assert mass_status(B, prob(B, max_context_len=0), **none) == B.PA_OK


EPTR = dict(mass=1 << 20, pos=2 << 20, hist=3 << 20, table=4 << 20, lens=5 << 20, kp=6 << 20, vp=7 << 20, mo=8 << 20,
            po=9 << 20, ho=10 << 20, lo=11 << 20, ws=12 << 20)


def evict_status(B, p, budget=100, sinks=0, recent=0, nbytes=1 << 30, **ptr):
    d = dict(EPTR, **ptr)
    return B.raw_status("pa_evict", ctypes.byref(p), budget, sinks, recent, *[d[k] for k in EPTR],
                        ctypes.c_size_t(nbytes), None)


def test_evict_workspace(B):
    # header, request records, counts, two lists of at most min(budget, max_context_len - budget) rows
    assert B.pa_evict_workspace_size(prob(B), 100) == 256 + 256 + 256 + 4 * 8 * 2 * 100 * 4
    assert B.pa_evict_workspace_size(prob(B), 1000) == 256 + 256 + 256 + 4 * 8 * 2 * 24 * 4
    assert B.pa_evict_workspace_size(prob(B), 5000) == 768
    n = ctypes.c_size_t()
    for kw, budget, want in ((dict(), 0, "INVALID_ARG"), (dict(batch=-1), 5, "INVALID_ARG"),
                             (dict(max_context_len=(1 << 19) + 1), 5, "UNSUPPORTED"),
                             (dict(batch=8192), 5, "UNSUPPORTED")):
        st = B.raw_status("pa_evict_workspace_size", ctypes.byref(prob(B, **kw)), budget, ctypes.byref(n))
        assert st == getattr(B, "PA_ERR_" + want), kw


@pytest.mark.parametrize("p,args,want", [
    ({}, dict(budget=0), "INVALID_ARG"), ({}, dict(sinks=-1), "INVALID_ARG"), ({}, dict(recent=-1), "INVALID_ARG"),
    ({}, dict(sinks=60, recent=41), "INVALID_ARG"), (dict(kv_dtype=0), {}, "INVALID_ARG"),
    (dict(block_size=0), {}, "INVALID_ARG"), (dict(k_scale_mode=7), {}, "INVALID_ARG"),
    (dict(v_is_k_prefix=2), {}, "INVALID_ARG"),
    (dict(head_dim_k=100), {}, "UNSUPPORTED"), (dict(head_dim_v=4), {}, "UNSUPPORTED"),
    (dict(kv_dtype=5, head_dim_k=16, head_dim_v=32), {}, "UNSUPPORTED"),
    ({}, dict(ws=None), "WORKSPACE"), ({}, dict(ws=(1 << 20) + 128), "WORKSPACE"), ({}, dict(nbytes=1000), "WORKSPACE"),
    ({}, dict(mass=None), "INVALID_ARG"), ({}, dict(pos=None), "INVALID_ARG"), ({}, dict(hist=None), "INVALID_ARG"),
    ({}, dict(table=None), "INVALID_ARG"), ({}, dict(lens=None), "INVALID_ARG"), ({}, dict(kp=None), "INVALID_ARG"),
    ({}, dict(vp=None), "INVALID_ARG"), ({}, dict(mo=None), "INVALID_ARG"), ({}, dict(po=None), "INVALID_ARG"),
    ({}, dict(ho=None), "INVALID_ARG"), ({}, dict(lo=None), "INVALID_ARG"),
    ({}, dict(kp=(1 << 20) + 8), "INVALID_ARG"), ({}, dict(vp=(1 << 20) + 8), "INVALID_ARG"),
    ({}, dict(mass=(1 << 20) + 2), "INVALID_ARG"), ({}, dict(lo=(1 << 20) + 2), "INVALID_ARG"),
])
def test_evict_refusals(B, p, args, want):
    assert evict_status(B, prob(B, **p), **args) == getattr(B, "PA_ERR_" + want)


def test_evict_of_nothing_is_a_no_op(B):
    none = {k: None for k in EPTR if k != "ws"}
    assert evict_status(B, prob(B, batch=0), **none) == B.PA_OK
