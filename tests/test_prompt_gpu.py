"""pa_prompt_attention on the GPU against the float64 oracle (oracle/prompt.py).

Tolerances.  A weight p in (0, 1] enters the value product rounded once to the
dtype (half a step, u = 2^-9 / 2^-12 relative for bf16 / f16: eps / 2), its sum
unrounded; so |out - exact| <= u * sum_t w_t |v_t| <= u * max |v| from that,
fp32 accumulation of n terms adds at most n * 2^-24 of the same sum, and the
output is rounded once more, eps / 2 of its value.  Scores in fp32 are off by at
most (D + 2) * 2^-24 * scale * sum |q k|, which moves a weight by that much,
relatively, and the output by at most twice it times max |v|."""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as OP
import paged_attention_quantized_gb300 as pa
from paged_attention_quantized_gb300 import build as pabuild

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    pabuild.build()


def make(lq, lk, Hq, Hkv, D, dtype, seed=0, qs=1.0, gap=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda n, h: torch.randn(n, h, D, generator=g)
    cu = lambda l: torch.tensor([0] + list(l)).cumsum(0).to(torch.int32)
    q, k, v = (qs * t(sum(lq) + gap, Hq)).to(DT[dtype]), t(sum(lk) + gap, Hkv).to(DT[dtype]), t(sum(lk) + gap, Hkv).to(DT[dtype])
    return q, k, v, cu(lq), cu(lk)


def call(q, k, v, cu_q, cu_k, causal=True, out_dtype=None, scale=None, err=None, lse=True, stream=None, **strides):
    dtype = "bf16" if q.dtype == torch.bfloat16 else "f16"
    Tq, Hq, D = q.shape
    p = pa.prompt_problem(num_seqs=len(cu_q) - 1, total_q=Tq, total_k=k.shape[0], num_q_heads=Hq,
                          num_kv_heads=k.shape[1], head_dim=D, dtype=dtype, out_dtype=out_dtype, causal=causal,
                          softmax_scale=scale, **strides)
    out = torch.full((Tq, Hq, D), -77.0, dtype=DT[out_dtype or dtype], device="cuda")
    ls = torch.full((Tq, Hq), -77.0, device="cuda") if lse else None
    dev = [x if x.is_cuda else x.cuda() for x in (q, k, v, cu_q, cu_k)]
    torch.cuda.synchronize()
    pa.prompt_attention(p, *dev, out, ls, dev_error=err, stream=stream)
    torch.cuda.synchronize()
    return out, ls


def check(q, k, v, cu_q, cu_k, out, lse, causal=True, scale=None):
    D = q.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    ref, rl = OP.prompt_attention(q, k, v, cu_q.tolist(), cu_k.tolist(), scale, causal)
    rows = ~np.isnan(rl)
    vmax = float(v[torch.isfinite(v)].abs().max()) if v.numel() else 0.0
    n = max([int(b - a) for a, b in zip(cu_k[:-1], cu_k[1:])] + [1])
    fin = lambda x: x[torch.isfinite(x)].abs().max().item() if x.numel() else 0.0
    score = (D + 2) * 2.0 ** -24 * scale * D * fin(q.double()) * fin(k.double())
    u = torch.finfo(q.dtype).eps / 2
    got = out.double().cpu().numpy()
    tol = vmax * (u + (n + D) * 2.0 ** -24 + 2 * score) + torch.finfo(out.dtype).eps / 2 * np.abs(ref)
    assert np.isfinite(got[rows]).all()
    assert (np.abs(got - ref)[rows] <= tol[rows]).all(), float((np.abs(got - ref) - tol)[rows].max())
    assert (got[~rows] == -77.0).all()       # rows of no sequence are left as they were
    if lse is not None:
        gl = lse.double().cpu().numpy()
        f = rows & np.isfinite(rl)
        assert np.array_equal(gl[rows & ~f], rl[rows & ~f])
        # fp32: the score error, the sum's, one rounding of the value
        assert (np.abs(gl[f] - rl[f]) <= score + (n + 4) * 2.0 ** -24 + 2.0 ** -23 * np.abs(rl[f])).all()
        assert (gl[~rows] == -77.0).all()


SHAPES = [  # lq, lk (None: the same), Hq, Hkv, D, dtype, causal
    ([1], None, 1, 1, 64, "f16", True),
    ([37, 70], None, 4, 1, 64, "f16", True),
    ([1, 2, 1, 127, 128, 129, 130], None, 8, 2, 64, "bf16", True),
    ([33, 0, 64, 65, 1], None, 8, 1, 128, "bf16", True),
    ([31, 32, 33, 63, 64, 300], None, 32, 8, 128, "bf16", True),
    ([200, 17], None, 6, 1, 128, "f16", True),          # 126 of 128 rows of a tile
    ([50, 260], None, 5, 5, 128, "f16", True),
    ([9, 1, 40], [200, 1, 40], 64, 8, 128, "f16", True),  # keys in front
    ([40, 5, 3], [20, 0, 300], 4, 2, 64, "bf16", True),   # rows that see nothing
    ([40, 5], [300, 129], 16, 2, 128, "bf16", False),
    ([7, 129], [0, 128], 4, 4, 64, "f16", False),
    ([1, 130, 65], None, 8, 2, 256, "bf16", True),
    ([20, 3], [400, 131], 12, 2, 256, "f16", True),
    ([70, 5], [257, 64], 4, 4, 256, "bf16", False),
    ([3, 50], None, 128, 1, 64, "bf16", True),          # one token's heads fill a tile
    ([3, 50], None, 100, 1, 128, "f16", True),
    ([2] * 70 + [5] * 30, None, 4, 2, 64, "f16", True),  # more sequences than a warp's registers hold
]


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,dtype,causal", SHAPES, ids=lambda x: str(x)[:40])
def test_matches_oracle(lq, lk, Hq, Hkv, D, dtype, causal):
    x = make(lq, lk or lq, Hq, Hkv, D, dtype, seed=len(lq), gap=3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(*x, causal=causal, err=err)
    assert err.item() == 0
    check(*x, out, lse, causal)


@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_output_types_and_scales(out_dtype, D):
    x = make([70, 3], [90, 3], 4, 2, D, "bf16", seed=3)
    out, lse = call(*x, out_dtype=out_dtype, scale=0.3)
    check(*x, out, lse, True, 0.3)
    out2, _ = call(*x, out_dtype=out_dtype, scale=0.3, lse=False)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_climbing_scores_rescale(D):
    # keys grow along the sequence, so that the maximum moves at almost every block, and
    # shrink, so that it never does
    for s in (1.0, -1.0):
        q, k, v, cq, ck = make([90], [900], 4, 2, D, "f16", seed=4)
        ramp = torch.linspace(0.1, 6.0, 900)
        if s < 0:
            ramp = ramp.flip(0)
        k = (k.float() * ramp[:, None, None]).half()
        out, lse = call(q, k, v, cq, ck)
        check(q, k, v, cq, ck, out, lse)


def test_many_tiles_and_long_keys():
    # several tiles per CTA, checked against float64 on the GPU
    lq = [1500, 3, 700, 64, 2000, 1]
    q, k, v, cq, ck = make(lq, lq, 32, 4, 128, "bf16", seed=5)
    out, lse = call(q, k, v, cq, ck)
    ref, rl = dense(q, k, v, cq, ck)
    close(out, lse, ref, rl, v)


def dense(q, k, v, cq, ck, causal=True):
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    G = q.shape[1] // k.shape[1]
    for a, b, c, d in zip(cq[:-1], cq[1:], ck[:-1], ck[1:]):
        a, b, c, d = int(a), int(b), int(c), int(d)
        for h in range(q.shape[1]):
            z = q[a:b, h].cuda().double() @ k[c:d, h // G].cuda().double().T / math.sqrt(q.shape[2])
            if causal:
                i = torch.arange(b - a, device="cuda")[:, None]
                z.masked_fill_(torch.arange(d - c, device="cuda") > i + (d - c) - (b - a), -math.inf)
            lse[a:b, h] = torch.logsumexp(z, 1)
            out[a:b, h] = torch.softmax(z, 1) @ v[c:d, h // G].cuda().double()
    return out, lse


def close(out, lse, ref, rl, v):
    u = torch.finfo(out.dtype).eps / 2
    vmax = float(v.abs().max())
    assert bool(((out.double() - ref).abs() <= vmax * (u + 2e-4) + u * ref.abs()).all())
    assert bool(((lse.double() - rl).abs() <= 1e-5 * (1 + rl.abs())).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_keys_and_values_may_hold_anything(D):
    # the next sequence's rows, the future of the same sequence, and rows of no sequence
    q, k, v, cq, ck = make([100, 150], [100, 150], 4, 1, D, "bf16", seed=6, gap=5)
    want, wl = call(q, k, v, cq, ck)
    for bad in (math.nan, math.inf, -math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[100:], v2[100:] = bad, bad              # all of the second sequence and the gap
        out, lse = call(q, k2, v2, cq, ck)
        assert torch.equal(out[:100], want[:100]) and torch.equal(lse[:100], wl[:100])
        for t in (60, 99):                         # later keys of the first one
            k2, v2 = k.clone(), v.clone()
            k2[t], v2[t] = bad, bad
            out, lse = call(q, k2, v2, cq, ck)
            assert torch.equal(lse[:t], wl[:t])
            # the rows before it: another order of additions, so both are only within
            # check()'s bound of the exact value -- weights rounded to the dtype against
            # sum w |v| <= max |v|, and one rounding of the output
            u = torch.finfo(out.dtype).eps / 2
            d = (out[:t].double() - want[:t].double()).abs()
            bound = 2 * (float(v.abs().max()) * (u + 400 * 2.0 ** -24) + u * want[:t].abs().double()) + 1e-5
            assert bool((d <= bound).all()), (bad, t)
            assert torch.equal(out[100:250], want[100:250])
            assert not torch.isfinite(out[t:100].float()).all(-1).any()


def test_strides_of_a_fused_projection():
    # q, k and v as slices of one [tokens, Hq + 2 Hkv, D] tensor
    g = torch.Generator().manual_seed(7)
    Hq, Hkv, D = 8, 2, 64
    x = torch.randn(90, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = torch.tensor([0, 30, 90], dtype=torch.int32)
    s = (Hq + 2 * Hkv) * D
    out, lse = call(q, k, v, cu, cu, q_stride=s, k_stride=s, v_stride=s)
    check(*(t.cpu().contiguous() for t in (q, k, v)), cu, cu, out, lse)


def test_bad_prefix_sums_are_flagged():
    b = pa.binding()
    q, k, v, cq, ck = make([40, 30, 20], [40, 30, 20], 4, 2, 64, "f16", seed=8)
    want, wl = call(q, k, v, cq, ck)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, 40, 70, 91], dtype=torch.int32)     # keys past the end
    out, lse = call(q, k, v, cq, bad, err=err)
    assert err.item() == b.PA_DEV_ERR_CONTEXT_LEN
    assert torch.equal(out[:70], want[:70]) and torch.isnan(out[70:].float()).all() and torch.isnan(lse[70:]).all()
    err.zero_()
    bad = torch.tensor([0, 40, -1, 20], dtype=torch.int32)     # a decreasing and a negative query range
    out, lse = call(q, k, v, bad, ck, err=err)
    assert err.item() == b.PA_DEV_ERR_CONTEXT_LEN
    assert torch.equal(out[:40], want[:40]) and (out[40:] == -77).all() and (lse[40:] == -77).all()


def test_streams_graphs_and_repeats_agree():
    q, k, v, cq, ck = (x.cuda() for x in make([300, 70, 1, 90], [300, 200, 1, 90], 8, 2, 128, "bf16", seed=9))
    want, wl = call(q, k, v, cq, ck)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    p = pa.prompt_problem(num_seqs=4, total_q=461, total_k=591, num_q_heads=8, num_kv_heads=2, head_dim=128)
    outs = [torch.empty_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip((s1, s2), outs):
            pa.prompt_attention(p, q, k, v, cq, ck, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    with torch.cuda.stream(s1):
        with torch.cuda.graph(g, stream=s1):
            pa.prompt_attention(p, q, k, v, cq, ck, out, lse)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    # another packing of the same sequences: the rows are bitwise the same
    order = [2, 0, 3, 1]
    rq = torch.cat([torch.arange(int(cq[i]), int(cq[i + 1])) for i in order])
    rk = torch.cat([torch.arange(int(ck[i]), int(ck[i + 1])) for i in order])
    cu = lambda c: torch.tensor([0] + [int(c[i + 1] - c[i]) for i in order]).cumsum(0).to(torch.int32)
    out, lse = call(q[rq].contiguous(), k[rk].contiguous(), v[rk].contiguous(), cu(cq), cu(ck))
    assert torch.equal(out, want[rq]) and torch.equal(lse, wl[rq])


def test_empty_problems_and_wrong_tensors():
    q, k, v, cq, ck = (x.cuda() for x in make([5], [5], 4, 2, 64, "f16"))
    p = pa.prompt_problem(num_seqs=0, total_q=0, total_k=0, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype="f16")
    pa.prompt_attention(p, q[:0], k[:0], v[:0], cq[:1], ck[:1], torch.empty_like(q[:0]))
    p = pa.prompt_problem(num_seqs=1, total_q=5, total_k=5, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype="f16")
    out = torch.empty_like(q)
    for bad in (dict(q=q.float()), dict(q=q[:4]), dict(k=q), dict(v=v.cpu()), dict(cq=cq.long()), dict(ck=ck[:1]),
                dict(out=out[:, :, :32]), dict(q=q.transpose(0, 1)), dict(k=torch.cat([k, k], 1)[:, ::2])):
        a = dict(q=q, k=k, v=v, cq=cq, ck=ck, out=out)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.prompt_attention(p, a["q"], a["k"], a["v"], a["cq"], a["ck"], a["out"])


@pytest.mark.parametrize("B", [33, 65, 700, 5000])
def test_many_short_sequences(B):
    # more sequences than the tile search keeps at hand, of one to three lengths of blocks
    g = torch.Generator().manual_seed(B)
    lq = torch.randint(1, 4, (B,), generator=g).tolist()
    lk = [a + int(x) for a, x in zip(lq, torch.randint(0, 2, (B,), generator=g) * (200 if B < 1000 else 5))]
    q, k, v, cq, ck = make(lq, lk, 4, 2, 64, "bf16", seed=B)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(q, k, v, cq, ck, err=err)
    assert err.item() == 0
    check(q, k, v, cq, ck, out, lse)


def test_prefix_sums_that_name_rows_over_and_over_are_refused():
    b = pa.binding()
    q, k, v, _, _ = make([400], [400], 4, 2, 64, "bf16", seed=1)
    cu = torch.tensor([0, 400] * 40, dtype=torch.int32)      # 40 times the whole, 39 times backwards
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(q, k, v, cu, cu, err=err)
    assert err.item() == b.PA_DEV_ERR_CONTEXT_LEN
    assert (out == -77).all() and (lse == -77).all()
