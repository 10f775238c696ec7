"""pa_attention_mass on the GPU against the float64 oracle (oracle/evict.py).

Tolerance, relative to the sum of weights a call adds: a score s = scale sum
q k is off by at most D * 2^-24 (fp32 additions) plus 2^-22 (queries as one
exact or two f16 / bf16 terms) of A = scale * D * max |q'| * max |k'| (q' with
its folded scale, k' the codes), and by 2^-22 of |s| + |lse| from the roundings
of the scale, of lse * log2 e and of their difference; a weight follows it
relatively, plus 2^-22 of ex2; R positive weights add R * 2^-24.  The total is
rounded twice."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import evict as OE
import paged_attention_quantized_gb300 as pa
from paged_attention_quantized_gb300 import build as pabuild
from paged_attention_quantized_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    pabuild.build()


def tamed(w):
    """Per-channel recipes with queries small enough for scores of order one."""
    if w.k_scale_mode == "channel":
        w.q = (w.q.float() / 1e5).to(w.q.dtype)
    return w


def lse_of(w):
    _, lse = oracle.attention(w)
    return torch.from_numpy(lse.reshape(w.B, w.n, w.Hq)).float()


def token_scaled(w, seed=3):
    """The E4M3 workload w with per-token scales in its K blocks (V stays as it is)."""
    g = torch.Generator().manual_seed(seed)
    codes = w.k_pool.reshape(w.num_blocks, -1)
    s = torch.exp(torch.randn(w.num_blocks, w.Hkv * w.bs, generator=g)) * 0.05
    pool = torch.cat([codes, s.view(torch.uint8).reshape(w.num_blocks, -1)], 1).contiguous()
    return dataclasses.replace(w, k_pool=pool, k_scale=None, k_scale_mode="token")


def scores_lse(w):
    """Log-sum-exps straight from the oracle's K rows (for modes the dense oracle does not take)."""
    out = np.full((w.B, w.n, w.Hq), -np.inf)
    G = w.Hq // w.Hkv
    for b in range(w.B):
        L = int(w.context_lens[b])
        for h in range(w.Hq):
            k = OE.k_rows(w, b, h // G)
            for j in range(w.n):
                vis = max(0, L - (w.n - 1 - j)) if w.causal else L
                if vis:
                    x = w.softmax_scale * (k[:vis] @ w.q[b, j, h].double().numpy())
                    out[b, j, h] = x.max() + math.log(np.exp(x - x.max()).sum())
    return torch.from_numpy(out).float()


def run(w, lse, mass, decay=1.0, stream=None):
    d = w.to("cuda")
    p = pa.problem(d)
    m, err = mass.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    l = lse.cuda()
    torch.cuda.synchronize()
    pa.attention_mass(d, p, l, m, decay=decay, dev_error=err, stream=stream)
    torch.cuda.synchronize()
    return m.cpu(), int(err.item())


def bound(w, top, lse, added, out):
    q = w.q.double().abs().max().item() * (w.k_scale.double().max().item() if w.k_scale_mode == "channel" else 1.0)
    k = {"e4m3": 448.0, "int8": 128.0, "int4": 8.0}.get(w.kv_dtype)
    if k is None:
        x = w.k_pool
        k = x[torch.isfinite(x.float())].double().abs().max().item() if x.dtype != torch.uint8 else 6.0
    elif w.k_scale_mode == "tensor":
        k *= float(w.k_scale[0])
    elif w.k_scale_mode == "token":
        k *= 0.05 * math.exp(5)
    A = w.softmax_scale * w.Dk * q * k
    fl = lse[torch.isfinite(lse)].abs().max().item() if torch.isfinite(lse).any() else 0.0
    R = (w.Hq // w.Hkv) * w.n
    rel = A * (w.Dk * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -22 * (top + fl + 1) + R * 2.0 ** -24
    return np.abs(added) * rel + 2.0 ** -23 * np.abs(out) + 1e-30


def check(w, lse, decay=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    mass = torch.rand(w.B, w.Hkv, w.max_context_len, generator=g)
    want, top = OE.attention_mass(w, lse, mass, decay)
    got, bits = run(w, lse, mass, decay)
    assert bits == 0
    got = got.double().numpy()
    added = want - (decay * mass.double().numpy())
    for b in range(w.B):
        L = int(w.context_lens[b])
        err = np.abs(got[b, :, :L] - want[b, :, :L])
        tol = bound(w, top, lse, added[b, :, :L], want[b, :, :L])
        assert (err <= tol).all(), (float((err / tol).max()), b)
        assert np.array_equal(got[b, :, L:], mass[b, :, L:].double().numpy())   # left as they were
    return want


CASES = [  # the warp-level kernel takes up to 8 rows per kv head (16 at head dim 64), the tensor-memory one the others
    ("tiny", dict()),
    ("tiny", dict(context_lens=[1, 0, 17, 129])),
    ("bf16", dict(context_lens=[5, 300], Hq=8, Hkv=2)),
    ("bf16", dict(context_lens=[200, 33], Hq=16, Hkv=1, D=64, bs=32)),
    ("bf16", dict(context_lens=[130, 1, 257], Hq=8, Hkv=2, n=3)),
    ("bf16", dict(context_lens=[260, 40], Hq=8, Hkv=2, n=20, D=256)),
    ("bf16", dict(context_lens=[300], Hq=24, Hkv=8, n=6, D=64)),
    ("e4m3", dict(context_lens=[200, 77], Hq=8, Hkv=2)),
    ("e4m3", dict(context_lens=[129, 30], Hq=16, Hkv=2, D=128, n=17)),
    ("e4m3", dict(context_lens=[65, 140], Hq=8, Hkv=1, D=64, n=5, bs=64)),
    ("int8", dict(context_lens=[100, 150], Hq=8, Hkv=2)),
    ("int8", dict(context_lens=[140, 131], Hq=16, Hkv=2, n=32)),
    ("int8", dict(context_lens=[70], Hq=4, Hkv=1, n=9, D=256)),
    ("int4", dict(context_lens=[100, 150], Hq=8, Hkv=2)),
    ("int4", dict(context_lens=[140, 40], Hq=8, Hkv=1, n=5)),
    ("int4", dict(context_lens=[90], Hq=8, Hkv=2, n=12, D=256)),
]


@pytest.mark.parametrize("name,kw", CASES, ids=lambda x: str(x))
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
def test_matches_oracle(name, kw, decay):
    w = tamed(W.make(name, **kw))
    check(w, lse_of(w), decay)


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 9])
def test_query_and_code_types(q_dtype, n):
    # queries of the other 16-bit type than the codes', and unscaled 8-bit codes
    for kv in ("f16", "bf16", "e4m3"):
        w = W.make("bf16" if kv != "e4m3" else "e4m3", context_lens=[70, 131], Hq=8, Hkv=2, D=128, n=n, poison=False)
        w.q = w.q.to(W.TORCH_FLOAT[q_dtype])
        w.q_dtype = q_dtype
        if kv == "f16":
            w.k_pool = w.k_pool.to(torch.float16) if w.k_pool.dtype != torch.uint8 else \
                w.k_pool.view(torch.bfloat16).to(torch.float16)
            w.kv_dtype = "f16"
        check(w, scores_lse(w))


def test_per_token_scales():
    for n, D in ((1, 128), (2, 64), (12, 128), (7, 256)):
        w = token_scaled(W.make("e4m3", context_lens=[70, 131], Hq=8, Hkv=2, D=D, n=n, poison=False))
        w.q = (w.q.float() * 0.2).to(w.q.dtype)
        check(w, scores_lse(w))


@pytest.mark.parametrize("num_sms", [0, 1])
@pytest.mark.parametrize("name,kw", [("e4m3", dict(Hq=8, Hkv=2, n=3, D=256)), ("e4m3", dict(Hq=32, Hkv=2, n=1, D=128)),
                                     ("int8", dict(Hq=8, Hkv=2, n=4)), ("int4", dict(Hq=18, Hkv=2, n=1)),
                                     ("bf16", dict(Hq=8, Hkv=2, n=4)), ("bf16", dict(Hq=10, Hkv=2, n=2, D=64))],
                         ids=lambda x: str(x))
def test_nine_to_sixteen_rows_on_both_kernels(name, kw, num_sms):
    # quantized codes of wide heads: the tensor-core kernel while there is at most one
    # (request, kv head) per SM, the warp-level one with more of them (num_sms = 1)
    w = tamed(W.make(name, context_lens=[300, 0, 129, 7, 640], **kw))
    lse = lse_of(w)
    g = torch.Generator().manual_seed(1)
    mass = torch.rand(w.B, w.Hkv, w.max_context_len, generator=g)
    want, top = OE.attention_mass(w, lse, mass, 1.0)
    d = w.to("cuda")
    m, err = mass.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.attention_mass(d, pa.problem(d, num_sms=num_sms), lse.cuda(), m, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = m.cpu().double().numpy()
    for b in range(w.B):
        L = int(w.context_lens[b])
        tol = bound(w, top, lse, want[b, :, :L] - mass[b, :, :L].double().numpy(), want[b, :, :L])
        assert (np.abs(got[b, :, :L] - want[b, :, :L]) <= tol).all()
        assert np.array_equal(got[b, :, L:], mass[b, :, L:].double().numpy())


@pytest.mark.parametrize("n", [2, 5, 12, 16, 32])
def test_long_shares_through_every_buffer(n):
    # one SM walks every tile: the operand buffers come round many times, with as many
    # of them as the rows of the query leave room for
    for name, kw in (("bf16", dict(Hq=16, Hkv=2)), ("int8", dict(Hq=16, Hkv=2)), ("bf16", dict(Hq=16, Hkv=2, D=64))):
        w = tamed(W.make(name, context_lens=[2300, 1100], n=n, **kw))
        lse = lse_of(w)
        mass = torch.zeros(w.B, w.Hkv, w.max_context_len)
        want, top = OE.attention_mass(w, lse, mass, 1.0)
        d = w.to("cuda")
        m = mass.cuda()
        pa.attention_mass(d, pa.problem(d, num_sms=1), lse.cuda(), m)
        torch.cuda.synchronize()
        got = m.cpu().double().numpy()
        for b in range(w.B):
            L = int(w.context_lens[b])
            tol = bound(w, top, lse, want[b, :, :L], want[b, :, :L])
            assert (np.abs(got[b, :, :L] - want[b, :, :L]) <= tol).all()


def test_more_rows_than_a_chunk():
    for name, kw in (("int8", dict(Hq=64, Hkv=2, n=9)), ("bf16", dict(Hq=64, Hkv=2, n=5, D=256))):
        w = tamed(W.make(name, context_lens=[150, 12], **kw))
        check(w, lse_of(w), 0.5)


def test_rows_that_saw_nothing_and_empty_requests():
    for n, kw in ((4, dict(Hq=8, Hkv=2)), (12, dict(Hq=8, Hkv=2))):
        w = W.make("bf16", context_lens=[2, 0, n, 40], n=n, **kw)
        w.causal = True
        lse = lse_of(w)
        assert torch.isneginf(lse[0, 0]).all() and torch.isneginf(lse[1]).all()
        check(w, lse)
        check(w, torch.full_like(lse, -math.inf))      # nobody votes


def test_sums_to_the_number_of_rows():
    # every row gives away a weight of one: exact up to the tolerance of the weights
    w = W.make("bf16", context_lens=[1000, 3], Hq=8, Hkv=2, n=1)
    d = w.to("cuda")
    p = pa.problem(d)
    out, lse, ws = pa.alloc(d, p)
    pa.run(d, p, out, ws, lse)
    m = torch.full((2, 2, 1000), math.nan, device="cuda")
    pa.attention_mass(d, p, lse, m, decay=0.0)
    torch.cuda.synchronize()
    for b, L in enumerate((1000, 3)):
        assert (m[b, :, :L].double().sum(-1) - 4).abs().max() <= 4 * 1e-3    # lse: bf16 MMA scores, 1e-3 as in its tests
        assert torch.isnan(m[b, :, L:]).all()                               # decay 0 reads nothing, writes [0, L)


@pytest.mark.parametrize("n", [1, 12])
def test_masked_and_unused_codes_may_be_nan(n):
    # NaN codes in unused slots, the null block and slack (the poisoned recipe); a NaN key
    # reaches its own entry only
    w = W.make("e4m3", context_lens=[61, 130], Hq=8, Hkv=2, D=128, n=n, poison=True)
    lse = lse_of(w)
    want = check(w, lse)
    mass = torch.zeros(w.B, w.Hkv, w.max_context_len)
    base, _ = run(w, lse, mass)
    pool = w.k_pool.clone()
    flat = pool.view(torch.uint8).reshape(w.num_blocks, w.Hkv, w.bs, w.Dk)
    flat[int(w.block_table[1, 40 // w.bs]), 1, 40 % w.bs, 5] = 0x7F
    got, _ = run(dataclasses.replace(w, k_pool=pool), lse, mass)
    assert torch.isnan(got[1, 1, 40])
    got[1, 1, 40] = base[1, 1, 40]
    assert torch.equal(got, base)


@pytest.mark.parametrize("n", [1, 12])
def test_relocation_repeats_streams_and_graphs_are_bitwise(n):
    w = W.make("bf16", context_lens=[300, 77, 1000], Hq=8, Hkv=2, n=n)
    lse, mass = lse_of(w), torch.rand(3, 2, 1000)
    a, _ = run(w, lse, mass)
    b, _ = run(W.relocate(w, seed=4), lse, mass)
    c, _ = run(w, lse, mass, stream=torch.cuda.Stream())
    assert torch.equal(a, b) and torch.equal(a, c)
    d = w.to("cuda")
    p, l, m = pa.problem(d), lse.cuda(), mass.cuda()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            pa.attention_mass(d, p, l, m)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(m.cpu(), a)
    g.replay()
    torch.cuda.synchronize()
    again, _ = run(w, lse, a)
    assert torch.equal(m.cpu(), again)


@pytest.mark.parametrize("n", [1, 12])
def test_broken_requests(n):
    b = pa.binding()
    w = W.make("bf16", context_lens=[100, 100, 100], Hq=8, Hkv=2, n=n)
    lse, mass = lse_of(w), torch.rand(3, 2, 100)
    table, lens = w.block_table.clone(), w.context_lens.clone()
    table[1, 2] = 0                           # the null block at a visible position
    lens[2] = 101
    want, _ = run(w, lse, mass)
    got, bits = run(dataclasses.replace(w, block_table=table, context_lens=lens), lse, mass)
    assert bits == b.PA_DEV_ERR_BLOCK_ID | b.PA_DEV_ERR_CONTEXT_LEN
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], mass[2])
    assert torch.isnan(got[1, :, 32:48]).all()
    got[1, :, 32:48] = want[1, :, 32:48]
    assert torch.equal(got[1], want[1])


def test_refusals():
    w = W.make("bf16", device="cuda", context_lens=[20], Hq=4, Hkv=2)
    b = pa.binding()
    p = pa.problem(w)
    lse, m = torch.zeros(1, 1, 4, device="cuda"), torch.zeros(1, 2, 20, device="cuda")
    for bad in (dict(lse=lse.double()), dict(lse=lse[:, :, :3]), dict(mass=m[:, :, :10]), dict(mass=m.cpu()),
                dict(mass=m.transpose(1, 2))):
        a = dict(lse=lse, mass=m)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.attention_mass(w, p, a["lse"], a["mass"])
    with pytest.raises(b.PaError):
        pa.attention_mass(w, p, lse, m, decay=math.inf)
    lat = W.make("latent", device="cuda", context_lens=[20], Hq=4)
    with pytest.raises(b.PaError):
        pa.attention_mass(lat, pa.problem(lat), torch.zeros(1, 2, 4, device="cuda"), m)
