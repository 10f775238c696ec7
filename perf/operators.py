"""Measured cases of three operators that belong together around a paged KV cache.

  prompt   attention over whole prompts: packed sequences of different lengths,
           grouped heads, causal (aligned at the end when a sequence's keys are
           longer than its queries, as after a cached prefix), with log-sum-exp
  mass     attention weight that every cached token received from the newest
           query rows, added to a running total (the scores of an eviction)
  evict    keep the `budget` tokens of the largest accumulated weight of every
           (request, kv head), always with the first and the newest tokens, and
           move the kept ones to the front of the paged cache

`run` computes them with elementary torch operations, or -- with `own` set --
with this package's calls on the same inputs.  Sequence lengths are a function
of the case alone; the values are drawn from the seed on the GPU.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

KV_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8, "int8": torch.uint8}
BYTES = {"f16": 2, "bf16": 2, "e4m3": 1, "int8": 1}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # two short fp16 prompts of one group of heads: launch latency
        dict(name="prompt_tiny", op="prompt", B=2, q_lo=37, q_hi=70, pre_lo=0, pre_hi=0, Hq=4, Hkv=1, D=64,
             dtype="f16", causal=True),
        # a serving batch of chat prompts, very different lengths, packed without padding
        dict(name="prompt_ragged", op="prompt", B=32, q_lo=16, q_hi=1024, pre_lo=0, pre_hi=0, Hq=32, Hkv=8, D=128,
             dtype="bf16", causal=True),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, q_lo=16384, q_hi=16384, pre_lo=0, pre_hi=0, Hq=32, Hkv=8, D=128,
             dtype="bf16", causal=True),
        # prompts of the wide-head model that the E4M3 verify batch belongs to
        dict(name="prompt_wide_heads", op="prompt", B=4, q_lo=1024, q_hi=4096, pre_lo=0, pre_hi=0, Hq=32, Hkv=8,
             D=256, dtype="bf16", causal=True),
        # the next chunk of prompts whose first part is there already
        dict(name="prompt_chunk", op="prompt", B=8, q_lo=64, q_hi=512, pre_lo=1024, pre_hi=8192, Hq=64, Hkv=8, D=128,
             dtype="f16", causal=True),
        # one decode step of two short requests: launch latency
        dict(name="mass_tiny", op="mass", B=2, lo=37, hi=70, n=1, Hq=4, Hkv=1, D=64, bs=16, q_dtype="f16",
             kv="f16"),
        # one decode step of the bf16 serving batch
        dict(name="mass_decode", op="mass", B=64, lo=512, hi=8192, n=1, Hq=32, Hkv=8, D=128, bs=16, q_dtype="bf16",
             kv="bf16"),
        # a verify step of the E4M3 batch: four causal rows per request
        dict(name="mass_verify_e4m3", op="mass", B=32, lo=1024, hi=32768, n=4, Hq=32, Hkv=8, D=256, bs=32,
             q_dtype="bf16", kv="e4m3"),
        # the last 32 rows of prompts vote on an INT8 cache with per-channel scales
        dict(name="mass_window_int8", op="mass", B=16, lo=2048, hi=16384, n=32, Hq=64, Hkv=8, D=128, bs=16,
             q_dtype="f16", kv="int8"),
        # every step of a long generation: a few tokens over the budget
        dict(name="evict_step", op="evict", B=64, lo=2049, hi=2064, budget=2048, sinks=4, recent=256, again=True,
             Hkv=8, D=128, bs=16, kv="bf16"),
        # once after the prompts: down to 2048 tokens
        dict(name="evict_prompt", op="evict", B=16, lo=2048, hi=16384, budget=2048, sinks=4, recent=64, again=False,
             Hkv=8, D=128, bs=16, kv="bf16"),
        # the long E4M3 batch down to 4096 tokens
        dict(name="evict_e4m3", op="evict", B=32, lo=1024, hi=32768, budget=4096, sinks=16, recent=512, again=False,
             Hkv=8, D=256, bs=32, kv="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "mass", "mass", "evict"])
    Hq, Hkv = rng.choice([(4, 1), (32, 8), (64, 8), (6, 1), (8, 8), (16, 2)])
    D = rng.choice([64, 128, 128, 256])
    if op == "prompt":
        while True:
            B = _log_int(rng, 1, 48)
            hi = _log_int(rng, 1, 8192)
            pre = rng.choice([0, 0, _log_int(rng, 1, 8192)])
            if B * Hq * hi * (hi + pre) <= 1 << 32:
                break
        return dict(op=op, B=B, q_lo=_log_int(rng, 1, hi), q_hi=hi, pre_lo=pre // 2, pre_hi=pre, Hq=Hq, Hkv=Hkv, D=D,
                    dtype=rng.choice(["f16", "bf16"]), causal=rng.random() < 0.85)
    kv = rng.choice(["f16", "bf16", "e4m3", "int8"])
    bs = rng.choice([16, 32, 64])
    if op == "mass":
        n = rng.choice([1, 1, 2, 4, _log_int(rng, 5, 32)])
        while True:
            B, hi = _log_int(rng, 1, 96), _log_int(rng, n, 32768)
            if B * Hkv * hi * max(D, n * (Hq // Hkv)) <= 1 << 30:
                break
        return dict(op=op, B=B, lo=_log_int(rng, n, hi), hi=hi, n=n, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                    q_dtype="bf16" if kv == "bf16" else "f16" if kv in ("f16", "int8") else rng.choice(["f16", "bf16"]),
                    kv=kv)
    while True:
        B, hi = _log_int(rng, 1, 96), _log_int(rng, 64, 32768)
        if B * Hkv * hi * D * BYTES[kv] <= 1 << 31:
            break
    again = rng.random() < 0.4
    budget = max(32, hi - rng.randint(1, 32)) if again else _log_int(rng, 32, hi)
    return dict(op=op, B=B, lo=budget + 1 if again else _log_int(rng, 32, hi), hi=max(hi, budget + 1), budget=budget,
                sinks=rng.choice([0, 1, 4]), recent=rng.randint(0, budget // 4), again=again, Hkv=Hkv, D=D, bs=bs,
                kv=kv)


def _rng(c):
    return random.Random("lengths " + repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _q_k_lens(c):
    """Query and key lengths of the prompts: log-uniform in the case's ranges, the longest among them."""
    r = _rng(c)
    lq = [_log_int(r, c["q_lo"], c["q_hi"]) for _ in range(c["B"])]
    lq[r.randrange(c["B"])] = c["q_hi"]
    pre = [r.randint(c["pre_lo"], c["pre_hi"]) for _ in lq]
    return lq, [a + b for a, b in zip(lq, pre)]


def _lens(c):
    """Context lengths of the cache: uniform in the case's range, the longest among them."""
    r = _rng(c)
    L = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    L[r.randrange(c["B"])] = c["hi"]
    return L


# --------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _cache(c, L, g, planes):
    """A paged cache: blocks of [Hkv][bs][D] in a permuted order, block 0 never used."""
    bs, D, Hkv = c["bs"], c["D"], c["Hkv"]
    cols = [-(-x // bs) for x in L]
    blocks = 1 + sum(cols)
    ids = 1 + torch.randperm(blocks - 1, generator=g, device="cuda")
    width = max(cols)
    col = torch.arange(width, device="cuda")
    n_cols = torch.tensor(cols, device="cuda")
    before = torch.cumsum(n_cols, 0) - n_cols
    used = col[None] < n_cols[:, None]
    table = torch.where(used, ids[torch.where(used, before[:, None] + col[None], 0)], 0).to(torch.int32)
    pools, scale = [], None
    for _ in range(planes):
        x = _randn(g, blocks, Hkv, bs, D, dtype=torch.bfloat16 if c["kv"] == "bf16" else torch.float16)
        if c["kv"] == "e4m3":       # one scale for the plane
            scale = torch.full((1,), 0.05, device="cuda")
            x = (x / 0.05).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif c["kv"] == "int8":     # a scale per kv head and channel, within a factor of ten
            scale = 10.0 ** (torch.rand(Hkv, D, generator=g, device="cuda") - 0.5) / 127
            x = torch.round(x * (127 / 3)).clamp(-127, 127).to(torch.int8).view(torch.uint8)
        pools.append(x)
    return SimpleNamespace(block_table=table, context_lens=torch.tensor(L, dtype=torch.int32, device="cuda"), B=c["B"],
                           Hkv=Hkv, Dk=D, Dv=D, bs=bs, num_blocks=blocks, max_blocks_per_seq=width,
                           max_context_len=max(L), kv_dtype=c["kv"], k_scale=scale, v_scale=scale,
                           k_scale_mode={"e4m3": "tensor", "int8": "channel"}.get(c["kv"], "none"),
                           v_scale_mode={"e4m3": "tensor", "int8": "channel"}.get(c["kv"], "none"), v_is_k_prefix=False,
                           softmax_scale=1 / math.sqrt(D), k_pool=pools[0], v_pool=pools[1] if planes > 1 else None,
                           causal=True, n=1, Hq=Hkv, q_dtype="bf16", out_dtype="f32")


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "prompt":
        lq, lk = _q_k_lens(c)
        dt = KV_TORCH[c["dtype"]]
        st = SimpleNamespace(
            op="prompt", D=c["D"], causal=c["causal"], max_q=max(lq), max_k=max(lk), scale=1 / math.sqrt(c["D"]),
            q=(2 * _randn(g, sum(lq), c["Hq"], c["D"])).to(dt), k=_randn(g, sum(lk), c["Hkv"], c["D"]).to(dt),
            v=_randn(g, sum(lk), c["Hkv"], c["D"]).to(dt),
            cu_q=torch.tensor([0] + lq, device="cuda").cumsum(0).to(torch.int32),
            cu_k=torch.tensor([0] + lk, device="cuda").cumsum(0).to(torch.int32))
        st.out = torch.empty_like(st.q)
        st.lse = torch.empty(sum(lq), c["Hq"], device="cuda")
        if own:
            import paged_attention_quantized_gb300 as pa
            st.p = pa.prompt_problem(num_seqs=c["B"], total_q=sum(lq), total_k=sum(lk), num_q_heads=c["Hq"],
                                     num_kv_heads=c["Hkv"], head_dim=c["D"], dtype=c["dtype"], causal=c["causal"])
        return st
    L = _lens(c)
    if c["op"] == "mass":
        w = _cache(c, L, g, 1)
        w.n, w.Hq, w.q_dtype = c["n"], c["Hq"], c["q_dtype"]
        w.q = _randn(g, w.B, w.n, w.Hq, w.Dk).to(KV_TORCH[c["q_dtype"]])
        st = SimpleNamespace(op="mass", w=w)
        # what the attention of the same step returned
        st.lse = torch.empty(w.B, w.n, w.Hq, device="cuda")
        for b in range(w.B):
            s = _scores(w, slice(b, b + 1))
            st.lse[b] = torch.logsumexp(s, -1).view(w.Hkv, w.n, w.Hq // w.Hkv).transpose(0, 1).reshape(w.n, w.Hq)
        st.mass = torch.rand(w.B, w.Hkv, w.max_context_len, generator=g, device="cuda") * 0.01
        if own:
            import paged_attention_quantized_gb300 as pa
            st.p = pa.problem(w)
        return st
    w = _cache(c, L, g, 2)
    st = SimpleNamespace(op="evict", w=w, budget=c["budget"], sinks=c["sinks"], recent=c["recent"])
    # accumulated attention weight has a long tail
    st.mass = torch.exp(1.5 * _randn(g, w.B, w.Hkv, w.max_context_len))
    base, dropped = (c["budget"], 700 + seed % 5) if c["again"] else (0, 0)
    st.positions = torch.zeros(w.B, w.Hkv, w.max_context_len, dtype=torch.int32, device="cuda")
    if base:    # what an earlier eviction kept: the first, the newest and some between, in no order
        at = torch.arange(base + dropped, device="cuda")
        key = torch.rand(w.B, w.Hkv, base + dropped, generator=g, device="cuda")
        key = torch.where((at < c["sinks"]) | (at >= base + dropped - c["recent"]), key - 1, key)
        kept = key.argsort(-1)[..., :base]
        mixed = torch.rand(w.B, w.Hkv, base, generator=g, device="cuda").argsort(-1)
        st.positions[..., :base] = kept.gather(-1, mixed).to(torch.int32)
    st.history = torch.tensor([[base, dropped]] * w.B, dtype=torch.int32, device="cuda")
    st.mass_out, st.positions_out = torch.zeros_like(st.mass), torch.zeros_like(st.positions)
    st.history_out, st.lens_out = torch.zeros_like(st.history), torch.zeros_like(w.context_lens)
    if own:
        import paged_attention_quantized_gb300 as pa
        st.p = pa.problem(w)
        st.workspace = torch.empty(pa.evict_workspace_bytes(st.p, st.budget), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------ the operators


def _prompt(s):
    """Padded to the longest sequence: scores, mask, softmax, values."""
    cu_q, cu_k = s.cu_q.long(), s.cu_k.long()
    lq, lk = cu_q.diff(), cu_k.diff()
    i = torch.arange(s.max_q, device="cuda")
    t = torch.arange(s.max_k, device="cuda")
    at_q = (cu_q[:-1, None] + i).clamp(max=s.q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + t).clamp(max=s.k.shape[0] - 1)
    Hkv, G = s.k.shape[1], s.q.shape[1] // s.k.shape[1]
    B = lq.numel()
    q = s.q[at_q].float().view(B, s.max_q, Hkv, G, s.D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * s.max_q, s.D)
    k = s.k[at_k].float().permute(0, 2, 3, 1)
    v = s.v[at_k].float().permute(0, 2, 1, 3)
    seen = t < lk[:, None, None]
    if s.causal:
        seen = seen & (t <= i[:, None] + (lk - lq)[:, None, None])
    x = torch.matmul(q * s.scale, k).view(B, Hkv, G, s.max_q, s.max_k)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * s.max_q, s.max_k), v).view(B, Hkv, G, s.max_q, s.D)
    o = torch.where(total > 0, o / total, 0)
    lse = (m + total.log())[..., 0]
    tok = torch.arange(s.q.shape[0], device="cuda")
    b = torch.searchsorted(cu_q, tok, right=True) - 1
    j = tok - cu_q[b]
    return [o[b, :, :, j].reshape(s.q.shape).to(s.q.dtype), lse[b, :, :, j].reshape(s.q.shape[:2])]


def _values(w, pool, scale, blocks):
    x = pool[blocks]
    if w.kv_dtype == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * scale
    if w.kv_dtype == "int8":
        return x.view(torch.int8).float() * scale[:, None, :]
    return x.float()


def _scores(w, rows=slice(None)):
    """softmax_scale * q . k of every cached token, -inf where a row does not see it: [b, Hkv, n * G, t]."""
    table = w.block_table[rows].long()
    b = table.shape[0]
    k = _values(w, w.k_pool, w.k_scale, table).permute(0, 2, 1, 3, 4).reshape(b, w.Hkv, -1, w.Dk)
    G = w.Hq // w.Hkv
    q = w.q[rows].float().view(b, w.n, w.Hkv, G, w.Dk).transpose(1, 2).reshape(b, w.Hkv, w.n * G, w.Dk)
    x = torch.matmul(q * w.softmax_scale, k.transpose(2, 3))
    t = torch.arange(x.shape[-1], device="cuda")
    j = torch.arange(w.n, device="cuda").repeat_interleave(G)
    vis = w.context_lens[rows, None] - (w.n - 1 - j)
    return x.masked_fill_((t >= vis[..., None])[:, None], -math.inf)


def _mass(s):
    w = s.w
    lse = s.lse.view(w.B, w.n, w.Hkv, w.Hq // w.Hkv).transpose(1, 2).reshape(w.B, w.Hkv, -1, 1)
    got = _scores(w).sub_(lse).exp_().sum(2)[..., : w.max_context_len]
    s.mass += got
    return [s.mass]


def _evict(s):
    w = s.w
    L = w.context_lens.long()[:, None, None]
    slot = torch.arange(w.max_context_len, device="cuda")
    base, dropped = (s.history[:, i, None, None].long() for i in (0, 1))
    pos = torch.where(slot < base, s.positions.long(), dropped + slot)
    always = (pos < s.sinks) | (pos >= L + dropped - s.recent)
    key = torch.where(slot < L, torch.where(always, math.inf, s.mass), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    left = L.clamp(max=s.budget)
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, order, (slot < left).expand(key.shape))
    b, g, dst = torch.nonzero(~kept & (slot < left), as_tuple=True)
    src = torch.nonzero(kept & (slot >= left), as_tuple=True)[2]
    s.mass_out.copy_(torch.where(slot < left, s.mass, torch.where(slot < L, 0, s.mass_out)))
    s.positions_out.copy_(torch.where(slot < left, pos, s.positions_out))
    s.mass_out[b, g, dst] = s.mass[b, g, src]
    s.positions_out[b, g, dst] = pos[b, g, src].to(torch.int32)
    to, of = (w.block_table[b, x // w.bs].long() for x in (dst, src))
    for pool in (w.k_pool, w.v_pool):
        pool[to, g, dst % w.bs] = pool[of, g, src % w.bs]
    s.lens_out.copy_(left[:, 0, 0])
    s.history_out.copy_(torch.stack([left[:, 0, 0], (dropped + L - left)[:, 0, 0]], 1))


def run(state):
    s = state
    if own:
        import paged_attention_quantized_gb300 as pa
    if s.op == "prompt":
        if not own:
            return _prompt(s)
        pa.prompt_attention(s.p, s.q, s.k, s.v, s.cu_q, s.cu_k, s.out, s.lse)
        return [s.out, s.lse]
    if s.op == "mass":
        if not own:
            return _mass(s)
        pa.attention_mass(s.w, s.p, s.lse, s.mass)
        return [s.mass]
    if own:
        pa.evict(s.w, s.p, s.budget, s.mass, s.positions, s.history, s.mass_out, s.positions_out, s.history_out,
                 s.lens_out, s.workspace, sinks=s.sinks, recent=s.recent)
    else:
        _evict(s)
    as_values = (lambda x: x.view(torch.float8_e4m3fn) if s.w.kv_dtype == "e4m3" else
                 x.view(torch.int8) if s.w.kv_dtype == "int8" else x)
    return [as_values(s.w.k_pool), as_values(s.w.v_pool), s.mass_out, s.positions_out, s.history_out, s.lens_out]


def work(case):
    c = case
    if c["op"] == "prompt":
        lq, lk = _q_k_lens(c)
        # row i of a sequence sees keys 0 .. i + lk - lq when causal
        pairs = sum(a * b - a * (a - 1) // 2 if c["causal"] else a * b for a, b in zip(lq, lk))
        return {"bytes": 4.0 * c["D"] * (sum(lq) * c["Hq"] + sum(lk) * c["Hkv"]) + 4.0 * sum(lq) * c["Hq"],
                "flops": 4.0 * c["D"] * c["Hq"] * pairs}
    L = _lens(c)
    row = c["D"] * BYTES[c["kv"]]
    if c["op"] == "mass":
        return {"bytes": float(sum(L) * c["Hkv"] * (row + 8) + c["B"] * c["n"] * c["Hq"] * (2 * c["D"] + 4)),
                "flops": 2.0 * c["D"] * c["Hq"] * sum(c["n"] * x - c["n"] * (c["n"] - 1) // 2 for x in L)}
    got = 0.0
    for x in L:
        k = min(x, c["budget"])
        # a kept token past the new end moves into the slot of one before it
        # that goes: of k slots at the front, k * (1 - k / x) on average
        moved = k * (1 - k / x)
        # mass in and out, positions out (and in, where there are any), K and V rows read and written
        got += 8 * x + 4 * k + (4 * k if c["again"] else 0) + moved * 4 * row
    return {"bytes": got * c["Hkv"], "flops": 0.0}


# ------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "prompt":
        lq, lk = _q_k_lens(c)
        G = c["Hq"] // c["Hkv"]
        out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s.lse.shape, dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for a, n in zip(lq, lk):
            for h in range(c["Hq"]):
                k, v = (x[k0:k0 + n, h // G].double() for x in (s.k, s.v))
                for r in range(0, a, 4096):
                    e = min(a, r + 4096)
                    z = s.q[q0 + r:q0 + e, h].double() @ k.T / math.sqrt(c["D"])
                    if c["causal"]:
                        row = torch.arange(r, e, device="cuda")[:, None]
                        z[torch.arange(n, device="cuda")[None] > row + (n - a)] = -math.inf
                    lse[q0 + r:q0 + e, h] = torch.logsumexp(z, 1)
                    out[q0 + r:q0 + e, h] = torch.softmax(z, 1) @ v
            q0, k0 = q0 + a, k0 + n
        return [out, lse]
    L = _lens(c)
    w = s.w
    if c["op"] == "mass":
        got = s.mass.double()
        G = w.Hq // w.Hkv
        for b, x in enumerate(L):
            page = w.block_table[b, : -(-x // w.bs)].long()
            for g in range(w.Hkv):
                k = w.k_pool[page, g].reshape(-1, w.Dk)[:x]
                if c["kv"] == "e4m3":
                    k = k.view(torch.float8_e4m3fn).double() * w.k_scale.double()
                elif c["kv"] == "int8":
                    k = k.view(torch.int8).double() * w.k_scale[g].double()
                k = k.double()
                for j in range(w.n):
                    see = x - (w.n - 1 - j)
                    h = slice(g * G, (g + 1) * G)
                    z = w.q[b, j, h].double() @ k[:see].T / math.sqrt(w.Dk)
                    got[b, g, :see] += torch.exp(z - s.lse[b, j, h].double()[:, None]).sum(0)
        return [got]
    mass = s.mass.double().cpu()
    out = torch.zeros_like(mass)
    positions, history = s.positions.cpu(), s.history.cpu().tolist()
    for b, x in enumerate(L):
        base, dropped = history[b]
        left = min(x, c["budget"])
        for g in range(w.Hkv):
            pos = torch.cat([positions[b, g, :base].long(), dropped + torch.arange(base, x)])
            m = mass[b, g, :x].clone()
            m[(pos < c["sinks"]) | (pos >= x + dropped - c["recent"])] = math.inf
            kept = torch.sort(torch.argsort(-m, stable=True)[:left]).values
            stay, come = kept[kept < left], kept[kept >= left]
            free = torch.ones(left, dtype=torch.bool)
            free[stay] = False
            out[b, g, stay] = mass[b, g, stay]
            out[b, g, torch.nonzero(free)[:, 0]] = mass[b, g, come]
    return [None, None, out, None, None, None]
