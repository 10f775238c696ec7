"""Waits that run out in the prompt and weight kernels, against the test build
of the library (2 ms waits): the high bits of the device error word name a copy
of CTA 0 that goes missing.  The kernels set PA_DEV_ERR_TIMEOUT and return; the
rows or entries they did not finish are NaN, the others right, and the context
stays usable."""
import os
import subprocess
import sys

import pytest

from paged_attention_quantized_gb300 import build as pabuild

pytestmark = pytest.mark.gpu

SCRIPT = r"""
import ctypes, math, sys
import torch
import paged_attention_quantized_gb300 as pa
from paged_attention_quantized_gb300 import workloads as W
b = pa.binding()
good = (b._lib.pa_prompt_attention, b._lib.pa_attention_mass)
lib = ctypes.CDLL(sys.argv[1])
for name in ("pa_prompt_attention", "pa_attention_mass"):
    getattr(lib, name).argtypes = getattr(b._lib, name).argtypes
    getattr(lib, name).restype = ctypes.c_int

def nan_or_equal(got, want):
    bad = torch.isnan(got.float())
    assert torch.equal(torch.where(bad, want, got), want)
    return bad

for D in (64, 128, 256):
    lens = [700, 40, 300]          # 700 more keys in front of the first: every tile of it has six blocks or more
    T, TK = sum(lens), sum(lens) + 700
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").bfloat16() for n, h in ((T, 8), (TK, 2), (TK, 2)))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    ck = torch.tensor([0, 1400, 1440, 1740], dtype=torch.int32).cuda()
    p = pa.prompt_problem(num_seqs=3, total_q=T, total_k=TK, num_q_heads=8, num_kv_heads=2, head_dim=D)
    want, wl = torch.empty_like(q), torch.empty(T, 8, device="cuda")
    pa.prompt_attention(p, q, k, v, cu, ck, want, wl)
    for unit in (0, 1, 3, 6):
        out, lse = torch.zeros_like(want), torch.zeros_like(wl)
        err = torch.tensor([(unit + 1) << 8], dtype=torch.int32, device="cuda")
        st = lib.pa_prompt_attention(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(),
                                     ck.data_ptr(), out.data_ptr(), lse.data_ptr(), err.data_ptr(), pa.stream_handle())
        assert st == 0
        torch.cuda.synchronize()
        assert err.item() & 0xFF == b.PA_DEV_ERR_TIMEOUT, (D, unit, err.item())
        bad = nan_or_equal(out, want)
        assert bad.any() and not bad.all(), (D, unit)
        nan_or_equal(lse, wl)
    out, err = torch.zeros_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.prompt_attention(p, q, k, v, cu, ck, out, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, want)

for name, kw in (("bf16", dict(D=128)), ("e4m3", dict(D=64))):
    w = W.make(name, device="cuda", context_lens=[900, 5, 2000], Hq=8, Hkv=2, n=9, poison=False, **kw)
    p = pa.problem(w)
    lse = torch.full((3, 9, 8), 3.0, device="cuda")
    want = torch.zeros(3, 2, 2000, device="cuda")
    pa.attention_mass(w, p, lse, want)
    for tile in (0, 1):
        m = torch.zeros_like(want)
        err = torch.tensor([(tile + 1) << 8], dtype=torch.int32, device="cuda")
        ks = None if w.k_scale is None else w.k_scale.data_ptr()
        p1 = pa.problem(w, num_sms=1)        # one CTA holds every tile
        st = lib.pa_attention_mass(ctypes.byref(p1), 1.0, w.q.data_ptr(), w.k_pool.data_ptr(), w.block_table.data_ptr(),
                                   w.context_lens.data_ptr(), ks, lse.data_ptr(), m.data_ptr(), err.data_ptr(),
                                   pa.stream_handle())
        assert st == 0
        torch.cuda.synchronize()
        assert err.item() & 0xFF == b.PA_DEV_ERR_TIMEOUT
        assert nan_or_equal(m, want).any()
    m = torch.zeros_like(want)
    pa.attention_mass(w, p, lse, m)
    torch.cuda.synchronize()
    assert torch.equal(m, want)
print("ok")
"""


def test_missing_copies_time_out():
    pabuild.build()
    lib = pabuild.build(variant="fi")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT, lib], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
