"""Paged decode / verify attention over a quantized paged KV cache on GB300.

The computation lives in libpa.so (CUDA, sm_103a) behind the C ABI of
include/pa.h; this package is its thin Python face:

  * `_binding`  -- ctypes declarations of pa_workspace_size / pa_plan / pa_run /
                   pa_combine / pa_attention / pa_insert / pa_sparse_attention /
                   pa_fp4_logits / pa_prompt_attention / pa_attention_mass /
                   pa_evict / pa_get_error (same names);
  * `problem()` / `run()` -- marshal a batch held in torch CUDA tensors into
                   those calls (pointers, sizes, the current stream);
  * `workloads` -- seeded synthetic inputs (no attention arithmetic).

The library is loaded lazily so that `workloads` can be used without it.
"""
from __future__ import annotations

import math
from typing import Optional

__all__ = ["problem", "workspace_bytes", "run", "insert", "sparse_run", "fp4_problem", "fp4_logits",
           "prompt_problem", "prompt_attention", "attention_mass", "evict_workspace_bytes", "evict",
           "stream_handle", "binding"]


def binding():
    from . import _binding
    return _binding


def problem(w, *, num_sms: int = 0, grid_ctas: int = 0,
            max_context_len: Optional[int] = None, out_dtype: Optional[str] = None):
    """pa_problem for a workload-shaped batch (see workloads.Workload)."""
    b = binding()
    return b.Problem(
        batch=w.B, next_n=w.n, num_q_heads=w.Hq, num_kv_heads=w.Hkv, head_dim_k=w.Dk, head_dim_v=w.Dv,
        block_size=w.bs, num_blocks=w.num_blocks, max_blocks_per_seq=w.max_blocks_per_seq,
        max_context_len=w.max_context_len if max_context_len is None else max_context_len,
        q_dtype=b.DTYPE[w.q_dtype], kv_dtype=b.DTYPE[w.kv_dtype],
        out_dtype=b.DTYPE[out_dtype or w.out_dtype], k_scale_mode=b.SCALE[w.k_scale_mode],
        v_scale_mode=b.SCALE[w.v_scale_mode], causal=int(bool(w.causal)),
        v_is_k_prefix=int(bool(w.v_is_k_prefix)), num_sms=num_sms, grid_ctas=grid_ctas,
        softmax_scale=float(w.softmax_scale))


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def stream_handle(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def workspace_bytes(p) -> int:
    return binding().pa_workspace_size(p)


def run(w, p, out, workspace, lse=None, stream=None, *, steps: str = "all") -> None:
    """Enqueue the attention for workload tensors already on the device.

    steps: "all" (pa_attention), or any of "plan", "run", "combine"
    separated by '+'.  All buffers are caller-owned torch tensors."""
    b = binding()
    s = stream_handle(stream)
    ws, wsb = _ptr(workspace), workspace.numel() * workspace.element_size()
    args_run = (_ptr(w.q), _ptr(w.k_pool), _ptr(w.v_pool), _ptr(w.block_table), _ptr(w.context_lens),
                _ptr(w.k_scale), _ptr(w.v_scale))
    if steps == "all":
        b.pa_attention(p, *args_run, ws, wsb, _ptr(out), _ptr(lse), s)
        return
    for step in steps.split("+"):
        if step == "plan":
            b.pa_plan(p, _ptr(w.context_lens), _ptr(w.k_scale), ws, wsb, s)
        elif step == "run":
            b.pa_run(p, *args_run, ws, wsb, _ptr(out), _ptr(lse), s)
        elif step == "combine":
            b.pa_combine(p, _ptr(w.v_scale), ws, wsb, _ptr(out), _ptr(lse), s)
        else:
            raise ValueError(step)


def insert(w, p, k_new, v_new=None, dev_error=None, stream=None) -> None:
    """Enqueue pa_insert: write the new rows k_new / v_new ([B, n, Hkv, D]
    torch CUDA tensors, f32 / f16 / bf16) into w's pools in place.  dev_error:
    optional int32 CUDA tensor of one element that collects the error bits."""
    b = binding()
    src = {"torch.float32": b.PA_F32, "torch.float16": b.PA_F16, "torch.bfloat16": b.PA_BF16}[str(k_new.dtype)]
    b.pa_insert(p, src, _ptr(k_new), _ptr(v_new), _ptr(w.block_table), _ptr(w.context_lens), _ptr(w.k_scale),
                _ptr(w.v_scale), _ptr(w.k_pool), _ptr(w.v_pool), _ptr(dev_error), stream_handle(stream))


def sparse_run(w, p, sel, out, workspace, lse=None, stream=None) -> None:
    """Enqueue pa_sparse_attention for workload tensors on the device; sel is
    an int32 [B, n, top_k] CUDA tensor of selected logical positions and
    workspace a uint8 tensor of pa_sparse_workspace_size bytes."""
    b = binding()
    top_k = int(sel.shape[-1])
    b.pa_sparse_attention(p, top_k, _ptr(sel), _ptr(w.q), _ptr(w.k_pool), _ptr(w.v_pool), _ptr(w.block_table),
                          _ptr(w.context_lens), _ptr(w.k_scale), _ptr(w.v_scale), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), stream_handle(stream))


def out_torch_dtype(name: str):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def alloc(w, p, device="cuda"):
    """(out, lse, workspace) tensors sized for problem p (NaN-filled out)."""
    import torch
    out = torch.full((w.B, w.n, w.Hq, w.Dv), math.nan, dtype=out_torch_dtype(w.out_dtype), device=device)
    lse = torch.full((w.B, w.n, w.Hq), math.nan, dtype=torch.float32, device=device)
    nbytes = workspace_bytes(p)
    ws = torch.zeros(max(256, nbytes), dtype=torch.uint8, device=device)
    return out, lse, ws


def fp4_problem(w, *, num_sms: int = 0, grid_ctas: int = 0, out_stride: int = 0):
    """pa_fp4_problem for an FP4 MQA-logits batch (see workloads.Fp4Logits)."""
    b = binding()
    return b.Fp4Problem(batch=w.B, next_n=w.n, num_heads=w.H, head_dim=w.D, sf_vec_size=w.sf_vec, block_size=w.bs,
                        num_blocks=w.num_blocks, max_blocks_per_seq=w.max_blocks_per_seq,
                        max_context_len=w.max_context_len, out_dtype=b.DTYPE[w.out_dtype], out_stride=out_stride,
                        causal=int(bool(w.causal)), rectify=int(bool(w.rectify)),
                        sf_interleaved=int(bool(w.sf_interleaved)), num_sms=num_sms, grid_ctas=grid_ctas)


def fp4_logits(w, p, out, workspace, stream=None) -> None:
    """Enqueue pa_fp4_logits for an Fp4Logits batch on the device; out is a
    [B * next_n, >= max_context_len] tensor of the problem's output dtype
    (its row stride is taken from p.out_stride, 0 = max_context_len) and
    workspace a uint8 tensor of pa_fp4_logits_workspace_size bytes."""
    b = binding()
    b.pa_fp4_logits(p, _ptr(w.q), _ptr(w.sf_q), _ptr(w.kv_fused), _ptr(w.weights), _ptr(w.context_lens),
                    _ptr(w.block_table), _ptr(workspace), workspace.numel(), _ptr(out), stream_handle(stream))


_late = None  # torch and the binding, imported at the first call that needs them


def _torch_and_binding():
    global _late
    if _late is None:
        import torch
        b = binding()
        _late = (torch, b, {b.PA_F32: torch.float32, b.PA_F16: torch.float16, b.PA_BF16: torch.bfloat16},
                 torch.cuda.current_device, torch._C._cuda_getCurrentRawStream)
    return _late


def _need(t, name: str, dtype, numel: int, dev: int) -> int:
    """The address of a contiguous CUDA tensor of at least numel elements on the current device dev, or a ValueError
    (dtype None: any)."""
    if t.get_device() != dev or (dtype is not None and t.dtype is not dtype) or t.numel() < numel \
            or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor of at least {numel} elements of {dtype or 'any type'} on "
                         f"device {dev} is needed, got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def prompt_problem(*, num_seqs: int, total_q: int, total_k: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   dtype: str = "bf16", out_dtype: Optional[str] = None, causal: bool = True,
                   softmax_scale: Optional[float] = None, q_stride: int = 0, k_stride: int = 0, v_stride: int = 0):
    """pa_prompt_problem for packed prompts: num_seqs sequences of total_q
    query and total_k key rows in all.  Strides are the elements between rows
    (0 = contiguous [rows][heads][head_dim]); softmax_scale defaults to
    1/sqrt(head_dim), out_dtype to dtype."""
    b = binding()
    return b.PromptProblem(num_seqs=num_seqs, total_q=total_q, total_k=total_k, num_q_heads=num_q_heads,
                           num_kv_heads=num_kv_heads, head_dim=head_dim, dtype=b.DTYPE[dtype],
                           out_dtype=b.DTYPE[out_dtype or dtype], causal=int(bool(causal)), q_stride=q_stride,
                           k_stride=k_stride, v_stride=v_stride,
                           softmax_scale=1.0 / math.sqrt(head_dim) if softmax_scale is None else softmax_scale)


def prompt_attention(p, q, k, v, cu_q, cu_k, out, lse=None, dev_error=None, stream=None) -> None:
    """Enqueue pa_prompt_attention: causal (or full) attention of packed
    prompts.  q [total_q, Hq, D] and k, v [total_k, Hkv, D] (rows q_stride,
    k_stride, v_stride elements apart, each row contiguous), cu_q and cu_k
    int32 [num_seqs + 1], out [total_q, Hq, D], lse optional float32
    [total_q, Hq], dev_error an optional int32 tensor of one element that
    collects the error bits."""
    torch, b, types, device, raw_stream = _torch_and_binding()
    dev = device()
    st = raw_stream(dev) if stream is None else stream.cuda_stream
    dt, D, tq, tk, Hq, Hkv = types.get(p.dtype), p.head_dim, p.total_q, p.total_k, p.num_q_heads, p.num_kv_heads

    def rows(t, name, heads, stride, n):
        stride, sh, by = stride or heads * D, t.shape, t.stride()
        if t.get_device() != dev or t.dtype is not dt or len(sh) != 3 or sh[0] < n or sh[1] != heads or sh[2] != D \
                or (n > 0 and (by[2] != 1 or by[1] != D or (by[0] != stride and n > 1))):
            raise ValueError(f"{name}: [{n}, {heads}, {D}] rows of {dt}, {stride} elements apart, on device {dev} are "
                             f"needed, got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
        return t.data_ptr()

    i32 = torch.int32
    b.pa_prompt_attention(p, rows(q, "q", Hq, p.q_stride, tq), rows(k, "k", Hkv, p.k_stride, tk),
                          rows(v, "v", Hkv, p.v_stride, tk), _need(cu_q, "cu_q", i32, p.num_seqs + 1, dev),
                          _need(cu_k, "cu_k", i32, p.num_seqs + 1, dev),
                          _need(out, "out", types.get(p.out_dtype), tq * Hq * D, dev),
                          None if lse is None else _need(lse, "lse", torch.float32, tq * Hq, dev),
                          None if dev_error is None else _need(dev_error, "dev_error", i32, 1, dev), st)


def attention_mass(w, p, lse, mass, decay: float = 1.0, dev_error=None, stream=None) -> None:
    """Enqueue pa_attention_mass for a workload on the device: add to mass
    (float32 [B, Hkv, max_context_len]) the softmax weight every cached token
    receives from the query rows w.q, given their log-sum-exps lse
    (float32 [B, n, Hq], as pa_attention wrote them)."""
    torch, b, types, device, raw_stream = _torch_and_binding()
    dev = device()
    st = raw_stream(dev) if stream is None else stream.cuda_stream
    B, rows = p.batch, p.batch * p.next_n * p.num_q_heads
    i32, f32 = torch.int32, torch.float32
    b.pa_attention_mass(p, decay, _need(w.q, "q", types.get(p.q_dtype), rows * p.head_dim_k, dev),
                        _need(w.k_pool, "k_pool", None, 1, dev),
                        _need(w.block_table, "block_table", i32, B * p.max_blocks_per_seq, dev),
                        _need(w.context_lens, "context_lens", i32, B, dev),
                        None if w.k_scale is None else _need(
                            w.k_scale, "k_scale", f32,
                            p.num_kv_heads * p.head_dim_k if p.k_scale_mode == b.PA_SCALE_CHANNEL else 1, dev),
                        _need(lse, "lse", f32, rows, dev),
                        _need(mass, "mass", f32, B * p.num_kv_heads * p.max_context_len, dev),
                        None if dev_error is None else _need(dev_error, "dev_error", i32, 1, dev), st)


def evict_workspace_bytes(p, budget: int) -> int:
    return binding().pa_evict_workspace_size(p, budget)


def evict(w, p, budget: int, mass, positions, history, mass_out, positions_out, history_out, lens_out, workspace, *,
          sinks: int = 0, recent: int = 0, stream=None) -> None:
    """Enqueue pa_evict for a workload on the device: keep, per request and kv
    head, the first `sinks` and newest `recent` tokens and those of the largest
    mass, `budget` in all, at the front of w's pools (moved in place).  mass
    float32 and positions int32 [B, Hkv, max_context_len], history int32
    [B, 2]; the *_out tensors may be the inputs themselves and lens_out
    w.context_lens."""
    torch, b, _, device, raw_stream = _torch_and_binding()
    dev = device()
    st = raw_stream(dev) if stream is None else stream.cuda_stream
    B, rows = p.batch, p.batch * p.num_kv_heads * p.max_context_len
    i32, f32 = torch.int32, torch.float32
    b.pa_evict(p, budget, sinks, recent, _need(mass, "mass", f32, rows, dev),
               _need(positions, "positions", i32, rows, dev), _need(history, "history", i32, 2 * B, dev),
               _need(w.block_table, "block_table", i32, B * p.max_blocks_per_seq, dev),
               _need(w.context_lens, "context_lens", i32, B, dev), _need(w.k_pool, "k_pool", None, 1, dev),
               None if w.v_pool is None else _need(w.v_pool, "v_pool", None, 1, dev),
               _need(mass_out, "mass_out", f32, rows, dev), _need(positions_out, "positions_out", i32, rows, dev),
               _need(history_out, "history_out", i32, 2 * B, dev), _need(lens_out, "lens_out", i32, B, dev),
               _need(workspace, "workspace", torch.uint8, 1, dev), workspace.numel(), st)
