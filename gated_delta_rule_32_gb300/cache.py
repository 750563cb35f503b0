"""The paged 8-bit cache of a hybrid model's attention layers: tensor-level
calls of kda_page_plan, kda_page_release, kda_cache_append and
kda_cache_attn (include/kda.h), which say what each computes.

A step of a serving loop::

    plan = page_plan(new_lens, ctx_lens, block_table, free_pages, free_count, T, page)
    cache_append(k, v, plan.runs, k_codes, v_codes, k_scale, v_scale)
    out, lse = cache_attend(q, plan.cu_seqlens, plan.kv_lens, block_table,
                            k_codes, v_codes, k_scale, v_scale)
    ctx_lens, free_count = plan.kv_lens, plan.free_count

plan.cu_seqlens is also what the packed gated delta rule forward takes.  The
plan serves every layer of the step.  Nothing here computes: tensors are
checked, outputs allocated and the library called, on the current stream of
the tensors' device (or `stream`).  Errors that the host can see raise
ValueError or KdaError before anything is queued; those that only the device
can see go to `dev_status` (an int32 CUDA tensor of one element) if given.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import kda
from .kda import KDA_E4M3, KDA_I8, KDA_OK, KdaError

_CODES = {torch.int8: KDA_I8, torch.float8_e4m3fn: KDA_E4M3}


class PagePlan(NamedTuple):
    """One step's bookkeeping (all int32 CUDA tensors)."""
    cu_seqlens: torch.Tensor   # [R + 1] packed offsets of the new tokens
    kv_lens: torch.Tensor      # [R] cached and new tokens
    slots: torch.Tensor        # [T] page * page_size + offset of each new token
    positions: torch.Tensor    # [T] position of each new token in its request
    runs: torch.Tensor         # [runs, 4] row, tokens, page, offset
    free_count: torch.Tensor   # [1] pages left on the stack


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(dev, **tensors):
    for name, x in tensors.items():
        if x.dtype != torch.int32 or not x.is_contiguous() or x.device != dev:
            raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, dev))


def _device(x, name):
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    return dev


def _call(dev, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    with torch.cuda.device(dev):
        rc = fn(*args, (stream or torch.cuda.current_stream(dev)).cuda_stream)
    if rc != KDA_OK:
        raise KdaError(fn.__name__, rc)


def _pool(dev, k_codes, v_codes, k_scale, v_scale):
    """(num_pages, Hkv, page, d, code) of one layer's cache."""
    _need(k_codes.dim() == 4 and k_codes.shape == v_codes.shape, "codes must be [pages, Hkv, page, d]")
    _need(k_codes.dtype in _CODES and v_codes.dtype == k_codes.dtype,
          "codes must be int8 or float8_e4m3fn")
    num, H, page, d = k_codes.shape
    for x in (k_codes, v_codes):
        _need(x.is_contiguous() and x.device == dev, "codes must be contiguous, on one device")
    for x in (k_scale, v_scale):
        _need(x.dtype == torch.float32 and x.shape == (num, H) and x.is_contiguous()
              and x.device == dev, "scales must be contiguous float32 [pages, Hkv]")
    return num, H, page, d, _CODES[k_codes.dtype]


def _rows(x, name, dev):
    """Checks a [T, H, d] bf16 tensor whose heads and channels are contiguous; its token stride."""
    _need(x.dim() == 3 and x.dtype == torch.bfloat16 and x.device == dev,
          "%s must be a bfloat16 tensor [T, heads, d] on %s" % (name, dev))
    T, H, d = x.shape
    _need(T == 0 or (x.stride(2) == 1 and (x.stride(1) == d or H == 1)),
          "%s must have contiguous heads and channels" % name)
    return x.stride(0) if T > 1 else H * d


def page_plan(new_lens, ctx_lens, block_table, free_pages, free_count, T, page, dev_status=None,
              stream=None):
    """Bookkeeping of a step in which request r brings new_lens[r] tokens (at
    most T in all) to its ctx_lens[r] cached ones: a PagePlan.  New page
    numbers come from the top of the stack free_pages[: free_count] and are
    entered into block_table [R, max_pages] in place."""
    dev = _device(new_lens, "new_lens")
    _ints(dev, new_lens=new_lens, ctx_lens=ctx_lens, block_table=block_table,
          free_pages=free_pages, free_count=free_count)
    R = new_lens.numel()
    _need(ctx_lens.numel() == R and block_table.dim() == 2 and block_table.shape[0] == R,
          "ctx_lens must be [R] and block_table [R, max_pages]")
    n = kda.kda_page_runs(R, T, page)
    _need(n > 0, "no requests, a negative T or a page size that is not 16, 32, 64 or 128")
    sizes = [4 * n, R + 1, R, T, T, 1]
    runs, cu, kv, slots, positions, left = torch.empty(
        sum(sizes), dtype=torch.int32, device=dev).split_with_sizes(sizes)
    _call(dev, stream, kda.kda_page_plan, new_lens, ctx_lens, R, T, page, block_table,
          block_table.shape[1], free_pages, free_count, free_pages.numel(), cu, kv, slots,
          positions, runs, left, dev_status)
    return PagePlan(cu, kv, slots, positions, runs.view(n, 4), left)


def page_release(release, kv_lens, block_table, free_pages, free_count, page, dev_status=None,
                 stream=None):
    """Requests with release[r] != 0 give their pages back to the stack; all
    tensors but `release` are updated in place."""
    dev = _device(release, "release")
    _ints(dev, release=release, kv_lens=kv_lens, block_table=block_table, free_pages=free_pages,
          free_count=free_count)
    R = release.numel()
    _need(kv_lens.numel() == R and block_table.dim() == 2 and block_table.shape[0] == R,
          "kv_lens must be [R] and block_table [R, max_pages]")
    _call(dev, stream, kda.kda_page_release, release, R, page, kv_lens, block_table,
          block_table.shape[1], free_pages, free_count, free_pages.numel(), dev_status)


def cache_append(k, v, runs, k_codes, v_codes, k_scale, v_scale, dev_status=None, stream=None):
    """Quantises a step's keys and values (bf16 [T, Hkv, d], any token stride)
    into the cache by a plan's runs; codes and scales are updated in place."""
    dev = _device(k_codes, "k_codes")
    num, H, page, d, code = _pool(dev, k_codes, v_codes, k_scale, v_scale)
    ks, vs = _rows(k, "k", dev), _rows(v, "v", dev)
    _need(k.shape == v.shape and k.shape[1:] == (H, d), "k and v must be [T, Hkv, d]")
    _ints(dev, runs=runs)
    _need(runs.dim() == 2 and runs.shape[1] == 4, "runs must be [n, 4]")
    _call(dev, stream, kda.kda_cache_append, k, v, ks, vs, k.shape[0], runs, runs.shape[0],
          k_codes, v_codes, k_scale, v_scale, num, page, H, d, code, dev_status)


def cache_attend(q, cu_seqlens, kv_lens, block_table, k_codes, v_codes, k_scale, v_scale,
                 scale=None, max_new=None, dev_status=None, stream=None):
    """Causal attention of a step's queries (bf16 [T, Hq, d], any token
    stride) over the cache: (out bf16 [T, Hq, d], lse fp32 [T, Hq]).  `scale`
    defaults to d ** -0.5; max_new is the most new tokens any request has
    (default: T)."""
    dev = _device(k_codes, "k_codes")
    num, Hkv, page, d, code = _pool(dev, k_codes, v_codes, k_scale, v_scale)
    qs = _rows(q, "q", dev)
    T, Hq, dq = q.shape
    _need(dq == d and Hq % Hkv == 0, "q must be [T, Hq, d], Hq a multiple of the cache's heads")
    _ints(dev, cu_seqlens=cu_seqlens, kv_lens=kv_lens, block_table=block_table)
    R = kv_lens.numel()
    _need(cu_seqlens.numel() == R + 1 and block_table.dim() == 2 and block_table.shape[0] == R,
          "cu_seqlens must be [R + 1] and block_table [R, max_pages]")
    if max_new is None:
        max_new = T
    if scale is None:
        scale = d ** -0.5
    out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        nb = kda.kda_cache_attn_workspace_bytes(R, T, max_new, Hq, Hkv, d)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    if ws is not None and stream is not None:
        ws.record_stream(stream)  # (freed for reuse only after the work on `stream`)
    _call(dev, stream, kda.kda_cache_attn, q, qs, cu_seqlens, kv_lens, block_table,
          block_table.shape[1], k_codes, v_codes, k_scale, v_scale, out, lse, R, T, max_new, Hq,
          Hkv, d, num, page, code, scale, ws, nb, dev_status)
    return out, lse
