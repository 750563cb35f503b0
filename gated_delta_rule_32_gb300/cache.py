"""The paged 8-bit cache of a hybrid model's attention layers: tensor-level
calls of kda_page_plan, kda_page_release, kda_cache_append and
kda_cache_attn (include/kda.h), which say what each computes.

A step of a serving loop::

    plan = page_plan(new_lens, ctx_lens, block_table, free_pages, free_count, T, page)
    cache_append(k, v, plan.runs, k_codes, v_codes, k_scale, v_scale)
    out, lse = cache_attend(q, plan.cu_seqlens, plan.kv_lens, block_table,
                            k_codes, v_codes, k_scale, v_scale, max_new=max_new)
    ctx_lens, free_count = plan.kv_lens, plan.free_count

plan.cu_seqlens is also what the packed gated delta rule forward takes.  The
plan serves every layer of the step.  Nothing here computes: tensors are
checked, outputs allocated and the library called, on the current stream of
the tensors' device, or on `stream`, which then also owns the outputs' memory
(record_stream() them where another stream uses them).  Errors that the host can see raise
ValueError or KdaError before anything is queued; those that only the device
can see go to `dev_status` (an int32 CUDA tensor of one element, set by every
call it is given to: one for each call whose status is wanted).  Without it
they go unnoticed: after a plan that did not fit, or for a request with more
than max_new tokens, rows of the attention's output are never written.
"""
from __future__ import annotations

import functools
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


def _index(x, name):
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return x.get_device()


def _ints(dev, names, *tensors):
    for i, x in enumerate(tensors):
        if x.dtype is not torch.int32 or not x.is_contiguous() or x.get_device() != dev:
            raise ValueError("%s must be a contiguous int32 tensor on cuda:%d"
                             % (names.split()[i], dev))


def _call(dev, dev_status, name, *args):
    """The library's function `name`(*args, dev_status, stream) with device
    `dev` and its current stream.  (A decode step's calls are short: no
    context manager where the device is current, no Stream object.)"""
    fn = getattr(kda._lib or kda.load(), name)
    status = None
    if dev_status is not None:
        if dev_status.dtype is not torch.int32 or dev_status.get_device() != dev or \
                dev_status.numel() < 1:
            raise ValueError("dev_status must be an int32 tensor of one element on cuda:%d" % dev)
        status = dev_status.data_ptr()
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, status, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, status, stream)
    if rc != KDA_OK:
        raise KdaError(name, rc)


def _pool(dev, k_codes, v_codes, k_scale, v_scale):
    """(num_pages, Hkv, page, d, code) of one layer's cache."""
    shape, dtype = k_codes.shape, k_codes.dtype
    code = _CODES.get(dtype)
    _need(len(shape) == 4 and v_codes.shape == shape, "codes must be [pages, Hkv, page, d]")
    _need(code is not None and v_codes.dtype is dtype, "codes must be int8 or float8_e4m3fn")
    _need(k_codes.is_contiguous() and v_codes.is_contiguous() and v_codes.get_device() == dev,
          "codes must be contiguous, on one device")
    scales = shape[:2]
    for x in (k_scale, v_scale):
        if x.dtype is not torch.float32 or x.shape != scales or not x.is_contiguous() or \
                x.get_device() != dev:
            raise ValueError("scales must be contiguous float32 [pages, Hkv]")
    return (*shape, code)


def _stride(x, name, dev):
    """Checks a [T, H, d] bf16 tensor whose heads and channels are contiguous; its token stride."""
    _need(x.dim() == 3 and x.dtype is torch.bfloat16 and x.get_device() == dev,
          "%s must be a bfloat16 tensor [T, heads, d] on cuda:%d" % (name, dev))
    T, H, d = x.shape
    t, h, c = x.stride()
    _need(T == 0 or (c == 1 and (h == d or H == 1)),
          "%s must have contiguous heads and channels" % name)
    return t if T > 1 else H * d


def page_plan(new_lens, ctx_lens, block_table, free_pages, free_count, T, page, dev_status=None,
              stream=None):
    """Bookkeeping of a step in which request r brings new_lens[r] tokens (at
    most T in all) to its ctx_lens[r] cached ones: a PagePlan.  New page
    numbers come from the top of the stack free_pages[: free_count] and are
    entered into block_table [R, max_pages] in place.  free_pages has room for
    every page of the pool: its length is the pool's size."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return page_plan(new_lens, ctx_lens, block_table, free_pages, free_count, T, page,
                             dev_status)
    dev = _index(new_lens, "new_lens")
    _ints(dev, "new_lens ctx_lens block_table free_pages free_count", new_lens, ctx_lens,
          block_table, free_pages, free_count)
    R = new_lens.numel()
    _need(ctx_lens.numel() == R and block_table.dim() == 2 and block_table.shape[0] == R,
          "ctx_lens must be [R] and block_table [R, max_pages]")
    n = (kda._lib or kda.load()).kda_page_runs(R, T, page)
    _need(n > 0, "no requests, a negative T or a page size that is not 16, 32, 64 or 128")
    kw = {"dtype": torch.int32, "device": new_lens.device}
    runs = torch.empty((n, 4), **kw)
    # (one allocation for the others, pieces of it)
    cu, kv, slots, positions, left = torch.empty(2 * R + 2 * T + 2, **kw).unsafe_split_with_sizes(
        (R + 1, R, T, T, 1))
    plan = PagePlan(cu, kv, slots, positions, runs, left)
    _call(dev, dev_status, "kda_page_plan", new_lens.data_ptr(), ctx_lens.data_ptr(), R, T,
          page, block_table.data_ptr(), block_table.shape[1], free_pages.data_ptr(),
          free_count.data_ptr(), free_pages.numel(), cu.data_ptr(), kv.data_ptr(),
          slots.data_ptr(), positions.data_ptr(), runs.data_ptr(), left.data_ptr())
    return plan


def page_release(release, kv_lens, block_table, free_pages, free_count, page, dev_status=None,
                 stream=None):
    """Requests with release[r] != 0 give their pages back to the stack; all
    tensors but `release` are updated in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return page_release(release, kv_lens, block_table, free_pages, free_count, page,
                                dev_status)
    dev = _index(release, "release")
    _ints(dev, "release kv_lens block_table free_pages free_count", release, kv_lens, block_table,
          free_pages, free_count)
    R = release.numel()
    _need(kv_lens.numel() == R and block_table.dim() == 2 and block_table.shape[0] == R,
          "kv_lens must be [R] and block_table [R, max_pages]")
    _call(dev, dev_status, "kda_page_release", release.data_ptr(), R, page,
          kv_lens.data_ptr(), block_table.data_ptr(), block_table.shape[1], free_pages.data_ptr(),
          free_count.data_ptr(), free_pages.numel())


def cache_append(k, v, runs, k_codes, v_codes, k_scale, v_scale, dev_status=None, stream=None):
    """Quantises a step's keys and values (bf16 [T, Hkv, d], any token stride)
    into the cache by a plan's runs; codes and scales are updated in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_append(k, v, runs, k_codes, v_codes, k_scale, v_scale, dev_status)
    dev = _index(k_codes, "k_codes")
    num, H, page, d, code = _pool(dev, k_codes, v_codes, k_scale, v_scale)
    ks, vs = _stride(k, "k", dev), _stride(v, "v", dev)
    T = k.shape[0]
    _need(k.shape == v.shape and k.shape[1] == H and k.shape[2] == d, "k and v must be [T, Hkv, d]")
    _ints(dev, "runs", runs)
    _need(runs.dim() == 2 and runs.shape[1] == 4, "runs must be [n, 4]")
    _call(dev, dev_status, "kda_cache_append", k.data_ptr(), v.data_ptr(), ks, vs, T,
          runs.data_ptr(), runs.shape[0], k_codes.data_ptr(), v_codes.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), num, page, H, d, code)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(dev, R, T, max_new, Hq, Hkv, d):
    with torch.cuda.device(dev):
        return kda.kda_cache_attn_workspace_bytes(R, T, max_new, Hq, Hkv, d)


def cache_attend(q, cu_seqlens, kv_lens, block_table, k_codes, v_codes, k_scale, v_scale,
                 scale=None, max_new=None, dev_status=None, stream=None):
    """Causal attention of a step's queries (bf16 [T, Hq, d], any token
    stride) over the cache: (out bf16 [T, Hq, d], lse fp32 [T, Hq]); rows past
    cu_seqlens[R] are left as they were allocated.  `scale`
    defaults to d ** -0.5; max_new is the most new tokens any request has.  Its
    default, T, is always right but runs kernels for that many rows: a decode step
    of 64 requests takes 155 us so, 139 with max_new=1, 2 long ones 83 and 78."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_attend(q, cu_seqlens, kv_lens, block_table, k_codes, v_codes, k_scale,
                                v_scale, scale, max_new, dev_status)
    dev = _index(k_codes, "k_codes")
    num, Hkv, page, d, code = _pool(dev, k_codes, v_codes, k_scale, v_scale)
    qs = _stride(q, "q", dev)
    T, Hq, dq = q.shape
    _need(dq == d and Hq % Hkv == 0, "q must be [T, Hq, d], Hq a multiple of the cache's heads")
    _ints(dev, "cu_seqlens kv_lens block_table", cu_seqlens, kv_lens, block_table)
    R = kv_lens.numel()
    _need(cu_seqlens.numel() == R + 1 and block_table.dim() == 2 and block_table.shape[0] == R,
          "cu_seqlens must be [R + 1] and block_table [R, max_pages]")
    if max_new is None:
        max_new = T
    if scale is None:
        scale = d ** -0.5
    device = k_codes.device
    out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=device)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=device)
    nb = _workspace_bytes(dev, R, T, max_new, Hq, Hkv, d)
    ws = torch.empty(nb, dtype=torch.uint8, device=device)
    _call(dev, dev_status, "kda_cache_attn", q.data_ptr(), qs, cu_seqlens.data_ptr(),
          kv_lens.data_ptr(), block_table.data_ptr(), block_table.shape[1], k_codes.data_ptr(),
          v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), out.data_ptr(),
          lse.data_ptr(), R, T, max_new, Hq, Hkv, d, num, page, code, scale,
          ws.data_ptr() if nb else None, nb)
    return out, lse
