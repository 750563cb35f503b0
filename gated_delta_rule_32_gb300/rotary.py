"""Rotary positions of a step's queries and keys: the tensor-level call of
kda_rotary (include/kda.h), which says what it computes, and the usual
frequencies.

    freq, amplitude = rotary_frequencies(d, scaling="yarn", factor=4.0, trained=4096)
    plan = page_plan(...)
    q, k = rotary_embed(q, k, plan.positions, freq, amplitude=amplitude)
    cache_append(k, v, plan.runs, ...)
"""
from __future__ import annotations

import math

import torch
from torch.autograd.graph import increment_version

from .cache import _index, _need
from .linear import _DTYPES, _forward_only, _launch


def rotary_frequencies(part, base=10000.0, scaling=None, factor=1.0, trained=4096, fast=32.0,
                       slow=1.0, device="cuda"):
    """(frequencies, amplitude): float64 [part / 2] radians a token, and what
    queries and keys are multiplied by.  Pair i turns by base ** (-2 i / part).
    scaling, for contexts `factor` times as long as the `trained` tokens:

      None      as they are
      "linear"  every frequency divided by factor
      "ntk"     a larger base: base * factor ** (part / (part - 2)), which
                divides the slowest frequency by factor and keeps the fastest
      "yarn"    pairs with at least `fast` turns in the trained length are
                kept, those with at most `slow` divided by factor, a ramp in
                the pair's index between; amplitude 0.1 ln(factor) + 1
    """
    _need(part >= 2 and part % 2 == 0, "part must be even")
    _need(base > 0 and factor >= 1.0 and trained > 0, "base, factor or trained out of range")
    i = torch.arange(part // 2, dtype=torch.float64)
    amplitude = 1.0
    if scaling == "ntk":
        _need(part > 2, "ntk scaling needs more than one pair")
        base = base * factor ** (part / (part - 2))
    f = base ** (-2.0 * i / part)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        _need(fast > slow > 0 and base > 1, "yarn scaling needs fast > slow > 0 and base > 1")
        # the pair that makes n turns in the trained length has index at(n)

        def at(n):
            return part * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), part - 1)
        # (hi <= 0: not even the fastest pair makes more than `slow` turns)
        ramp = ((i - lo) / (hi - lo)).clamp(0.0, 1.0) if hi > lo else (i >= hi).double()
        f = f * (1 - ramp) + f / factor * ramp
        amplitude = 0.1 * math.log(factor) + 1.0
    else:
        _need(scaling in (None, "ntk"), "scaling must be None, 'linear', 'ntk' or 'yarn'")
    return f.to(device), amplitude


def _stride(x, name, dev, dtype, T, d):
    if x.dim() != 3 or x.dtype is not dtype or x.get_device() != dev or x.shape[0] != T or \
            x.shape[2] != d:
        raise ValueError("%s must be [T, heads, d] of one type on cuda:%d" % (name, dev))
    t, h, c = x.stride()
    H = x.shape[1]
    if T > 0 and (c != 1 or (h != d and H > 1)):
        raise ValueError("%s must have contiguous heads and channels" % name)
    return t if T > 1 else H * d


def rotary_embed(q, k, positions, frequencies, interleaved=False, amplitude=1.0, inverse=False,
                 inplace=False, stream=None):
    """q [T, Hq, d] and k [T, Hk, d] (or None), bfloat16 or float32 with any
    token stride, turned to positions (int32 [T]; a plan's are): (q, k), new
    contiguous tensors, or q and k themselves where `inplace`.  Rows with a
    negative position are left as they were (allocated).  frequencies: float64
    [part / 2], radians a token; part <= d channels of each head are turned, in
    pairs (i, i + part / 2) or, interleaved, (2 i, 2 i + 1).  `inverse` turns
    back, which is also the gradient's map: autograd has none of its own here, and
    tensors that want a gradient are refused where gradients are enabled."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rotary_embed(q, k, positions, frequencies, interleaved, amplitude, inverse,
                                inplace)
    _forward_only("rotary_embed", q, k, frequencies)
    dev = _index(q, "q")
    code = _DTYPES.get(q.dtype)
    _need(code is not None and q.dim() == 3, "q must be [T, heads, d], bfloat16 or float32")
    T, Hq, d = q.shape
    qs = _stride(q, "q", dev, q.dtype, T, d)
    if positions.dtype is not torch.int32 or positions.shape != (T,) or \
            not positions.is_contiguous() or positions.get_device() != dev:
        raise ValueError("positions must be a contiguous int32 tensor [T] on cuda:%d" % dev)
    if frequencies.dtype is not torch.float64 or frequencies.dim() != 1 or \
            not frequencies.is_contiguous() or frequencies.get_device() != dev:
        raise ValueError("frequencies must be a contiguous float64 tensor [part / 2] on cuda:%d" % dev)
    Hk, ks, kp = 0, 0, None
    if k is not None:
        ks = _stride(k, "k", dev, q.dtype, T, d)
        Hk, kp = k.shape[1], k.data_ptr()
    if inplace:
        qo, ko, qos, kos = q, k, qs, ks
    else:
        qo, qos, kos = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device), Hq * d, Hk * d
        ko = None if k is None else torch.empty((T, Hk, d), dtype=q.dtype, device=q.device)
    _launch(dev, "kda_rotary", q.data_ptr(), qs, qo.data_ptr(), qos, kp, ks,
           None if ko is None else ko.data_ptr(), kos, positions.data_ptr(),
           frequencies.data_ptr(), T, Hq, Hk, d, 2 * frequencies.numel(), amplitude, interleaved,
           inverse, code)
    if inplace:
        increment_version(q)
        if k is not None:
            increment_version(k)
    return qo, ko
