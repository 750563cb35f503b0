"""Linear attention with a decay for each head: tensor-level calls of
kda_linear_fwd and kda_linear_decode (include/kda.h), which say what each
computes.

    S_t = exp(a_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   a_t = min(log_decay_t, 0)

A token with a log_decay below -104 (-inf, say) forgets the state before it,
whatever that holds.

A prompt, then tokens::

    out, state = linear_attend(q, k, v, log_decay, scale=scale)
    out = linear_decode(q1, k1, v1, log_decay1, state, scale=scale)     # state in place

q and k are [B, T, Hk, dk], v [B, T, H, dv], bfloat16 or float32, H a multiple
of Hk (each head of q and k serves H / Hk heads of v); log_decay is float32,
[B, T, H] or one value for each head, [H].  q, k, v and log_decay may be views
of a projection's output: any distance between tokens, the same for all rows.
Nothing here computes: tensors are checked, outputs allocated and the library
called, on the current stream of the tensors' device, or on `stream`, which
then also owns the outputs' memory.  Errors that the host can see raise
ValueError or KdaError before anything is queued.  No call has a gradient: where
one would be lost (gradients are enabled and a tensor wants one) it is refused,
and autograd learns which tensors have changed in place.
"""
from __future__ import annotations

import functools

import torch
from torch.autograd.graph import increment_version

from . import kda
from .cache import _call, _index, _need
from .kda import KDA_BF16, KDA_F32, KDA_OK, KdaError

_DTYPES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}


# (messages are put together only where they are raised: a decode step's calls are short)

def _rows(x, name, dev, dtype):
    """Checks a [B, T, heads, d] tensor whose heads and channels are contiguous
    and whose rows follow each other at one distance: that distance."""
    if x.dim() != 4 or x.dtype is not dtype or x.get_device() != dev:
        raise ValueError("%s must be [B, T, heads, d] of one type (bfloat16 or float32) on cuda:%d"
                         % (name, dev))
    B, T, H, d = x.shape
    b, t, h, c = x.stride()
    if B * T == 0:
        return H * d
    if (c != 1 and d > 1) or (h != d and H > 1):
        raise ValueError("%s must have contiguous heads and channels" % name)
    if B > 1 and T > 1 and b != T * t:
        raise ValueError("%s must have its rows at one distance" % name)
    return t if T > 1 else b if B > 1 else H * d


def _decay(a, B, T, H, dev):
    if a.dtype is not torch.float32 or a.get_device() != dev:
        raise ValueError("log_decay must be a float32 tensor on cuda:%d" % dev)
    if a.dim() == 1:
        _need(a.shape[0] == H and (H == 1 or a.stride(0) == 1), "log_decay must be [H], contiguous")
        return 0
    _need(a.shape == (B, T, H), "log_decay must be [B, T, H] or [H]")
    b, t, h = a.stride()
    if B * T == 0:
        return H
    _need(h == 1 or H == 1, "log_decay must have contiguous heads")
    _need(B == 1 or T == 1 or b == T * t, "log_decay must have its rows at one distance")
    return t if T > 1 else b if B > 1 else H


def _forward_only(name, *tensors):
    if torch.is_grad_enabled():
        for x in tensors:
            if x is not None and x.requires_grad:
                raise ValueError("%s has no gradient, and a tensor wants one: call it under "
                                 "torch.no_grad(), or detach the tensor" % name)


def _state(x, name, shape, dev):
    if x.dtype is not torch.float32 or x.shape != shape or not x.is_contiguous() or \
            x.get_device() != dev:
        raise ValueError("%s must be a contiguous float32 tensor %s on cuda:%d"
                         % (name, list(shape), dev))


def _shapes(q, k, v, log_decay):
    dev = _index(q, "q")
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    _need(code is not None, "q must be bfloat16 or float32")
    qs, ks, vs = _rows(q, "q", dev, dtype), _rows(k, "k", dev, dtype), _rows(v, "v", dev, dtype)
    B, T, Hk, dk = q.shape
    Bv, Tv, H, dv = v.shape
    _need(k.shape == q.shape and Bv == B and Tv == T and Hk > 0 and H % Hk == 0,
          "q and k must be [B, T, Hk, dk], v [B, T, H, dv], H a multiple of Hk")
    return dev, code, qs, ks, vs, _decay(log_decay, B, T, H, dev), B, T, H, Hk, dk, dv


@functools.lru_cache(maxsize=256)
def _workspace_bytes(dev, N, T, H, dk, dv, code, packed):
    with torch.cuda.device(dev):
        return kda.kda_linear_workspace_bytes(N, T, H, dk, dv, code, packed)


def linear_attend(q, k, v, log_decay, init_state=None, cu_seqlens=None, scale=1.0, dev_status=None,
                  stream=None):
    """Whole prompts: (out [B, T, H, dv], final_state [N, H, dk, dv] float32).
    Packed batches: cu_seqlens (int32 [N + 1], a plan's is one) with B = 1; rows
    past the last sequence are left as they were allocated.  init_state
    [N, H, dk, dv] defaults to zero.  bfloat16 with heads of 64 and 128 runs on
    the tensor cores in chunks of 128 tokens of a sequence, where weights and what
    queries read of the state are rounded to bfloat16, and where a NaN or an
    infinity in v reaches all rows of its chunk, those before it too; other types
    and sizes run token by token in float32."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_attend(q, k, v, log_decay, init_state, cu_seqlens, scale, dev_status)
    _forward_only("linear_attend", q, k, v, log_decay, init_state)
    dev, code, qs, ks, vs, ds, B, T, H, Hk, dk, dv = _shapes(q, k, v, log_decay)
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or B != 1 or \
                cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous() or \
                cu_seqlens.get_device() != dev:
            raise ValueError("cu_seqlens must be a contiguous int32 tensor [N + 1] on cuda:%d, "
                             "with B = 1" % dev)
        N = cu_seqlens.numel() - 1
    if init_state is not None:
        _state(init_state, "init_state", (N, H, dk, dv), dev)
    device = q.device
    out = torch.empty((B, T, H, dv), dtype=q.dtype, device=device)
    final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=device)
    nb = _workspace_bytes(dev, N, T, H, dk, dv, code, int(cu_seqlens is not None))
    ws = torch.empty(nb, dtype=torch.uint8, device=device) if nb else None
    _call(dev, dev_status, "kda_linear_fwd", q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
          log_decay.data_ptr(), ds, None if init_state is None else init_state.data_ptr(),
          out.data_ptr(), final.data_ptr(), N, T, H, Hk, dk, dv,
          None if cu_seqlens is None else cu_seqlens.data_ptr(), code, scale,
          None if ws is None else ws.data_ptr(), nb)
    return out, final


def linear_decode(q, k, v, log_decay, state, scale=1.0, stream=None):
    """T tokens of each of N sequences (q [N, T, Hk, dk], v [N, T, H, dv]), token
    by token: out [N, T, H, dv]; state [N, H, dk, dv] float32 is updated in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_decode(q, k, v, log_decay, state, scale)
    _forward_only("linear_decode", q, k, v, log_decay, state)
    dev, code, qs, ks, vs, ds, N, T, H, Hk, dk, dv = _shapes(q, k, v, log_decay)
    _state(state, "state", (N, H, dk, dv), dev)
    out = torch.empty((N, T, H, dv), dtype=q.dtype, device=q.device)
    _launch(dev, "kda_linear_decode", q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
           log_decay.data_ptr(), ds, state.data_ptr(), out.data_ptr(), N, T, H, Hk, dk, dv, code,
           scale)
    increment_version(state)
    return out


def _launch(dev, name, *args):
    """The library's function `name`(*args, stream) with device `dev` and its
    current stream."""
    fn = getattr(kda._lib or kda.load(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != KDA_OK:
        raise KdaError(name, rc)
