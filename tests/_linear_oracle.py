"""Linear attention with a decay for each head, and rotary positions, in 64
bits: the recurrence token by token, the turn pair by pair.  Shares no code
with the library.

Beside the outputs, `attend` gives the sums of magnitudes that errors are
bounded by: the same recurrence over |q|, |k|, |v| and |S0|, where a rounding
of any product, weight or state by a factor of 1 + e moves a result by at most
e times that sum."""
import math

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2   # a rounding's most, relative


def attend(q, k, v, decay, state, scale, lens=None):
    """q, k [B, T, Hk, dk], v [B, T, H, dv], decay [B, T, H] or [H], state
    [N, H, dk, dv] or None; lens: of a packed batch's sequences (B = 1).
    (out, state, magnitudes of out, of state); rows past the last sequence NaN."""
    B, T, H, dv = v.shape
    group, dk = H // k.shape[2], k.shape[3]
    decay = decay.double().clamp(max=0.0)
    decay = decay if decay.dim() == 3 else decay.expand(B, T, H)
    spans = [(b, 0, T) for b in range(B)]
    if lens is not None:
        spans, at = [], 0
        for n in lens:
            spans.append((0, at, at + n))
            at += n
    out = torch.full((B, T, H, dv), math.nan, dtype=torch.float64, device=v.device)
    mag, finals, mags = out.clone(), [], []
    for n, (b, t0, t1) in enumerate(spans):
        S = torch.zeros(H, dk, dv, dtype=torch.float64, device=v.device) if state is None else state[n].double()
        A = S.abs()
        qs, ks = (x[b, t0:t1].double().repeat_interleave(group, 1) for x in (q, k))
        vs, es = v[b, t0:t1].double(), decay[b, t0:t1].exp()
        for t in range(t1 - t0):
            kv = ks[t][:, :, None] * vs[t][:, None]
            e = es[t][:, None, None]
            S = torch.where(e == 0, 0.0, S * e) + kv
            A = torch.where(e == 0, 0.0, A * e) + kv.abs()
            out[b, t0 + t] = scale * torch.einsum("hd,hdv->hv", qs[t], S)
            mag[b, t0 + t] = abs(scale) * torch.einsum("hd,hdv->hv", qs[t].abs(), A)
        finals.append(S)
        mags.append(A)
    return out, torch.stack(finals), mag, torch.stack(mags)


def turn(x, positions, frequencies, interleaved=False, amplitude=1.0, inverse=False):
    """x [T, heads, d] turned (rows with a negative position NaN)."""
    part = 2 * len(frequencies)
    y = x.double().clone()
    for i, f in enumerate(frequencies.tolist()):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + part // 2)
        t = positions.double()[:, None] * f
        c, s = amplitude * torch.cos(t), amplitude * torch.sin(t) * (-1 if inverse else 1)
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    y[positions < 0] = math.nan
    return y
