"""Attention over the paged 8-bit cache in 64 bits, with error bounds that
follow what each row sums.  Shares no code with the library.

The kernels may err, beside the output's rounding to bf16 (half a unit, 2^-8 of
the value at most),

  * in a score by 2^-18 of the sum of its products' magnitudes (fp32, and f16
    queries), at most e in a row: weights then err by 2 e, numerator and sum
    of weights together;
  * in a weight by 2^-11 of it (f16);
  * in a small weight by 2^-25 of the row's reference, a score not above its
    largest, and of a power of two below twice the largest value scale that the
    row sees: in a token's value by 2^-24 p big |c|, p the row's largest
    normalised weight, big that scale, c the token's code over the top one;
  * in fp32 sums by 2^-12 (runs of 65536 tokens, 2^-24 for each addition of 16).

The relative errors d of the weights act as d |o| where they are alike and,
where they are independent with a variance of d^2 / 3, as 6 deviations of
sum_j p_j d_j v_j: d (6 / sqrt 3) sqrt(sum_j p_j^2 v_j^2).  The same way the
small weights' errors add up to 2^-24 p big (|sum_j c_j| + (6 / sqrt 3)
sqrt(sum_j c_j^2))."""
import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def attend(q, cu, kv, table, kc, vc, ks, vs, scale):
    """out, lse and the bounds on their errors (CPU, 64 bits); computed on the GPU."""
    T, HQ, D = q.shape
    H, G, page, top = kc.shape[1], HQ // kc.shape[1], kc.shape[2], TOP[kc.dtype]
    dev = "cuda"
    out = torch.zeros(T, HQ, D, dtype=torch.float64)
    lse = torch.full((T, HQ), -math.inf, dtype=torch.float64)
    tol_o = torch.zeros(T, HQ, D, dtype=torch.float64)
    tol_l = torch.zeros(T, HQ, dtype=torch.float64)
    qd = q.to(dev).double()
    for r in range(len(kv)):
        a, b, L = cu[r], cu[r + 1], kv[r]
        n = b - a
        if n == 0 or L == 0:
            continue
        pages = torch.tensor(table[r][:-(-L // page)], dtype=torch.long)
        seen = (L - n + 1 + torch.arange(n, device=dev)).clamp(min=0)
        hidden = torch.arange(L, device=dev)[None] >= seen[:, None]
        for h in range(H):
            k, v = ((x.view(torch.uint8)[pages, h].view(x.dtype).float().to(dev).double()
                     * (s[pages, h].to(dev).double() / top)[:, None, None]).reshape(-1, D)[:L]
                    for x, s in ((kc, ks), (vc, vs)))
            sc = vs[pages, h].to(dev).double().repeat_interleave(page)[:L]
            last = (seen - 1).clamp(min=0)
            big = torch.cummax(sc, 0).values[last]
            c = v / torch.where(sc > 0, sc, 1.0)[:, None]
            codes = c.cumsum(0)[last].abs() + 6 / math.sqrt(3) * c.square().cumsum(0)[last].sqrt()
            x = qd[a:b, h * G:(h + 1) * G]                               # [n, G, D]
            s = (scale * (x @ k.T)).masked_fill(hidden[:, None], -math.inf)
            mag = (abs(scale) * (x.abs() @ k.abs().T)).masked_fill(hidden[:, None], 0.0).amax(-1)
            m = s.amax(-1, keepdim=True)
            w = torch.exp(s - torch.where(m.isfinite(), m, 0.0))
            l = w.sum(-1, keepdim=True)
            p = w / torch.where(l > 0, l, 1.0)
            o = p @ v
            deep = (p.square() @ v.square()).sqrt()
            e = (mag * 2.0 ** -18)[..., None]
            small = 2.0 ** -24 * p.amax(-1, keepdim=True) * (big[:, None] * codes)[:, None]
            d = 2 * e + 2.0 ** -11
            t = (2.0 ** -8 + 2.0 ** -12 + d) * o.abs() + \
                (2.0 ** -12 + d * 6 / math.sqrt(3)) * deep + small
            at = slice(h * G, (h + 1) * G)
            out[a:b, at], lse[a:b, at] = o.cpu(), (m + l.log())[..., 0].cpu()
            tol_o[a:b, at], tol_l[a:b, at] = t.cpu(), (e[..., 0] + 2.0 ** -18).cpu()
    return out, lse, tol_o, tol_l
