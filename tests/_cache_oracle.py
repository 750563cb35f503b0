"""The paged cache's operators in plain Python and 64-bit torch on the CPU:
the page plan step by step, the append element by element from its formula,
the attention as a softmax over gathered keys.  Shares no code with the
library."""
import math

import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def plan(new, ctx, table, stack, T, page, num_pages):
    """(cu, kv, slots, positions, runs, left, table): lists; `stack` is the
    free pages, top last; table a list of lists."""
    table, stack = [list(r) for r in table], list(stack)
    cu, kv, slots, positions, runs = [0], [], [], [], []
    for r, (n, c) in enumerate(zip(new, ctx)):
        for col in range(-(-c // page), -(-(c + n) // page)):
            table[r][col] = stack.pop()
        p = c
        while p < c + n:
            m = min(page - p % page, c + n - p)
            pg = table[r][p // page]
            runs.append([cu[-1] + p - c, m, pg, p % page])
            slots += [pg * page + (p + i) % page for i in range(m)]
            positions += list(range(p, p + m))
            p += m
        cu.append(cu[-1] + n)
        kv.append(c + n)
    most = max(1, min(T, T // page + 2 * len(new)))
    assert len(runs) <= most
    runs += [[0, 0, 0, 0]] * (most - len(runs))
    slots += [-1] * (T - len(slots))
    positions += [-1] * (T - len(positions))
    return cu, kv, slots, positions, runs, len(stack), table


def to_grid(x, dtype):
    """Nearest code of each value (as its value), ties to even."""
    if dtype == torch.int8:
        return x.round()
    a = x.abs()
    e = (torch.frexp(a).exponent - 1).clamp(min=-6)
    step = torch.exp2((e - 3).double())
    return (a / step).round() * step * x.sign()


def append(x, runs, codes, scale):
    """x [T, H, d], codes [pages, H, page, d], scale [pages, H]: new codes as
    values and scales, both in 64 bits."""
    dtype, top = codes.dtype, TOP[codes.dtype]
    codes, scale = codes.double(), scale.double()
    for row, count, page, off in runs:
        if not count:
            continue
        xs = x[row:row + count].double().transpose(0, 1)
        a0 = scale[page] if off else torch.zeros_like(scale[page])
        a1 = torch.maximum(a0, xs.abs().amax((1, 2)))
        div = torch.where(a1 > 0, a1, torch.ones_like(a1))[:, None, None]
        codes[page, :, :off] = to_grid(codes[page, :, :off] * a0[:, None, None] / div, dtype)
        codes[page, :, off:off + count] = to_grid(xs * top / div, dtype)
        scale[page] = a1
    return codes, scale


def attend(q, cu, kv, table, kc, vc, ks, vs, scale):
    """out, lse in 64 bits, and bounds on their error.

    The kernels may round, beside the output to bf16 (8 bits: half an ulp is
    up to 2^-8 relative): each weight to 11 bits (2^-11 relative, or 2^-25 absolute of
    the largest weight times the largest value scale), and fp32 sums of
    scores (2^-18 of the sum of magnitudes covers a chain of 128 products).
    A score error e changes a weight by a factor exp(e), the output by at
    most 2 e times the largest value."""
    T, HQ, D = q.shape
    H, page = kc.shape[1], kc.shape[2]
    G, top = HQ // H, TOP[kc.dtype]
    out = torch.zeros(T, HQ, D, dtype=torch.float64)
    lse = torch.full((T, HQ), -math.inf, dtype=torch.float64)
    tol_o = torch.zeros(T, HQ, 1, dtype=torch.float64)
    tol_l = torch.zeros(T, HQ, dtype=torch.float64)
    for r in range(len(kv)):
        a, b = cu[r], cu[r + 1]
        n, L = b - a, kv[r]
        if n == 0 or L == 0:
            continue
        pages = torch.tensor(table[r][:-(-L // page)], dtype=torch.long)
        for h in range(H):
            # (bytes are indexed: not every index operation takes 8-bit floats)
            k, v = ((x.view(torch.uint8)[pages, h].view(x.dtype).double()
                     * (s[pages, h].double() / top)[:, None, None]).reshape(-1, D)[:L]
                    for x, s in ((kc, ks), (vc, vs)))
            big = vs[pages, h].double().max()
            x = q[a:b, h * G:(h + 1) * G].double()                   # [n, G, D]
            s = scale * torch.einsum("ngd,ld->ngl", x, k)
            mag = (abs(scale) * torch.einsum("ngd,ld->ngl", x.abs(), k.abs())).amax(-1)
            seen = (L - n + 1 + torch.arange(n))[:, None]
            s = torch.where((torch.arange(L)[None] < seen)[:, None], s, -math.inf)
            m = s.amax(-1, keepdim=True)
            w = torch.exp(s - torch.where(m.isfinite(), m, 0.0))
            l = w.sum(-1, keepdim=True)
            o = torch.where(l > 0, (w / torch.where(l > 0, l, 1.0)) @ v, 0.0)
            out[a:b, h * G:(h + 1) * G] = o
            lse[a:b, h * G:(h + 1) * G] = (m + l.log())[..., 0]
            e = mag * 2.0 ** -18
            tol_o[a:b, h * G:(h + 1) * G] = ((2 * e + 2.0 ** -11 + L * 2.0 ** -25) * big)[..., None]
            tol_l[a:b, h * G:(h + 1) * G] = e + 2.0 ** -18
    return out, lse, tol_o + out.abs() * 2.0 ** -8, tol_l
