"""Cases that time the paged 8-bit cache's operators: the page plan, the append and the attention over the cache.

A hybrid model keeps a fixed-size state for its gated delta rule layers and a
growing cache of keys and values for its attention layers.  The three
operators here serve the second kind.  `run` computes them in plain 32-bit
torch operations where `own` is false and calls the library where it is true;
`exact` states them once more in 64 bits.

A code c of a page and head with scale s stands for the value c * s / 127
(int8) or c * s / 448 (e4m3): s is the largest magnitude the page and head
hold, the value of the largest code.
"""
import math
import random

import torch

own = False

TOP = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# --------------------------------------------------------------------------
# cases

def listed():
    def case(name, op, requests, chunks, new, ctx, page, hkv=8, g=4, d=128, code="int8", mix=1):
        return {"name": name, "op": op, "requests": requests, "chunks": chunks, "new": new,
                "ctx": ctx, "page": page, "hkv": hkv, "g": g, "d": d, "code": code, "mix": mix}
    return [
        # one decode step's bookkeeping for a full batch: nothing but latency
        case("plan_step", "plan", 64, 0, 1, 8192, 64),
        # a packed batch of prompts, about as many tokens as the framework's packed workload
        case("plan_prompts", "plan", 17, 17, 3915, 0, 64, mix=2),
        # one token of each of 64 requests into half-filled pages
        case("append_step", "append", 64, 0, 1, 2000, 64, mix=3),
        # the prompts' keys and values, e4m3 codes: a stream bound by memory
        case("append_prompts", "append", 17, 17, 3915, 0, 64, code="e4m3", mix=2),
        # short follow-up turns with odd sizes that start and end inside small pages
        case("append_turns", "append", 9, 9, 333, 700, 16, hkv=5, d=64, mix=4),
        # a single short request: the smallest call of a chat
        case("attend_one", "attend", 1, 0, 1, 700, 16, hkv=4, g=8, mix=5),
        # a decode step of a full batch with ragged contexts: bound by the cache's bytes
        case("attend_step", "attend", 64, 0, 1, 8192, 64, mix=6),
        # two requests with very long contexts: the cache split over the whole chip
        case("attend_long", "attend", 2, 0, 1, 262144, 128, hkv=4, g=8, code="e4m3", mix=7),
        # verifying four drafted tokens of each request, narrow heads
        case("attend_drafts", "attend", 32, 32, 4, 4096, 32, hkv=2, g=16, d=64, code="e4m3", mix=8),
        # whole prompts, ragged: bound by the matrix products
        case("attend_prompts", "attend", 9, 9, 4096, 0, 64, mix=9),
        # one piece of a long prompt whose earlier pieces are cached
        case("attend_piece", "attend", 1, 1, 2048, 32768, 64, hkv=4, g=8, code="e4m3", mix=10),
        # a piece of one prompt among other requests' decode steps, a head ratio that is no power of two
        case("attend_mixed", "attend", 17, 1, 512, 6000, 64, hkv=4, g=6, mix=11),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["plan", "append", "attend", "attend"])
    c = {"op": op, "page": rng.choice([16, 32, 64, 128]), "d": rng.choice([64, 128]),
         "code": rng.choice(["int8", "e4m3"]), "mix": rng.randrange(1 << 30)}
    if op == "plan":
        c |= {"requests": spread(1, 1024), "hkv": 8, "g": 4}
        many = rng.random() < 0.5
        c |= {"chunks": rng.randint(0, c["requests"]) if many else 0,
              "new": spread(2, max(3, 32768 // c["requests"])) if many else 1, "ctx": spread(1, 16384)}
        return c
    c |= {"hkv": rng.choice([1, 2, 3, 4, 5, 8]), "g": rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])}
    if op == "append":
        c |= {"requests": spread(1, 128)}
        many = rng.random() < 0.6
        c |= {"chunks": rng.randint(1, c["requests"]) if many else 0,
              "new": spread(2, max(3, 32768 // c["requests"])) if many else 1, "ctx": spread(1, 2000)}
        return c
    kind = rng.choice(["step", "drafts", "prompts", "mixed"])
    if kind in ("step", "drafts"):
        c["requests"] = spread(1, 128)
        most = min(131072, 524288 // c["requests"])
        c |= {"ctx": spread(1, most), "new": 1 if kind == "step" else rng.randint(2, 8)}
        c["chunks"] = 0 if kind == "step" else c["requests"]
    elif kind == "prompts":
        c["requests"] = spread(1, 16)
        c |= {"chunks": c["requests"], "new": spread(9, 2000), "ctx": rng.choice([0, spread(1, 4000)])}
    else:
        c |= {"requests": spread(2, 24), "chunks": 1, "new": spread(9, 700), "ctx": spread(1, 4000)}
    # no dearer than the largest listed case, and the plain form's scores fit the card
    while (work(c)["flops"] > 4e11 or work(c)["bytes"] > 6e8
           or c["requests"] * c["new"] * c["hkv"] * c["g"] * (c["ctx"] + c["new"]) > 4e9):
        big = max(("ctx", "requests", "new"), key=lambda k: c[k] * (16 if k == "requests" else 1))
        c[big] = (c[big] + 1) // 2
        c["chunks"] = min(c["chunks"], c["requests"])
    return c


def lens_of(case):
    """(new tokens, cached tokens) of every request: a ragged batch that the case alone fixes."""
    r = random.Random(case["mix"])
    R, chunks = case["requests"], case["chunks"]
    new = [r.randint(max(1, case["new"] // 8), case["new"]) if i < chunks else 1 for i in range(R)]
    if chunks == 1 or case["new"] <= 8:
        new[:chunks] = [case["new"]] * chunks
    ctx = [r.randint(max(1, case["ctx"] // 8), case["ctx"]) if case["ctx"] else 0 for _ in range(R)]
    ctx[0] = case["ctx"]
    return new, ctx


def up(a, b):
    return -(-a // b)


def runs_of(case):
    """The most runs (a request's new tokens in one page) that a batch of these sizes can have."""
    T = sum(lens_of(case)[0])
    return max(1, min(T, T // case["page"] + 2 * case["requests"]))


def work(case):
    new, ctx = lens_of(case)
    R, T, P, H, D = len(new), sum(new), case["page"], case["hkv"], case["d"]
    if case["op"] == "plan":
        pages = sum(up(n + c, P) - up(c, P) for n, c in zip(new, ctx))
        last = sum((c % P) != 0 for c in ctx)  # the half-filled pages' numbers are read
        return {"bytes": 4 * (2 * R + 2 + 2 * pages + last + 2 * R + 1 + 2 * T + 4 * runs_of(case)), "flops": 0}
    if case["op"] == "append":
        runs = sum(up(n + c, P) - c // P for n, c in zip(new, ctx))
        return {"bytes": 2 * T * H * D * 3 + runs * (16 + 2 * 2 * H * 4), "flops": 2 * T * H * D * 3}
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    held = sum(n + c for n, c in zip(new, ctx))
    pages = sum(up(n + c, P) for n, c in zip(new, ctx))
    rows = T * H * case["g"]
    return {"bytes": 2 * held * H * D + pages * (4 + 8 * H) + rows * (4 * D + 4) + 8 * R,
            "flops": 4 * seen * H * case["g"] * D}


# --------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    new, ctx = lens_of(case)
    R, T, P, H, D = len(new), sum(new), case["page"], case["hkv"], case["d"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    width = max(up(n + c, P) for n, c in zip(new, ctx)) + 1
    held = [up(c, P) for c in ctx]
    after = [up(n + c, P) for n, c in zip(new, ctx)]
    # a pool in use: pages in any order, a few spare ones
    num = sum(after) + 7
    order = torch.randperm(num, generator=gen, **dev).to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, **dev)
    have = held if case["op"] == "plan" else after
    cols = torch.arange(width, **dev)[None, :]
    have_t = torch.tensor(have, **dev)
    first = torch.cumsum(have_t, 0) - have_t
    at = (first[:, None] + cols).clamp(max=num - 1)
    table = torch.where(cols < have_t[:, None], order[at], table).contiguous()
    s = {"case": case, "own": own, "T": T, "page": P, "table": table, "max_new": max(new)}
    new_t, ctx_t = (torch.tensor(x, dtype=torch.int32, **dev) for x in (new, ctx))
    if case["op"] == "plan":
        free = torch.full((num,), -1, dtype=torch.int32, **dev)
        left = num - sum(held)
        free[:left] = order[sum(held):].flip(0)
        return s | {"new": new_t, "ctx": ctx_t, "free": free,
                    "left": torch.tensor([left], dtype=torch.int32, **dev)}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s |= {"cu": torch.tensor(cu, dtype=torch.int32, **dev), "kv": new_t + ctx_t}
    shape = (num, H, P, D)

    def pool():
        # what an append leaves: each page and head has a code at the top of the range
        x = torch.randn(shape, generator=gen, **dev)
        a = x.abs().amax((2, 3), keepdim=True)
        x = x * (TOP[case["code"]] / a)
        return (x.round() if case["code"] == "int8" else x).to(DTYPE[case["code"]])
    s |= {"kc": pool(), "vc": pool()}

    def scales(width):
        # magnitudes as bf16 inputs have them
        x = width * (2 + 2 * torch.rand(num, H, generator=gen, **dev))
        return x.to(torch.bfloat16).float()
    s |= {"ks": scales(1.0), "vs": scales(0.8)}
    if case["op"] == "append":
        # keys and values come as views of one projection's output
        kv = torch.randn(T, 2, H, D, generator=gen, **dev)
        kv[:, 0] *= torch.exp(0.5 * torch.randn(H, 1, generator=gen, **dev))
        kv = kv.to(torch.bfloat16)
        rows = []
        for r, (n, c) in enumerate(zip(new, ctx)):
            p = c
            while p < c + n:
                m = min(P - p % P, c + n - p)
                rows.append((cu[r] + p - c, m, r, p))
                p += m
        host = torch.zeros(runs_of(case), 4, dtype=torch.int32)
        host[:len(rows)] = torch.tensor(rows, dtype=torch.int32)
        runs = host.cuda()
        page = table[runs[:, 2].long(), (runs[:, 3] // P).long()]
        used = runs[:, 1] > 0
        runs[:, 3] = torch.where(used, runs[:, 3] % P, 0)
        runs[:, 2] = torch.where(used, page, 0)
        return s | {"k": kv[:, 0], "v": kv[:, 1], "runs": runs}
    q = torch.randn(T, H * case["g"], D, generator=gen, **dev).to(torch.bfloat16)
    return s | {"q": q}


# --------------------------------------------------------------------------
# the operators

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_32_gb300 as pkg
        if op == "plan":
            p = pkg.page_plan(s["new"], s["ctx"], s["table"], s["free"], s["left"], s["T"], s["page"])
            return [p.cu_seqlens, p.kv_lens, p.slots, p.positions, p.runs, p.free_count, s["table"]]
        if op == "append":
            pkg.cache_append(s["k"], s["v"], s["runs"], s["kc"], s["vc"], s["ks"], s["vs"])
            return [s["kc"], s["vc"], s["ks"], s["vs"]]
        return list(pkg.cache_attend(s["q"], s["cu"], s["kv"], s["table"], s["kc"], s["vc"], s["ks"],
                                     s["vs"], max_new=s["max_new"]))
    if op == "plan":
        return plain_plan(s)
    if op == "append":
        top = TOP[s["case"]["code"]]
        plain_append(s["k"], s["runs"], s["kc"], s["ks"], top)
        plain_append(s["v"], s["runs"], s["vc"], s["vs"], top)
        return [s["kc"], s["vc"], s["ks"], s["vs"]]
    return plain_attend(s)


def plain_plan(s):
    new, ctx, table, P, T = s["new"], s["ctx"], s["table"], s["page"], s["T"]
    R, dev = new.numel(), new.device
    kv = ctx + new
    cu = torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
    before, after = (ctx + P - 1) // P, (kv + P - 1) // P
    need = after - before
    first = need.cumsum(0) - need
    # the pages: from the top of the stack, request by request
    col = torch.arange(table.shape[1], device=dev)[None, :]
    at = s["left"] - 1 - (first[:, None] + col - before[:, None])
    fresh = (col >= before[:, None]) & (col < after[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    # the tokens
    t = torch.arange(T, device=dev, dtype=torch.int32)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    pos = ctx[r] + t - cu[r]
    live = t < cu[R]
    slots = torch.where(live, table[r, (pos // P).long()] * P + pos % P, -1)
    # the runs: a request's new tokens in one page
    parts = torch.where(new > 0, after - ctx // P, 0)
    ends = parts.cumsum(0)
    j = torch.arange(max(1, min(T, T // P + 2 * R)), device=dev)
    q = torch.searchsorted(ends, j, right=True).clamp(max=R - 1)
    p = ctx[q] // P + (j - (ends[q] - parts[q]))
    a, b = torch.maximum(p * P, ctx[q]), torch.minimum(p * P + P, kv[q])
    page = table[q, p.clamp(0, table.shape[1] - 1)]
    runs = torch.stack([cu[q] + a - ctx[q], b - a, page, a % P], 1)
    runs = torch.where((j < ends[-1])[:, None], runs, 0).to(torch.int32)
    return [cu, kv, slots.to(torch.int32), torch.where(live, pos, -1).to(torch.int32), runs,
            s["left"] - need.sum().to(torch.int32), table]


def plain_append(x, runs, codes, scale, top):
    P = codes.shape[2]
    runs = runs[runs[:, 1] > 0].long()
    row, count, page, off = runs.unbind(1)
    i = torch.arange(P, device=x.device)[None, :]
    fresh = (i >= off[:, None]) & (i < (off + count)[:, None])            # [J, P]
    old = i < off[:, None]
    xs = x.float()[(row[:, None] + i - off[:, None]).clamp(0, x.shape[0] - 1)].transpose(1, 2)  # [J, H, P, D]
    most = torch.where(fresh[:, None, :, None], xs.abs(), 0.0).amax((2, 3))
    had = torch.where((off > 0)[:, None], scale[page], 0.0)
    now = torch.maximum(had, most)
    div = torch.where(now > 0, now, 1.0)[:, :, None, None]
    held = codes[page]
    c = torch.where(fresh[:, None, :, None], (xs * top) / div, (held.float() * had[:, :, None, None]) / div)
    c = (c.round() if codes.dtype == torch.int8 else c).to(codes.dtype)
    # (bytes, since not every operation takes 8-bit floats)
    keep = (fresh | old)[:, None, :, None]
    codes.view(torch.uint8)[page] = torch.where(keep, c.view(torch.uint8), held.view(torch.uint8))
    scale[page] = now


def plain_attend(s):
    q, cu, kv, P = s["q"], s["cu"], s["kv"], s["page"]
    T, HQ, D = q.shape
    R, H, N = kv.numel(), s["kc"].shape[1], s["max_new"]
    G, dev, top = HQ // H, q.device, TOP[s["case"]["code"]]

    def gather(codes, scale):
        pages = s["table"].clamp(min=0).long()
        x = codes.view(torch.uint8)[pages].view(codes.dtype).float() * (scale[pages] / top)[..., None, None]
        return x.transpose(1, 2).reshape(R, H, -1, D)                     # [R, H, L, D]
    new = cu[1:] - cu[:-1]
    i = torch.arange(N, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=T - 1).long()
    qs = q.float()[rows].reshape(R, N, H, G, D).transpose(1, 2).reshape(R, H, N * G, D)
    x = torch.matmul(qs, gather(s["kc"], s["ks"]).transpose(2, 3)).mul_(D ** -0.5).reshape(R, H, N, G, -1)
    seen = (kv - new)[:, None] + i + 1
    dead = torch.arange(x.shape[-1], device=dev) >= seen[:, :, None]      # [R, N, L]
    x.masked_fill_(dead[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m.isfinite(), m, 0.0)).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(R, H, N * G, -1), gather(s["vc"], s["vs"])).reshape(R, H, N, G, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + l.log())[..., 0]
    t = torch.arange(T, device=dev, dtype=torch.int32)
    r = torch.searchsorted(cu[1:], t, right=True)
    n = (t - cu[r]).long()
    return [o[r, :, n].reshape(T, HQ, D).to(q.dtype), lse[r, :, n].reshape(T, HQ)]


# --------------------------------------------------------------------------
# the definition in 64 bits

def to_grid(x, code):
    """The nearest code of each value, ties to even."""
    if code == "int8":
        return x.round()
    a = x.abs()
    e = torch.frexp(a).exponent - 1                                       # a in [2^e, 2^(e+1))
    step = torch.exp2((e.clamp(min=-6) - 3).double())
    return (a / step).round() * step * x.sign()


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    code, top, P = case["code"], TOP[case["code"]], case["page"]
    new, ctx = lens_of(case)
    if case["op"] == "append":
        outs = []
        for x, codes, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
            codes, scale = codes.double(), scale.double()
            for row, count, page, off in s["runs"].tolist():
                if not count:
                    continue
                xs = x[row:row + count].double().transpose(0, 1)          # [H, count, D]
                had = scale[page].clone() if off else torch.zeros_like(scale[page])
                now = torch.maximum(had, xs.abs().amax((1, 2)))
                part = now[:, None, None].clamp(min=1e-300)
                codes[page, :, :off] = to_grid(codes[page, :, :off] * had[:, None, None] / part, code)
                codes[page, :, off:off + count] = to_grid(xs * top / part, code)
                scale[page] = now
            outs.append((codes, scale))
        return [outs[0][0], outs[1][0], outs[0][1], outs[1][1]]
    T, HQ, D = s["q"].shape
    H, G = case["hkv"], case["g"]
    if sum(n * c + n * n for n, c in zip(new, ctx)) * HQ * D * 4 > 6e12:
        return None
    o = torch.zeros(T, HQ, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, HQ), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for r, (n, c) in enumerate(zip(new, ctx)):
        pages = s["table"][r, :up(n + c, P)].long()
        for h in range(H):
            # [L, D]: the values that the codes stand for
            k, v = (a[:, h].view(torch.uint8)[pages].view(a.dtype).double().mul_(b[pages, h].double()[:, None, None] / top)
                    .reshape(-1, D)[:n + c] for a, b in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for g in range(G):
                x = s["q"][t:t + n, h * G + g].double() @ k.T / math.sqrt(D)
                x += torch.full_like(x, -math.inf).triu(c + 1)
                z = torch.logsumexp(x, 1)
                o[t:t + n, h * G + g] = torch.exp(x - z[:, None]) @ v
                lse[t:t + n, h * G + g] = z
        t += n
    return [o, lse]
