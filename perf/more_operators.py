"""Cases that time linear attention with a decay for each head (whole prompts and single tokens) and rotary positions.

A hybrid model's recurrent layers without the delta rule keep a state S of
[dk, dv] for each head, which decays by one factor a token:

    S_t = exp(a_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   a_t = min(log_decay, 0)

with a_t of its own for every token and head, or one for each head.  Their
queries and keys, and those of the attention layers beside them, carry rotary
positions: pair i of a head's first `rotary` channels is turned by position *
frequency_i.  `run` computes them in plain 32-bit torch operations where `own`
is false and calls the library where it is true; `exact` states them once
more in 64 bits, token by token.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------
# cases

def listed():
    def attend(name, rows, tokens, heads, key_heads=None, dk=128, dv=128, packed=False, decay="token", init=False,
               views=False, dtype="bf16", mix=1, op="attend"):
        return {"name": name, "op": op, "rows": rows, "tokens": tokens, "heads": heads, "key_heads": key_heads or heads,
                "dk": dk, "dv": dv, "packed": packed, "decay": decay, "init": init, "views": views, "dtype": dtype,
                "mix": mix}

    def rotary(name, requests, new, ctx, hq, hk, d, part, interleaved, stretch, dtype="bf16", mix=1):
        return {"name": name, "op": "rotary", "requests": requests, "new": new, "ctx": ctx, "hq": hq, "hk": hk, "d": d,
                "part": part, "interleaved": interleaved, "stretch": stretch, "dtype": dtype, "mix": mix}
    return [
        # a single short prompt on narrow heads: the smallest prompt of a chat, nothing but latency
        attend("attend_one", 1, 77, 8, dk=64, dv=64),
        # one prompt of a model with few heads: the framework's 4-head, 4096-token sizes
        attend("attend_few_heads", 1, 4096, 4, init=True),
        # the framework's benchmark sizes: two rows of 32 heads, bound by memory
        attend("attend_rows", 2, 32768, 32),
        # ragged prompts in one packed step, as many as the framework's packed workload; views of one projection
        attend("attend_packed", 17, 3915, 16, packed=True, init=True, views=True, mix=2),
        # one very long prompt with one decay for each head: the token axis split over the chip
        attend("attend_long", 1, 131072, 16, decay="head"),
        # queries and keys shared by 16 value heads each, narrow values, an odd length
        attend("attend_shared", 8, 2001, 32, key_heads=2, dv=64, views=True, mix=3),
        # 32-bit inputs on a head size of their own: what a user checks a model with
        attend("attend_f32", 2, 333, 4, dk=64, dv=32, decay="head", init=True, dtype="f32"),
        # a decode step of a full batch: bound by the state's bytes
        attend("decode_step", 64, 1, 32, op="decode"),
        # four drafted tokens of each request, shared keys, views of one projection
        attend("decode_drafts", 24, 4, 24, key_heads=3, dv=64, views=True, op="decode"),
        # positions of one decode step's queries and keys: latency
        rotary("rotary_step", 64, 1, 8192, 32, 8, 128, 128, False, 1.0),
        # ragged prompts far into stretched contexts: a stream bound by memory
        rotary("rotary_prompts", 17, 3915, 131072, 32, 8, 128, 128, False, 4.0, mix=2),
        # interleaved pairs in half of the channels, follow-up turns of odd sizes in 32 bits
        rotary("rotary_part", 9, 333, 700, 6, 2, 64, 32, True, 1.0, dtype="f32", mix=4),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    mix = rng.randrange(1 << 30)
    op = rng.choice(["attend", "attend", "decode", "rotary"])
    if op == "rotary":
        d = rng.choice([64, 128])
        step = rng.random() < 0.4
        c = {"op": op, "requests": spread(1, 256), "ctx": spread(1, 1000000), "hq": rng.choice([1, 4, 6, 8, 16, 32]),
             "hk": rng.choice([1, 2, 3, 4, 8]), "d": d, "part": rng.choice([d, d, d // 2, 16]),
             "interleaved": rng.random() < 0.5, "stretch": rng.choice([1.0, 4.0, 8.0]),
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "mix": mix}
        c["new"] = 1 if step else spread(2, max(3, 32768 // c["requests"]))
        while work(c)["bytes"] > 6e8:
            c["new"] = (c["new"] + 1) // 2
        return c
    c = {"op": op, "key_heads": rng.choice([1, 2, 3, 4, 8]), "decay": rng.choice(["token", "token", "head"]),
         "init": rng.random() < 0.5, "views": rng.random() < 0.5, "dtype": rng.choice(["bf16"] * 4 + ["f32"]), "mix": mix}
    c["heads"] = c["key_heads"] * rng.choice([1, 1, 2, 5])
    sizes = [64, 128] if c["dtype"] == "bf16" and rng.random() < 0.8 else [16, 32, 64, 128]
    c |= {"dk": rng.choice(sizes), "dv": rng.choice(sizes)}
    if op == "decode":
        return c | {"rows": spread(1, 128), "tokens": rng.choice([1, 1, 1, 2, 3, 4, 7, 16]), "packed": False}
    # (the tensor cores serve 16-bit inputs of 64 or 128 channels; the others run token by token: shorter)
    wide = c["dtype"] == "bf16" and min(c["dk"], c["dv"]) >= 64
    c |= {"rows": spread(1, 32), "tokens": spread(1, 32768 if wide else 1000), "packed": rng.random() < 0.5}
    while c["rows"] * c["tokens"] * c["heads"] > (1 << 20) or c["rows"] * c["tokens"] > (1 << 17):
        big = max(("tokens", "rows"), key=lambda k: c[k] * (64 if k == "rows" else 1))
        c[big] = (c[big] + 1) // 2
    return c


def lens_of(case):
    """Tokens of each sequence (rotary: of each request, and what it has cached): the case alone fixes them."""
    r = random.Random(case["mix"])
    if case["op"] == "rotary":
        new = [r.randint(max(1, case["new"] // 8), case["new"]) for _ in range(case["requests"])]
        ctx = [r.randint(0, case["ctx"]) for _ in range(case["requests"])]
        return new, ctx
    if not case["packed"]:
        return [case["tokens"]] * case["rows"]
    lens = [r.randint(max(1, case["tokens"] // 24), case["tokens"]) for _ in range(case["rows"])]
    lens[0] = case["tokens"]
    return lens


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "rotary":
        T = sum(lens_of(case)[0])
        n = T * (case["hq"] + case["hk"])
        return {"bytes": 2 * size * n * case["d"] + 4 * T + 4 * case["part"], "flops": 3 * n * case["part"]}
    lens = lens_of(case)
    T, N, H, HK, dk, dv = sum(lens), len(lens), case["heads"], case["key_heads"], case["dk"], case["dv"]
    states = 2 if case["op"] == "decode" or case["init"] else 1
    decay = 4 * H * (T if case["decay"] == "token" else 1)
    return {"bytes": size * T * (2 * HK * dk + 2 * H * dv) + decay + states * 4 * N * H * dk * dv + (4 * N + 4 if case["packed"] else 0),
            "flops": 4 * T * H * dk * dv}


# --------------------------------------------------------------------------
# inputs

def frequencies(part, stretch):
    """Radians a token of each pair (64 bits) and the amplitude: base 10000, and for contexts `stretch` times as long
    as the 4096 tokens of training the slow pairs slowed down, the fast ones kept, a ramp between."""
    n = part // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    if stretch == 1.0:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)                 # within the length of training
    keep = ((turns - 1) / (32 - 1)).clamp(0.0, 1.0)
    return f * keep + f / stretch * (1 - keep), 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    dtype = DTYPE[case["dtype"]]
    if case["op"] == "rotary":
        new, ctx = lens_of(case)
        T, hq, hk, d = sum(new), case["hq"], case["hk"], case["d"]
        # queries and keys come as views of one projection's output
        x = torch.randn(T, hq + 2 * hk, d, generator=gen, **dev).to(dtype)
        pos = torch.cat([torch.arange(c, c + n, dtype=torch.int32) for n, c in zip(new, ctx)]).cuda()
        f, amp = frequencies(case["part"], case["stretch"])
        return {"case": case, "q": x[:, :hq], "k": x[:, hq:hq + hk], "pos": pos, "f": f, "amp": amp}
    lens = lens_of(case)
    N, H, HK, dk, dv = len(lens), case["heads"], case["key_heads"], case["dk"], case["dv"]
    B, T = (1, sum(lens)) if case["packed"] else (N, case["tokens"])

    def normal(*shape):
        return torch.randn(*shape, generator=gen, **dev)

    def unit(heads, d):
        return torch.nn.functional.normalize(normal(B, T, heads, d), dim=-1).to(dtype)
    q, k, v = unit(HK, dk), unit(HK, dk), normal(B, T, H, dv).to(dtype)
    if case["views"]:
        x = torch.cat([y.flatten(2) for y in (q, k, v)], 2)
        q, k, v = (y.reshape(B, T, -1, d) for y, d in zip(x.split([HK * dk, HK * dk, H * dv], 2), (dk, dk, dv)))
    if case["decay"] == "token":
        # rates from a few tokens to some thousand, modulated by each token
        rate = torch.exp(normal(H) * 1.5 - 4.0)
        decay = -rate * torch.nn.functional.softplus(normal(B, T, H) + 1.0)
    else:
        decay = -torch.exp2(-8.0 * (torch.arange(H, **dev) + 1.0) / H) * (1.0 + 0.01 * torch.rand(H, generator=gen, **dev))
    s = {"case": case, "q": q, "k": k, "v": v, "decay": decay, "scale": dk ** -0.5, "cu": None, "state": None,
         "longest": max(lens)}
    if case["packed"]:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, **dev)
    if case["init"] or case["op"] == "decode":
        s["state"] = normal(N, H, dk, dv)
    return s


# --------------------------------------------------------------------------
# the operators

def run(s):
    case = s["case"]
    if own:
        import gated_delta_rule_32_gb300 as pkg
        if case["op"] == "rotary":
            return list(pkg.rotary_embed(s["q"], s["k"], s["pos"], s["f"], interleaved=case["interleaved"],
                                         amplitude=s["amp"]))
        if case["op"] == "decode":
            out = pkg.linear_decode(s["q"], s["k"], s["v"], s["decay"], s["state"], scale=s["scale"])
            return [out, s["state"]]
        return list(pkg.linear_attend(s["q"], s["k"], s["v"], s["decay"], s["state"], s["cu"], scale=s["scale"]))
    if case["op"] == "rotary":
        t = s["pos"].double()[:, None] * s["f"]
        cos, sin = ((fn(t) * s["amp"]).float()[:, None] for fn in (torch.cos, torch.sin))
        return [plain_rotary(x, cos, sin, case["part"], case["interleaved"]) for x in (s["q"], s["k"])]
    if case["op"] == "decode":
        out, state = plain_attend(s["q"], s["k"], s["v"], s["decay"], s["state"], s["scale"], 16)
        s["state"].copy_(state)
        return [out.to(s["v"].dtype), s["state"]]
    if s["cu"] is None:
        out, state = plain_attend(s["q"], s["k"], s["v"], s["decay"], s["state"], s["scale"], 64)
        return [out.to(s["v"].dtype), state]
    # packed: rows of the longest length, what is behind a sequence's end without weight
    cu, L = s["cu"].long(), s["longest"]
    i = torch.arange(L, device=cu.device)
    live = i < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[1] - 1)
    q, k, v = (torch.where(live[..., None, None], x[0][rows].float(), 0.0) for x in (s["q"], s["k"], s["v"]))
    decay = s["decay"] if s["decay"].dim() == 3 else s["decay"].expand(1, s["q"].shape[1], -1)
    decay = torch.where(live[..., None], decay[0][rows], 0.0)
    out, state = plain_attend(q, k, v, decay, s["state"], s["scale"], 64)
    return [out[live][None].to(s["v"].dtype), state]


def plain_attend(q, k, v, decay, state, scale, C):
    """Linear attention in chunks of C tokens: within a chunk by weighted products, across by the chunks' states."""
    B, T, H, dv = v.shape
    group, dk, n = H // k.shape[2], k.shape[3], -(-T // C)
    decay = decay if decay.dim() == 3 else decay.expand(B, T, H)

    def chunks(x):                                                       # [B, H, n, C, .]
        x = torch.nn.functional.pad(x.float(), (0, 0) * (x.dim() - 2) + (0, n * C - T))
        return x.reshape(B, n, C, *x.shape[2:]).movedim(3, 1)
    q, k = (chunks(x.repeat_interleave(group, 2) if group > 1 else x) for x in (q, k))
    v, a = chunks(v), chunks(decay.clamp(max=0.0))
    g = a.double().cumsum(-1)                                            # [B, H, n, C]
    behind = torch.ones(C, C, dtype=torch.bool, device=v.device).triu(1)
    w = (g[..., :, None] - g[..., None, :]).masked_fill_(behind, -math.inf).exp_().float()
    out = (q @ k.transpose(-1, -2)).mul_(w) @ v
    add = (k * (g[..., -1:] - g).exp().float()[..., None]).transpose(-1, -2) @ v       # what each chunk adds
    # the state before chunk c, and after the last: sums over the chunks before it (and the initial state)
    e = torch.nn.functional.pad(g[..., -1].cumsum(-1), (1, 0))           # [B, H, n + 1]
    later = torch.ones(n + 1, n, dtype=torch.bool, device=v.device).triu()
    m = (e[..., :, None] - e[..., None, 1:]).masked_fill_(later, -math.inf).exp_().float()
    states = (m @ add.reshape(B, H, n, -1)).reshape(B, H, n + 1, dk, dv)
    if state is not None:
        states += e.exp().float()[..., None, None] * state[:, :, None]
    out += g.exp().float()[..., None] * (q @ states[:, :, :-1])
    out = out.mul_(scale).movedim(1, 3).reshape(B, n * C, H, dv)[:, :T]
    return out, states[:, :, -1].contiguous()


def plain_rotary(x, cos, sin, part, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:part:2], y[..., 1:part:2]
    else:
        a, b = y[..., :part // 2], y[..., part // 2:part]
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., part:]], -1).to(x.dtype)


# --------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for i in range(case["part"] // 2):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["part"] // 2)
                t = (s["pos"].double() * s["f"][i])[:, None]
                c, z = torch.cos(t) * s["amp"], torch.sin(t) * s["amp"]
                y[..., a], y[..., b] = (x[..., a].double() * c - x[..., b].double() * z,
                                        x[..., a].double() * z + x[..., b].double() * c)
            outs.append(y)
        return outs
    lens = lens_of(case)
    longest, N, H, dk, dv = max(lens), len(lens), case["heads"], case["dk"], case["dv"]
    if longest * (1 + N * H * dk * dv / 4e6) > 400000:
        return None
    group = H // case["key_heads"]
    state = torch.zeros(N * H, dk, dv, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double().reshape(N * H, dk, dv)
    out = torch.zeros_like(s["v"], dtype=torch.float64)
    q, k, v = (x.double().flatten(0, 1) for x in (s["q"], s["k"], s["v"]))
    keep = torch.exp(s["decay"].double().clamp(max=0.0))
    keep = keep.flatten(0, 1) if keep.dim() == 3 else keep.expand(q.shape[0], H)
    flat = out.view(-1, H, dv)
    ends = torch.tensor(lens, device="cuda")
    first = torch.cumsum(ends, 0) - ends                                 # (dense rows follow each other too)
    same = min(lens) == longest
    for t in range(longest):
        on = slice(None) if same else (ends > t).nonzero()[:, 0]
        rows = (first + t)[on]
        kt, qt = (x[rows].repeat_interleave(group, 1).reshape(-1, dk) for x in (k, q))
        vt, at = v[rows].reshape(-1, 1, dv), keep[rows].reshape(-1, 1, 1)
        if same:
            state.mul_(at).baddbmm_(kt[:, :, None], vt)
            new = state
        else:
            new = state.view(N, H, dk, dv)[on].reshape(-1, dk, dv).mul_(at).baddbmm_(kt[:, :, None], vt)
            state.view(N, H, dk, dv)[on] = new.view(-1, H, dk, dv)
        flat[rows] = (torch.bmm(qt[:, None], new)[:, 0] * s["scale"]).view(-1, H, dv)
    return [out, state.view(N, H, dk, dv)]
