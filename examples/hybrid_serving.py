"""Serving a hybrid model: gated delta rule layers with a state of fixed size
beside attention layers with a paged 8-bit cache, on one GPU.

A batch of ragged prompts is taken in one packed step, then every request
decodes token by token; finished requests give their pages back and new ones
take their place.  One page plan serves every layer of a step: its cu_seqlens
is what the packed gated delta rule forward takes, its runs say where the
attention layers append, its lengths and the block table where they read.

    python examples/hybrid_serving.py [--code int8|e4m3] [--steps 16]

Weights are random; the projections are plain matrix products.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_32_gb300 as pkg  # noqa: E402
from gated_delta_rule_32_gb300 import kda  # noqa: E402

CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class Hybrid:
    """`layers`: a string of "k" (gated delta rule) and "a" (attention)."""

    def __init__(self, layers="kkka", width=512, heads=4, q_heads=8, kv_heads=2, dim=64, page=32,
                 requests=4, pages=256, pages_per_request=64, code="int8", seed=0):
        self.layers, self.width, self.heads = layers, width, heads
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(rows)
            return w.to(torch.bfloat16)
        ints = {"dtype": torch.int32, "device": "cuda"}
        self.w, self.state, self.cache = [], [], []
        for kind in layers:
            if kind == "k":
                # q, k, v, decay logits (128 channels a head), write strength
                self.w.append((weight(width, heads * (4 * 128 + 1)), weight(heads * 128, width)))
                self.state.append(torch.zeros(requests, heads, 128, 128, device="cuda"))
                self.cache.append(None)
            else:
                self.w.append((weight(width, (q_heads + 2 * kv_heads) * dim),
                               weight(q_heads * dim, width)))
                shape = (pages, kv_heads, page, dim)
                self.state.append(None)
                self.cache.append((torch.zeros(shape, dtype=CODES[code], device="cuda"),
                                   torch.zeros(shape, dtype=CODES[code], device="cuda"),
                                   torch.zeros(shape[:2], device="cuda"),
                                   torch.zeros(shape[:2], device="cuda")))
        # the pages' bookkeeping, shared by the attention layers
        self.table = torch.full((requests, pages_per_request), -1, **ints)
        self.lens = torch.zeros(requests, **ints)
        self.free = torch.arange(pages - 1, -1, -1, **ints)
        self.left = torch.full((1,), pages, **ints)
        # what the device finds: of the plan, the release, and each layer's two calls
        self.status = torch.zeros(2 + 2 * len(layers), **ints)

    def check(self):
        """Raises what the device has found since the last look (waits for it)."""
        found = self.status.tolist()
        if any(found):
            self.status.zero_()
            at = next(i for i, code in enumerate(found) if code)
            what = ["kda_page_plan", "kda_page_release"] + ["kda_cache_append", "kda_cache_attn"] * \
                len(self.layers)
            raise kda.KdaError(what[at], found[at])

    def step(self, x, new_lens, max_new):
        """x [T, width]: the packed new tokens, new_lens[r] of request r, at
        most max_new each.  Returns the last layer's output [T, width].  A step
        that does not fit raises before anything has changed; what the layers'
        calls find (more than max_new tokens, say) the next step or check() raises."""
        T = x.shape[0]
        plan = pkg.page_plan(new_lens, self.lens, self.table, self.free, self.left, T, self.page,
                             dev_status=self.status[0:1])
        self.check()
        for i, kind in enumerate(self.layers):
            y = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
            y = y @ self.w[i][0]
            if kind == "k":
                y = self.delta_rule(i, y, plan, max_new)
            else:
                q, k, v = (t.reshape(T, -1, self.dim) for t in y.split(
                    [n * self.dim for n in (self.q_heads, self.kv_heads, self.kv_heads)], dim=1))
                kc, vc, ks, vs = self.cache[i]
                # q, k, v stay views of the projection's output: token strides differ
                at = 2 + 2 * i
                pkg.cache_append(k, v, plan.runs, kc, vc, ks, vs, dev_status=self.status[at:at + 1])
                y, _ = pkg.cache_attend(q, plan.cu_seqlens, plan.kv_lens, self.table, kc, vc, ks, vs,
                                        max_new=max_new, dev_status=self.status[at + 1:at + 2])
            x = x + y.reshape(T, -1) @ self.w[i][1]
        self.lens, self.left = plan.kv_lens, plan.free_count
        return x

    def delta_rule(self, i, y, plan, max_new):
        T, H = y.shape[0], self.heads
        q, k, v, g, b = y.split([H * 128] * 4 + [H], dim=1)
        q, k, v, g = (t.reshape(1, T, H, 128).contiguous() for t in (q, k, v, g))
        q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
        b = torch.sigmoid(b).reshape(1, T, H).contiguous()
        state = self.state[i]
        if max_new == 1 and T == state.shape[0]:  # one token of every request
            out = torch.empty_like(v)
            rc = kda.kda_decode(q, k, v, g, b, state, out, T, 1, H, 128, 128, kda.KDA_BF16, 1.0,
                                torch.cuda.current_stream())
            if rc != kda.KDA_OK:
                raise kda.KdaError("kda_decode", rc)
        else:
            out, self.state[i] = pkg.forward(q, k, v, g, b, state, plan.cu_seqlens)
        return out

    def finish(self, done):
        """Requests with done[r] != 0 leave: their pages go back, their states to zero."""
        pkg.page_release(done, self.lens, self.table, self.free, self.left, self.page,
                         dev_status=self.status[1:2])
        self.check()
        for s in self.state:
            if s is not None:
                s.masked_fill_((done != 0)[:, None, None, None], 0.0)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--code", choices=sorted(CODES), default="int8")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    torch.manual_seed(1)
    lens = [301, 17, 96, 640]
    model = Hybrid(code=a.code, requests=len(lens))

    def tokens(n):
        return torch.randn(n, model.width, device="cuda").to(torch.bfloat16)
    ints = {"dtype": torch.int32, "device": "cuda"}
    model.step(tokens(sum(lens)), torch.tensor(lens, **ints), max(lens))
    one = torch.ones(len(lens), **ints)
    out = model.step(tokens(len(lens)), one, 1)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        out = model.step(out, one, 1)
    model.check()
    ms = (time.perf_counter() - t) / max(1, a.steps) * 1e3
    print("lengths %s, pages left %d, %.2f ms a decode step" % (model.lens.tolist(), model.left, ms))
    # the second request leaves, another takes its row
    model.finish(torch.tensor([0, 1, 0, 0], **ints))
    print("pages left %d after one request left" % model.left)
    out = model.step(tokens(3 + 50), torch.tensor([1, 50, 1, 1], **ints), 50)
    model.check()
    print("lengths %s, pages left %d, output finite: %s" % (
        model.lens.tolist(), model.left, bool(out.isfinite().all())))
    return model, out


if __name__ == "__main__":
    main()
