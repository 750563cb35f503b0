"""Rotary positions on the GPU against the 64-bit form, and the run of
operators that they begin: rotary, then linear attention over a prompt and
single tokens; plan, rotary, append, attention over the paged cache."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _cache_oracle, _linear_oracle as plain

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def made(T, Hq, Hk, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hk, d, generator=g, device="cuda").to(dtype)
    return x[:, :Hq], x[:, Hq:Hq + Hk]


def check(got, x, pos, f, angle=0.0, **kw):
    """Angles within 2^-25 of half a turn (an fp32 fraction of it) and one ulp or
    two of sine and cosine: 2^-21 of the pair's length; fp32 products; the rounding.
    `angle`: what else the angle may be off, in radians."""
    want = plain.turn(x.cpu(), pos.cpu(), f.cpu(), **kw)
    rows = pos.cpu() >= 0
    part = 2 * f.numel()
    y = x.cpu().double()
    size = y.abs()
    if part:
        if kw.get("interleaved"):
            a, b = y[..., 0:part:2], y[..., 1:part:2]
            size[..., 0:part:2] = size[..., 1:part:2] = (a * a + b * b).sqrt()
        else:
            a, b = y[..., :part // 2], y[..., part // 2:part]
            size[..., :part] = (a * a + b * b).sqrt().repeat(1, 1, 2)
    half = plain.BF16 if got.dtype is BF else 2.0 ** -24
    tol = half * want.abs() + (2.0 ** -20 + angle) * abs(kw.get("amplitude", 1.0)) * size
    err = (got.cpu().double() - want).abs()
    assert (err <= tol)[rows].all(), (err / tol)[rows].max()
    assert torch.equal(got[..., part:][pos >= 0], x[..., part:][pos >= 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,part", [(1, 1, 1, 64, 64), (5, 8, 2, 128, 128), (33, 3, 5, 64, 32), (2, 4, 1, 16, 16),
                                            (7, 2, 2, 192, 64), (300, 6, 1, 128, 112), (19, 1, 1, 512, 256)])
def test_turns(T, Hq, Hk, d, part, interleaved, dtype):
    q, k = made(T, Hq, Hk, d, dtype, seed=T)
    f, amp = pkg.rotary_frequencies(part)
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32, device="cuda")
    pos[0] = 0
    for inverse in (False, True):
        a, b = pkg.rotary_embed(q, k, pos, f, interleaved=interleaved, inverse=inverse, amplitude=1.25)
        check(a, q, pos, f, interleaved=interleaved, inverse=inverse, amplitude=1.25)
        check(b, k, pos, f, interleaved=interleaved, inverse=inverse, amplitude=1.25)


def test_far_positions():
    # frequencies and their turns are 64-bit floating point numbers: two roundings of 2^-53 in the
    # kernel and one in the plain form, times a position below 2^31, are below 2^-20 of a radian
    q, k = made(64, 2, 2, 64, F32)
    f, _ = pkg.rotary_frequencies(64)
    pos = torch.randint(1 << 30, (1 << 31) - 1, (64,), dtype=torch.int64, device="cuda").to(torch.int32)
    pos[0] = (1 << 31) - 1
    a, b = pkg.rotary_embed(q, k, pos, f)
    check(a, q, pos, f, angle=2.0 ** -20)
    check(b, k, pos, f, angle=2.0 ** -20)
    # frequencies above a turn a token
    f = torch.tensor([100.0, 7.5, 2 * math.pi, 0.0] * 4, dtype=torch.float64, device="cuda")
    a, b = pkg.rotary_embed(q, None, pos % 1000, f)
    assert b is None
    check(a, q, pos % 1000, f)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_rows_without_a_token(interleaved):
    q, k = made(40, 4, 2, 128, BF, seed=2)
    f, _ = pkg.rotary_frequencies(64)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    pos[7], pos[33:] = -1, -1
    a, b = pkg.rotary_embed(q, k, pos, f, interleaved=interleaved)
    q0, k0 = q.clone(), k.clone()
    v = q._base[:, 6:].clone()
    c, d = pkg.rotary_embed(q, k, pos, f, interleaved=interleaved, inplace=True)
    assert c is q and d is k
    on = pos >= 0
    assert torch.equal(q[on], a[on]) and torch.equal(k[on], b[on])
    assert torch.equal(q[~on], q0[~on]) and torch.equal(k[~on], k0[~on])
    assert torch.equal(q._base[:, 6:], v)


def test_no_tokens():
    q, k = made(0, 4, 2, 64, BF)
    f, _ = pkg.rotary_frequencies(64)
    a, b = pkg.rotary_embed(q, k, torch.zeros(0, dtype=torch.int32, device="cuda"), f)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)


def test_inverse_is_the_gradient():
    # <g, R x> = <R^T g, x> for each channel: against differences in 32 bits
    q, _ = made(9, 2, 1, 64, F32, seed=3)
    g, _ = made(9, 2, 1, 64, F32, seed=4)
    f, amp = pkg.rotary_frequencies(32, scaling="yarn", factor=4.0)
    pos = torch.arange(5, 14, dtype=torch.int32, device="cuda")

    def turn(x, **kw):
        return pkg.rotary_embed(x, None, pos, f, amplitude=amp, **kw)[0]
    grad = turn(g, inverse=True)
    for c in (0, 3, 16, 31, 40):
        up, down = q.clone(), q.clone()
        up[:, :, c] += 1.0
        down[:, :, c] -= 1.0
        slope = (g.double() * (turn(up).double() - turn(down).double())).sum(-1) / 2
        # (the map is linear: differences over a step of 2 err by fp32 roundings of values up to 6)
        assert (slope - grad[:, :, c].double()).abs().max() < 64 * 8 * 2.0 ** -23 * 6


def test_strides_by_token_and_streams():
    q, k = made(50, 4, 2, 64, BF, seed=5)
    f, _ = pkg.rotary_frequencies(64)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = pkg.rotary_embed(q.contiguous(), k.contiguous(), pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.rotary_embed(q, k, pos, f, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rotary_then_linear_attention():
    """A retention layer: a packed prompt, then two tokens of every request."""
    lens, H, d = [70, 200, 1, 133], 4, 128
    T, N = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    f, amp = pkg.rotary_frequencies(d)
    decay = torch.log(1 - torch.exp2(-5.0 - torch.arange(H, device="cuda")))
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    x = (normal(T, 3 * H, d) / d ** 0.25).to(BF)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    q, k = pkg.rotary_embed(x[:, :H], x[:, H:2 * H], pos, f, amplitude=amp)
    out, state = pkg.linear_attend(q[None], k[None], x[None, :, 2 * H:], decay, None, cu)
    y = (normal(N, 2, 3 * H, d) / d ** 0.25).to(BF)
    pos2 = (torch.tensor(lens, device="cuda")[:, None] + torch.arange(2, device="cuda")).to(torch.int32)
    flat = y.flatten(0, 1)
    q2, k2 = pkg.rotary_embed(flat[:, :H], flat[:, H:2 * H], pos2.flatten(), f, amplitude=amp)
    kept = state.clone()
    out2 = pkg.linear_decode(q2.view(N, 2, H, d), k2.view(N, 2, H, d), y[:, :, 2 * H:], decay, state)
    # the same from the definition: each request's prompt and tokens in one sequence.  The turned
    # queries and keys are rounded to 16 bits: both relative roundings count once more in each product
    at = 0
    for n, L in enumerate(lens):
        z = torch.cat([x[at:at + L], y[n]]).cpu()
        p = torch.arange(L + 2)
        qd, kd = (plain.turn(z[:, i * H:(i + 1) * H], p, f.cpu(), amplitude=amp)[None].cuda() for i in (0, 1))
        o, s, om, sm = plain.attend(qd, kd, z[None, :, 2 * H:].cuda(), decay, None, 1.0)
        got = torch.cat([out[0, at:at + L], out2[n]]).double()
        assert ((got - o[0]).abs() <= plain.BF16 * o[0].abs() + 3.1 * plain.BF16 * om[0]).all()
        # (independent roundings: norms add up as squares)
        assert (got - o[0]).norm() <= 2 * plain.BF16 * o[0].norm()
        assert ((state[n].double() - s[0]).abs() <= 1.01 * plain.BF16 * sm[0]).all()
        at += L
    assert not torch.equal(kept, state)


def test_plan_rotary_append_attend():
    """An attention layer: the plan's positions turn queries and keys, which go through the cache."""
    new, ctx, page, Hq, Hk, d = [40, 1, 17], [0, 0, 0], 16, 4, 2, 64
    T, R = sum(new), len(new)
    ints = {"dtype": torch.int32, "device": "cuda"}
    table = torch.full((R, 8), -1, **ints)
    free, left = torch.arange(15, -1, -1, **ints), torch.full((1,), 16, **ints)
    kc, vc = (torch.zeros(16, Hk, page, d, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(16, Hk, device="cuda") for _ in "kv")
    f, amp = pkg.rotary_frequencies(d)
    plan = pkg.page_plan(torch.tensor(new, **ints), torch.tensor(ctx, **ints), table, free, left, T + 3, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T + 3, Hq + 2 * Hk, d, generator=g, device="cuda").to(BF)
    x[T:] = math.nan
    want_q, want_k = (plain.turn(y.cpu(), plan.positions.cpu(), f.cpu()) for y in (x[:, :Hq], x[:, Hq:Hq + Hk]))
    q, k = pkg.rotary_embed(x[:, :Hq], x[:, Hq:Hq + Hk], plan.positions, f, inplace=True)
    assert plan.positions[T:].tolist() == [-1] * 3
    assert (q[:T].cpu().double() - want_q[:T]).abs().max() <= plain.BF16 * 8
    pkg.cache_append(k, x[:, Hq + Hk:], plan.runs, kc, vc, ks, vs)
    out, lse = pkg.cache_attend(q, plan.cu_seqlens, plan.kv_lens, table, kc, vc, ks, vs, max_new=40)
    o, l, to, tl = _cache_oracle.attend(q[:T].cpu(), plan.cu_seqlens.tolist(), plan.kv_lens.tolist(),
                                        table.tolist(), kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), d ** -0.5)
    assert ((out[:T].cpu().double() - o).abs() <= to).all()
    # and the cache holds the turned keys: codes within half a step of 1 / 127 of the page's largest
    for r in range(R):
        a = sum(new[:r])
        for i in range(new[r]):
            pg = table[r, i // page].item()
            held = kc[pg, :, i % page].double() * (ks[pg].double() / 127)[:, None]
            step = ks[pg].double()[:, None] / 127 * 0.51 + plain.BF16 * 8
            assert ((held.cpu() - want_k[a + i]).abs() <= step.cpu()).all()
