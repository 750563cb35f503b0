"""Attention over long contexts in the paged 8-bit cache, against 64 bits, by
bounds that follow the output's own size.

Many requests share one context's pages, so that a worker of the kernels takes
whole contexts and sums over all of their tokens by itself.  Scores are near each
other, so every token counts.  Beside the output's rounding to bf16 the kernels
may err, relative to the checked rows' L2 norm and in quadrature (the sources
are independent), by

    f16 weights    2^-11 / sqrt(3) of each term, at most that of the sum: 2.8e-4
    fp32 sums      2^-24 of the sum on the average for each of a run's additions,
                   always in one direction; runs of at most 2^16 tokens, 16 an
                   addition: 2.4e-4

which is 3.7e-4.  Rounding brings a value x + e no further from x than the
rounding of x is, and twice e: so the output's error is at most that of the exact
output rounded to bf16 and 7.4e-4.

The errors' common direction is taken against the exact output rounded to bf16:
the kernels' outputs differ from that where their errors, 5.2e-4 of the output
at most together, carry a value over a rounding's edge, by a unit of 2^-7 at
most, which has a variance of 5.2e-4 * 2^-7 in each of n independent values.
The mean may hold the fp32 sums' 2.4e-4 and six deviations.  n counts heads and
channels (the rows checked see nearly the same weights), and the values' spread
weighs larger ones more, by 1.25 for normal ones.
"""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests.test_cache_gpu import batch, call, check as within

pytestmark = pytest.mark.gpu
I8, F8 = torch.int8, torch.float8_e4m3fn
TOP = {I8: 127.0, F8: 448.0}
H, G, PAGE = 8, 4, 128


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def pool(pages, d, dtype, one_sign, gen):
    x = torch.randn(pages, H, PAGE, d, generator=gen, device="cuda")
    if one_sign:
        x = x.abs() + 0.5
    x = x * (TOP[dtype] / x.abs().amax((2, 3), keepdim=True))
    return (x.round() if dtype == I8 else x).to(dtype)


def values(codes, scale, h):
    """[tokens, d] in 64 bits of a head of all pages."""
    x = codes.view(torch.uint8)[:, h].contiguous().view(codes.dtype).float().double()
    return (x * (scale[:, h].double() / TOP[codes.dtype])[:, None, None]).reshape(-1, codes.shape[-1])


def errors(L, d, dtype, new, one_sign, R=None):
    """(relative L2 error, that of the exact output rounded to bf16, mean signed error
    against the latter, independent values checked, lse error)"""
    gen = torch.Generator(device="cuda").manual_seed(L + d)
    # contexts longer than the pool go through it again
    pages = min(L // PAGE, 2048)
    kc, vc = pool(pages, d, dtype, False, gen), pool(pages, d, dtype, one_sign, gen)
    ks, vs = (3 + torch.rand(pages, H, generator=gen, device="cuda") for _ in range(2))
    R = R or (64 if new == 1 else 19)
    cols = torch.arange(L // PAGE, device="cuda") % pages
    table = cols.to(torch.int32).repeat(R, 1).contiguous()
    ints = {"dtype": torch.int32, "device": "cuda"}
    cu, kv = torch.arange(R + 1, **ints) * new, torch.full((R,), L, **ints)
    q = (0.3 * torch.randn(R * new, H * G, d, generator=gen, device="cuda")).to(torch.bfloat16)
    status = torch.full((1,), 77, **ints)
    out, lse = pkg.cache_attend(q, cu, kv, table, kc, vc, ks, vs, max_new=new, dev_status=status)
    assert status.item() == 0
    e2 = b2 = x2 = signed = size = le = 0
    for h in range(H):
        k, v = values(kc, ks, h), values(vc, vs, h)
        for row in (0, R * new // 2 + new // 3, R * new - 1):
            seen = L - new + row % new + 1
            o = torch.zeros(G, d, dtype=torch.float64, device="cuda")
            s = (q[row, h * G:(h + 1) * G].double() @ k.T) * d ** -0.5      # of the pool's tokens
            m = s.amax(-1, keepdim=True)
            w = torch.exp(s - m)
            # how often the context goes over each token of the pool
            times = torch.zeros(pages * PAGE, dtype=torch.float64, device="cuda")
            times += seen // (pages * PAGE)
            times[: seen % (pages * PAGE)] += 1
            w = w * times
            total = w.sum(-1, keepdim=True)
            o = (w / total) @ v
            e = out[row, h * G:(h + 1) * G].double() - o
            e2, x2 = e2 + e.square().sum().item(), x2 + o.square().sum().item()
            best = o.to(torch.bfloat16).double()
            b2 += (best - o).square().sum().item()
            flips = out[row, h * G:(h + 1) * G].double() - best
            signed, size = signed + flips.sum().item(), size + o.abs().sum().item()
            want = (m + total.log())[:, 0]
            le = max(le, (lse[row, h * G:(h + 1) * G].double() - want).abs().max().item())
    return math.sqrt(e2 / x2), math.sqrt(b2 / x2), abs(signed / size), H * d, le


def check(rms, best, mean, n, le):
    assert rms <= best + 7.4e-4
    assert mean <= 2.4e-4 + 6 * math.sqrt(1.25 * 5.2e-4 * 2.0 ** -7 / n)
    assert le <= 2.0 ** -17


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [4096, 32768, 131072])
def test_decode_steps_of_long_contexts(L, d, dtype, one_sign):
    check(*errors(L, d, dtype, 1, one_sign))


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [32768, 131072])
def test_pieces_of_prompts_on_long_contexts(L, d, dtype, one_sign):
    check(*errors(L, d, dtype, 128, one_sign))


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("L,new,R", [(1 << 20, 1, 64), (1 << 20, 128, 19),   # whole contexts a worker
                                     (1 << 23, 1, 1), (1 << 21, 70, 1)])     # shared among workers
def test_contexts_of_a_million_tokens(L, new, R, dtype, one_sign):
    check(*errors(L, 64, dtype, new, one_sign, R))


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("new", [[1, 1], [90, 3]])
def test_huge_queries_meet_tiny_keys(dtype, new):
    # 2^110 and 2^-110: the scores are ordinary
    b = batch(new, [200, 100], 16, 2, 4, 64, dtype, seed=61)
    b["q"] *= 2.0 ** 110
    b["ks"] *= 2.0 ** -110
    within(b, *call(b))
