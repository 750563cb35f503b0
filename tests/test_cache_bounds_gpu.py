"""Attention over the paged 8-bit cache against 64 bits by bounds that follow
each row's own sums (_cache_bounds): long contexts, many requests, references
and value scales that are passed again and again."""
import pytest
import torch

from gated_delta_rule_32_gb300 import kda
from tests import _cache_bounds as exact
from tests.test_cache_gpu import F8, I8, batch, call, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def check(b, max_new=None, tight=0.02):
    """`tight`: the bound's norm relative to the output's at most, so that it can fail."""
    st = status()
    out, lse = call(b, max_new=max(b["new"]) if max_new is None else max_new, dev_status=st)
    assert st.item() == 0
    o, l, to, tl = exact.attend(b["q"], b["cu"], b["kv"], b["table"], b["kc"], b["vc"], b["ks"],
                                b["vs"], b["q"].shape[-1] ** -0.5)
    out, lse = out.cpu().double(), lse.cpu().double()
    none = l == -float("inf")
    assert torch.equal(lse == -float("inf"), none) and (out[none] == 0).all()
    assert ((out - o).abs() <= to).all(), ((out - o).abs() / to.clamp(min=1e-300)).max()
    assert ((lse - l).abs() <= tl)[~none].all()
    assert to.norm() <= tight * o.norm()


def made(new, ctx, page, H, G, d, dtype, seed):
    return batch(new, ctx, page, H, G, d, dtype, seed) | {"new": new}


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,ctx,page,H,G", [
    ([1, 1], [5000, 3], 16, 1, 6),
    ([1] * 5, [999, 1, 514, 40, 2000], 64, 2, 16),
    ([5, 1, 3], [77, 1500, 12], 32, 2, 7),
    ([7, 11, 2], [400, 90, 6000], 16, 1, 9),
    ([16, 8, 4, 1], [5000, 100, 64, 2000], 64, 2, 4),
    ([65, 200, 31], [1000, 0, 250], 32, 2, 12),
    ([400], [3000], 64, 1, 8),
    ([1, 150, 0, 1, 1], [800, 90, 40, 0, 333], 16, 2, 6),
])
def test_ordinary_batches(new, ctx, page, H, G, d, dtype):
    check(made(new, ctx, page, H, G, d, dtype, seed=sum(ctx) + d + G))


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,ctx", [([1, 1], [70000, 31]), ([2, 1], [40000, 33001]), ([40, 3], [70001, 9])])
def test_long_contexts(new, ctx, d, dtype):
    check(made(new, ctx, 128, 1, 8, d, dtype, seed=43 + d))


def requests(R, prompts, every):
    """Single tokens, `every`-th request without any, and prompts at some rows."""
    new = [0 if i % every == 3 else 1 for i in range(R)]
    ctx = [(37 * i) % 61 for i in range(R)]
    for at, n in prompts:
        new[at] = n
    return new, ctx


@pytest.mark.parametrize("dtype,R,prompts,H,G,d", [
    (I8, 300, [(5, 90), (150, 33), (299, 120)], 2, 5, 128),
    (F8, 300, [(0, 70)], 1, 16, 64),
    (F8, 1500, [(5, 90), (6, 300), (700, 65), (1499, 90)], 1, 4, 64),
    (I8, 1500, [], 2, 3, 64),
    (I8, 2000, [(i, 40) for i in range(0, 2000, 97)], 1, 2, 128),
])
def test_many_requests(dtype, R, prompts, H, G, d):
    new, ctx = requests(R, prompts, 7)
    check(made(new, ctx, 16, H, G, d, dtype, seed=R + G))


@pytest.mark.parametrize("dtype,G", [(I8, 2), (F8, 48)])
def test_most_requests_bring_nothing(dtype, G):
    new = [(1, 2, 5)[i // 61 % 3] if i % 61 == 0 else 0 for i in range(16384)]
    ctx = [20 if n else 0 for n in new]
    new[16000] = 70
    check(made(new, ctx, 16, 1, G, 64, dtype, seed=5))


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("span", [60.0, 700.0, -60.0, -700.0])
@pytest.mark.parametrize("new,ctx,d", [([1], [3000], 64), ([1, 2], [30000, 500], 128), ([60], [2500], 64),
                                       ([100, 1], [20000, 700], 128), ([3], [120000], 64),
                                       ([60], [150000], 64)])
def test_scores_and_value_scales_that_rise_or_fall_along_the_context(new, ctx, d, span, dtype):
    # scores change by `span` from the first page to the last, value scales by a
    # factor of 2^20 the same way: references and scales are passed all the time
    b = made(new, ctx, 64, 2, 4, d, dtype, seed=71)
    raw = b["kc"].view(torch.uint8)
    raw[..., 0] = 127 if dtype == I8 else 0x7e          # the top code: its value is the scale
    b["q"][..., 0] = 64.0
    for row in b["table"]:
        pages = [pg for pg in row if pg >= 0]
        at = torch.arange(len(pages)) / max(1, len(pages) - 1)
        up = at if span > 0 else 1 - at
        # (channel 0 alone gives 64 * scale * key scale)
        b["ks"][pages] = (0.05 + up * abs(span) / (64 * d ** -0.5))[:, None].to(torch.bfloat16).float()
        b["vs"][pages] = torch.exp2(20 * up - 10)[:, None].to(torch.bfloat16).float()
    raw[..., 1:] = raw[..., 1:] & (0x03 if dtype == I8 else 0x9f)  # the other channels: small
    check(b, tight=0.1)
