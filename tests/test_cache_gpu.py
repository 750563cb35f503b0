"""The paged 8-bit cache on the GPU against the plain 64-bit forms: the page
plan and release exactly, the append code for code, the attention within
bounds derived from the roundings it makes (_cache_oracle.attend)."""
import random

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _cache_oracle as plain

pytestmark = pytest.mark.gpu
I8, F8 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# plan and release

def pool_state(ctx, width, page, extra, seed):
    """A table whose requests hold their pages, and the free stack."""
    rng = random.Random(seed)
    held = [-(-c // page) for c in ctx]
    order = list(range(sum(held) + extra))
    rng.shuffle(order)
    table = []
    for h in held:
        table.append([order.pop() for _ in range(h)] + [-1] * (width - h))
    return table, order


@pytest.mark.parametrize("new,ctx,page,slack", [
    ([1], [0], 16, 0),
    ([1] * 64, [37 * i % 200 for i in range(64)], 16, 0),
    ([0, 5, 0, 0, 33, 0], [16, 0, 0, 31, 32, 7], 16, 4),          # requests that bring nothing
    ([0, 0], [3, 0], 32, 3),                                      # a step without tokens
    ([700, 1, 64, 63, 65, 128], [0, 63, 64, 1, 127, 64], 64, 9),
    ([3000, 1, 4096], [5, 127, 0], 128, 100),
    ([i % 3 for i in range(1500)], [i % 50 for i in range(1500)], 16, 1),
])
def test_plan(new, ctx, page, slack):
    T = sum(new) + slack
    width = max(-(-(n + c) // page) for n, c in zip(new, ctx)) + 2
    need = sum(-(-(n + c) // page) + c // -page for n, c in zip(new, ctx))
    table, stack = pool_state(ctx, width, page, need + 3, 1)
    num = len(stack) + sum(-(-c // page) for c in ctx)
    want = plain.plan(new, ctx, table, stack, T, page, num)
    tab = ints(table)
    free = ints(stack + [-5] * (num - len(stack)))
    st = status()
    got = pkg.page_plan(ints(new), ints(ctx), tab, free, ints([len(stack)]), T, page, dev_status=st)
    assert st.item() == 0
    for g, w, name in zip((got.cu_seqlens, got.kv_lens, got.slots, got.positions, got.runs,
                           got.free_count, tab), want, "cu kv slots positions runs left table".split()):
        assert g.cpu().tolist() == (w if isinstance(w, list) else [w]), name


@pytest.mark.parametrize("new,ctx,left,T,code", [
    ([-1, 2], [4, 4], 8, 8, kda.KDA_ERR_BAD_SEQLENS),
    ([1, 2], [4, -4], 8, 8, kda.KDA_ERR_BAD_SEQLENS),
    ([4, 5], [4, 4], 8, 8, kda.KDA_ERR_BAD_SEQLENS),              # more tokens than rows
    ([1, 2], [4, 95], 8, 8, kda.KDA_ERR_BAD_SEQLENS),             # past the table row
    ([2 ** 31 - 1, 2], [2 ** 31 - 1, 4], 8, 8, kda.KDA_ERR_BAD_SEQLENS),
    ([20, 20], [12, 12], 1, 64, kda.KDA_ERR_NO_PAGES),
    ([20, 20], [12, 12], -1, 64, kda.KDA_ERR_NO_PAGES),
    ([20, 20], [12, 12], 1000, 64, kda.KDA_ERR_NO_PAGES),         # a count past the pool
])
def test_plan_takes_nothing_when_it_fails(new, ctx, left, T, code):
    tab = ints([[3] + [-1] * 5, [2] + [-1] * 5])
    before = tab.clone()
    st = status()
    got = pkg.page_plan(ints(new), ints(ctx), tab, ints([0, 1] + [4] * 6), ints([left]), T, 16,
                        dev_status=st)
    assert st.item() == code
    assert got.cu_seqlens.tolist() == [0, 0, 0] and got.kv_lens.tolist() == ctx
    assert (got.slots == -1).all() and (got.positions == -1).all() and (got.runs == 0).all()
    assert got.free_count.item() == left and torch.equal(tab, before)


def test_plan_reports_pages_outside_the_pool():
    tab = ints([[99, -1], [1, -1]])
    st = status()
    got = pkg.page_plan(ints([2, 2]), ints([4, 4]), tab, ints([0] * 4), ints([2]), 4, 16, dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_PAGES
    assert got.slots.tolist() == [-1, -1, 20, 21]
    assert got.runs.tolist()[:2] == [[0, 0, 0, 0], [2, 2, 1, 4]]


def test_release():
    page, ctx = 16, [33, 0, 16, 5, 100]
    table, stack = pool_state(ctx, 8, page, 4, 3)
    num = len(stack) + sum(-(-c // page) for c in ctx)
    rel = [1, 1, 0, 1, 0]
    want = list(stack)
    for r in range(5):
        if rel[r]:
            want += table[r][:-(-ctx[r] // page)]
    tab, lens = ints(table), ints(ctx)
    free, left = ints(stack + [-1] * (num - len(stack))), ints([len(stack)])
    st = status()
    pkg.page_release(ints(rel), lens, tab, free, left, page, dev_status=st)
    assert st.item() == 0 and left.item() == len(want)
    assert free[:len(want)].tolist() == want
    assert lens.tolist() == [0, 0, 16, 0, 100]
    for r in range(5):
        assert tab[r].tolist() == ([-1] * 8 if rel[r] else table[r])
    # a plan takes them back from the top
    got = pkg.page_plan(ints([17, 0, 0, 0, 0]), lens, tab, free, left, 17, page)
    assert tab[0].tolist()[:2] == [want[-1], want[-2]] and got.free_count.item() == len(want) - 2


def test_release_changes_nothing_when_it_fails():
    tab, lens = ints([[0, 1], [2, -1]]), ints([20, 4])
    free, left = ints([3, -1, -1, -1]), ints([3])
    st = status()
    pkg.page_release(ints([1, 1]), lens, tab, free, left, 16, dev_status=st)   # 3 + 3 pages > 4
    assert st.item() == kda.KDA_ERR_BAD_PAGES
    assert lens.tolist() == [20, 4] and left.item() == 3 and tab.tolist() == [[0, 1], [2, -1]]
    lens = ints([-3, 40])
    left = ints([1])
    pkg.page_release(ints([1, 1]), lens, tab, free, left, 16, dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_SEQLENS and left.item() == 1


# ---------------------------------------------------------------------------
# append

def fresh_pool(num, H, page, d, dtype):
    """A pool of junk: every byte 0x7f (a NaN in e4m3), NaN scales."""
    codes = torch.full((num, H, page, d), 0x7f, dtype=torch.uint8, device="cuda").view(dtype)
    return codes, torch.full((num, H), float("nan"), device="cuda")


def values(T, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, d, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))
    # exact ties: entries that are simple fractions of the largest magnitude
    x[:, :, :4] = x[:, :, 4:8].abs().amax() * torch.tensor([1.0, 0.5, -0.25, 0.125])
    return x.to(torch.bfloat16)


def check_codes(codes, want, name):
    got = codes.cpu().double()
    assert torch.equal(got, want), (name, (got != want).sum().item())


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("page,d,H", [(16, 64, 1), (32, 128, 3), (64, 128, 2), (128, 64, 5), (128, 128, 1)])
def test_append_matches_exact_arithmetic(dtype, page, d, H):
    # three steps: prompts, single tokens, odd pieces; every code equals the
    # formula's in exact arithmetic, held codes are requantised when a scale grows
    steps = [[page + 3, 1, 2 * page, 0], [1, 1, 1, 1], [5, page, page - 1, 2 * page + 1]]
    lens, R = [0] * 4, 4
    width = 8
    num = 40
    order = list(range(num))
    random.Random(5).shuffle(order)
    free, left = ints(order), ints([num])
    tab = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    kc, ks = fresh_pool(num, H, page, d, dtype)
    vc, vs = fresh_pool(num, H, page, d, dtype)
    grew = 0
    for i, new in enumerate(steps):
        T = sum(new)
        p = pkg.page_plan(ints(new), ints(lens), tab, free, left, T, page)
        k = values(T, H, d, 10 * i) * (1.0 + i)
        v = values(T, H, d, 10 * i + 1)
        runs = p.runs.tolist()
        want = [plain.append(x, runs, c.cpu(), s.cpu()) for x, c, s in ((k, kc, ks), (v, vc, vs))]
        before = ks.clone()
        # a view of a fused projection's output: its own token stride
        kv = torch.stack([k, v], 1).cuda()
        st = status()
        pkg.cache_append(kv[:, 0], kv[:, 1], p.runs, kc, vc, ks, vs, dev_status=st)
        assert st.item() == 0
        grew += int((ks > before).sum())
        for (c, s), (wc, ws), name in zip(((kc, ks), (vc, vs)), want, "kv"):
            assert torch.equal(s.cpu().double().nan_to_num(-1), ws.nan_to_num(-1))
            check_codes(c, wc.nan_to_num(0), name) if dtype == I8 else \
                check_codes(c.float().nan_to_num(0), wc.nan_to_num(0), name)
        lens, left = p.kv_lens.tolist(), p.free_count
    assert grew > 0


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("mag", [0.0, 1e-38, 3e-20, 1e20, 3e38])
def test_append_magnitudes(dtype, mag):
    # zeros, tiny and huge values: no overflow inside, codes as exact arithmetic has them
    g = torch.Generator().manual_seed(3)
    x = ((torch.rand(20, 2, 64, generator=g) - 0.5) * 2 * mag).to(torch.bfloat16)
    kc, ks = fresh_pool(3, 2, 16, 64, dtype)
    vc, vs = fresh_pool(3, 2, 16, 64, dtype)
    runs = [[0, 16, 2, 0], [16, 4, 0, 0]]
    pkg.cache_append(x.cuda(), x.cuda(), ints(runs), kc, vc, ks, vs)
    zero = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(dtype)
    wc, ws = plain.append(x, runs, zero, torch.zeros(3, 2))
    for pg, n in ((2, 16), (0, 4)):
        assert torch.equal(kc.cpu().double()[pg, :, :n], wc[pg, :, :n])
        assert torch.equal(ks.cpu().double()[pg], ws[pg])
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


def test_append_marks_pages_with_infinities_and_nans():
    x = torch.randn(8, 2, 64).to(torch.bfloat16).cuda()
    y = x.clone()
    y[3, 1, 7] = float("nan")
    y[2, 0, 9] = float("inf")
    kc, ks = fresh_pool(2, 2, 16, 64, I8)
    vc, vs = fresh_pool(2, 2, 16, 64, I8)
    pkg.cache_append(x, y, ints([[0, 8, 1, 0]]), kc, vc, ks, vs)
    assert ks[1].isfinite().all() and vs[1].isnan().all()
    pkg.cache_append(x, x, ints([[0, 2, 1, 8]]), kc, vc, ks, vs)     # stays marked
    assert vs[1].isnan().all() and ks[1].isfinite().all()
    pkg.cache_append(x, x, ints([[0, 8, 1, 0]]), kc, vc, ks, vs)     # until reused
    assert vs[1].isfinite().all() and torch.equal(vs[1], ks[1])


@pytest.mark.parametrize("run", [[0, 4, 2, 0], [0, 4, -1, 0], [0, 4, 0, 13], [0, 17, 0, 0],
                                 [5, 4, 0, 0], [-1, 2, 0, 0], [0, -2, 0, 0], [0, 2, 0, -1]])
def test_append_skips_runs_outside(run):
    x = torch.randn(8, 1, 64).to(torch.bfloat16).cuda()
    kc, ks = fresh_pool(2, 1, 16, 64, I8)
    vc, vs = fresh_pool(2, 1, 16, 64, I8)
    st = status()
    pkg.cache_append(x, x, ints([run, [0, 0, 0, 0]]), kc, vc, ks, vs, dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_PAGES
    assert (kc == 0x7f).all() and ks.isnan().all() and (vc == 0x7f).all()


# ---------------------------------------------------------------------------
# attention

def batch(new, ctx, page, H, G, d, dtype, seed, spare=3, width=0):
    """A filled cache over a pool of junk, the step's queries."""
    g = torch.Generator().manual_seed(seed)
    kv = [n + c for n, c in zip(new, ctx)]
    pages = [-(-x // page) for x in kv]
    num = sum(pages) + spare
    order = torch.randperm(num, generator=g).tolist()
    width = max(max(pages), 1) + width
    table, kc, vc = [], None, None
    junk = 0x7f
    kc, vc = (torch.full((num, H, page, d), junk, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.full((num, H), float("nan")) for _ in range(2))
    for x, n in zip(kv, pages):
        mine = [order.pop() for _ in range(n)]
        table.append(mine + [-1] * (width - n))
        for i, pg in enumerate(mine):
            m = min(page, x - i * page)
            for c, s in ((kc, ks), (vc, vs)):
                y = torch.randn(H, m, d, generator=g).clamp(-4, 4)
                a = y.abs().amax((1, 2), keepdim=True)
                y = y * (plain.TOP[dtype] / a)
                y = y.round().to(I8) if dtype == I8 else y.to(F8)
                c[pg, :, :m] = y.view(torch.uint8)
                # scales spread over a factor of 64, as outlier tokens make them
                s[pg] = (2.0 ** (6 * torch.rand(H, generator=g) - 2)).to(torch.bfloat16).float()
    ks *= 0.25
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(max(cu[-1], 1), H * G, d, generator=g)
    q = (q * torch.exp(torch.randn(q.shape[0], H * G, 1, generator=g))).to(torch.bfloat16)[:cu[-1]]
    return dict(q=q, cu=cu, kv=kv, table=table, kc=kc.view(dtype), vc=vc.view(dtype), ks=ks, vs=vs)


def call(b, scale=None, max_new=None, **kw):
    return pkg.cache_attend(b["q"].cuda(), ints(b["cu"]), ints(b["kv"]), ints(b["table"]),
                            b["kc"].cuda(), b["vc"].cuda(), b["ks"].cuda(), b["vs"].cuda(),
                            scale=scale, max_new=max_new, **kw)


def check(b, out, lse, scale=None):
    scale = b["q"].shape[-1] ** -0.5 if scale is None else scale
    o, l, to, tl = plain.attend(b["q"], b["cu"], b["kv"], b["table"], b["kc"], b["vc"], b["ks"],
                                b["vs"], scale)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert out.isfinite().all()
    none = l == -float("inf")
    assert torch.equal(lse == -float("inf"), none)
    eo = ((out - o).abs() - to).max() if out.numel() else 0
    assert eo <= 0, ("out", eo, ((out - o).abs() / to.clamp(min=1e-30)).max())
    el = ((lse - l).abs() - tl)[~none]
    assert not el.numel() or el.max() <= 0, ("lse", el.max())
    assert (out[none] == 0).all()


ONES = [1] * 5
SHAPES = [
    # (new, ctx, page, H, G): single tokens over lengths around the tiles' edges
    (ONES, [0, 1, 15, 16, 17], 16, 2, 4),
    (ONES, [30, 31, 32, 33, 62], 32, 1, 8),
    (ONES, [63, 64, 65, 126, 127], 64, 3, 5),
    (ONES, [127, 128, 129, 255, 256], 128, 2, 1),
    (ONES, [999, 1, 514, 40, 2000], 64, 2, 16),
    ([1], [0], 16, 1, 1),
    ([1, 1], [5000, 3], 16, 1, 6),
    # few tokens each (drafts), up to the few-row kernel's 16 rows and past it
    ([2, 3, 4, 1], [100, 5, 64, 0], 16, 2, 4),
    ([2, 2], [300, 1000], 64, 1, 8),
    ([5, 1, 3], [77, 1500, 12], 32, 2, 7),
    ([16, 1], [0, 0], 16, 3, 1),
    # groups of rows: up to 32 / 64 and past them, many parts and few
    ([5, 9, 20], [700, 33, 260], 32, 2, 3),
    ([7, 11, 2], [400, 90, 6000], 16, 1, 9),
    ([16, 8, 4, 1], [5000, 100, 64, 2000], 64, 2, 4),
    ([3] * 40, [50 * i for i in range(40)], 16, 4, 11),
    # prompts and pieces of prompts, odd lengths
    ([17], [0], 16, 1, 1),
    ([128], [0], 64, 1, 2),
    ([129, 1, 127], [0, 0, 0], 64, 2, 4),
    ([300, 45], [0, 513], 128, 1, 3),
    ([65, 200, 31], [1000, 0, 250], 32, 2, 12),
    ([400], [3000], 64, 1, 8),
    ([33], [40], 16, 1, 64),
    # a piece of a prompt among single tokens, requests that bring nothing
    ([1, 150, 0, 1, 1], [800, 90, 40, 0, 333], 16, 2, 6),
]


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "n%s-c%s-p%d-h%d-g%d" % (
    sum(s[0]), max(s[1]), s[2], s[3], s[4]))
def test_attend_matches_the_formula(shape, d, dtype):
    new, ctx, page, H, G = shape
    b = batch(new, ctx, page, H, G, d, dtype, seed=sum(ctx) + d + G)
    st = status()
    out, lse = call(b, max_new=max(new), dev_status=st)
    assert st.item() == 0
    check(b, out, lse)


@pytest.mark.parametrize("new,kv,G", [([4, 3], [2, 0], 2), ([40, 20, 1], [10, 0, 0], 4),
                                      ([200], [150], 3), ([300], [100], 1)])
def test_rows_that_see_nothing(new, kv, G):
    # more query rows than cached tokens: the first rows have no token to see
    b = batch([0] * len(new), kv, 16, 2, G, 64, F8, seed=7)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    b["cu"] = cu
    b["q"] = torch.randn(cu[-1], 2 * G, 64).to(torch.bfloat16)
    out, lse = call(b)
    check(b, out, lse)


@pytest.mark.parametrize("scale", [1.0, 0.02, -0.5, 0.0])
@pytest.mark.parametrize("new", [[1, 1], [40, 9]])
def test_other_scales(scale, new):
    b = batch(new, [200, 77], 32, 2, 4, 128, I8, seed=11)
    out, lse = call(b, scale=scale)
    check(b, out, lse, scale)


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 1, 20]])
def test_extreme_scores_and_queries(new):
    # scores of some hundreds, huge and tiny query rows: the maximum is taken out first
    b = batch(new, [500, 300, 64], 16, 1, 4, 64, I8, seed=13)
    b["q"][0] *= 60
    b["q"][-1] *= 2.0 ** -100
    b["q"][:, 1] = 0
    out, lse = call(b)
    check(b, out, lse)


@pytest.mark.parametrize("new", [[1, 1], [90, 1]])
def test_zero_pages_and_far_apart_scales(new):
    # a page of zeros (scale 0), value scales 2^-40 .. 2^40 apart
    b = batch(new, [200, 100], 16, 2, 4, 128, F8, seed=17)
    pg = b["table"][0][2]
    b["ks"][pg] = 0
    b["vs"][pg] = 0
    b["kc"].view(torch.uint8)[pg] = 0
    b["vc"].view(torch.uint8)[pg] = 0
    b["vs"][b["table"][0][5]] *= 2.0 ** 40
    b["vs"][b["table"][0][0]] *= 2.0 ** -40
    out, lse = call(b)
    check(b, out, lse)


@pytest.mark.parametrize("new", [[1, 1], [90, 20]])
def test_marked_page_reaches_only_those_who_see_it(new):
    b = batch(new, [200, 100], 16, 2, 4, 64, I8, seed=19)
    b["vs"][b["table"][0][1], 1] = float("nan")
    out, lse = call(b)
    n = new[0]
    assert out[:n, 4:].isnan().all() and out[:n, :4].isfinite().all()
    assert out[n:].isfinite().all()


@pytest.mark.parametrize("n,G", [(4, 4), (90, 2), (90, 8)])
@pytest.mark.parametrize("dtype", [I8, F8])
def test_marked_page_of_later_tokens_stays_unseen(n, G, dtype):
    # the last page, of new tokens only, is marked: queries before it are untouched
    page, ctx = 16, 48 - n % 16 + 2
    b = batch([n], [ctx], page, 1, G, 64, dtype, seed=53)
    clean, clean_lse = call(b)
    first = (ctx + n - 1) // page * page - ctx      # the first new token in the last page
    pg = b["table"][0][(ctx + n - 1) // page]
    b["vs"][pg] = float("nan")
    b["ks"][pg] = float("nan")
    out, lse = call(b)
    assert torch.equal(out[:first], clean[:first]) and torch.equal(lse[:first], clean_lse[:first])
    assert out[first:].isnan().all() and lse[first:].isnan().all()


@pytest.mark.parametrize("big", [2.0 ** 60, float("inf")])
@pytest.mark.parametrize("n,G,d", [(4, 2, 128), (8, 1, 64), (4, 4, 64), (9, 7, 128), (90, 2, 64),
                                   (150, 5, 128), (600, 1, 64)])
@pytest.mark.parametrize("dtype", [I8, F8])
def test_scales_of_later_pages_stay_unseen(n, G, d, dtype, big):
    # the pages that hold the later half of the new tokens have enormous scales:
    # what does not see them stays within the bounds that hold without them
    page, ctx = 16, 48 - n // 2 % 16
    b = batch([n], [ctx], page, 1, G, d, dtype, seed=59)
    o, l, to, tl = plain.attend(b["q"], b["cu"], b["kv"], b["table"], b["kc"], b["vc"], b["ks"],
                                b["vs"], d ** -0.5)
    col = (ctx + n // 2) // page
    first = col * page - ctx                         # the first new token in such a page
    assert 0 < first < n
    for pg in b["table"][0][col:]:
        b["vs"][pg] = big
        b["ks"][pg] = big
    out, lse = call(b)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert ((out - o).abs() <= to)[:first].all()
    assert ((lse - l).abs() <= tl)[:first].all()


@pytest.mark.parametrize("new", [[1] * 7, [30, 1, 70]])
def test_token_stride_other_stream_and_no_lse(new):
    b = batch(new, [50 + 60 * i for i in range(len(new))], 64, 2, 4, 128, I8, seed=23)
    T, Hq, d = b["q"].shape
    wide = torch.randn(T, Hq + 3, d).to(torch.bfloat16).cuda()
    wide[:, 1:Hq + 1] = b["q"].cuda()
    want = call(b)
    dev = dict(cu=ints(b["cu"]), kv=ints(b["kv"]), table=ints(b["table"]))
    pools = [b[k].cuda() for k in ("kc", "vc", "ks", "vs")]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pkg.cache_attend(wide[:, 1:Hq + 1], dev["cu"], dev["kv"], dev["table"], *pools, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # no lse, the library's own workspace
    out = torch.empty_like(got[0])
    kc = pools[0]
    rc = kda.kda_cache_attn(wide[:, 1:Hq + 1], wide.stride(0), dev["cu"], dev["kv"], dev["table"],
                            dev["table"].shape[1], *pools, out, None, len(new), T, T, Hq, 2, d,
                            kc.shape[0], kc.shape[2], kda.KDA_I8, d ** -0.5, None, 0, None,
                            torch.cuda.current_stream())
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(out, got[0])


def test_padding_rows_are_left_alone_and_results_repeat():
    b = batch([1, 40, 2], [700, 20, 3000], 32, 2, 4, 128, F8, seed=29)
    first = call(b)
    for _ in range(3):
        again = call(b)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    T, Hq, d = b["q"].shape
    q = torch.cat([b["q"], torch.full((9, Hq, d), float("nan")).to(torch.bfloat16)]).cuda()
    out = torch.full((T + 9, Hq, d), 5.0).to(torch.bfloat16).cuda()
    lse = torch.full((T + 9, Hq), 5.0, device="cuda")
    tab = ints(b["table"])
    rc = kda.kda_cache_attn(q, q.stride(0), ints(b["cu"]), ints(b["kv"]), tab, tab.shape[1],
                            b["kc"].cuda(), b["vc"].cuda(), b["ks"].cuda(), b["vs"].cuda(), out, lse,
                            3, T + 9, T + 9, Hq, 2, d, b["kc"].shape[0], 32, kda.KDA_E4M3, d ** -0.5,
                            None, 0, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(out[:T], first[0]) and torch.equal(lse[:T], first[1])
    assert (out[T:] == 5).all() and (lse[T:] == 5).all()


@pytest.mark.parametrize("change,code", [
    (dict(cu=[0, 3, 2]), kda.KDA_ERR_BAD_SEQLENS), (dict(cu=[0, 1, 9]), kda.KDA_ERR_BAD_SEQLENS),
    (dict(kv=[-1, 40]), kda.KDA_ERR_BAD_SEQLENS), (dict(kv=[40, 4000]), kda.KDA_ERR_BAD_SEQLENS),
    (dict(bad_page=-1), kda.KDA_ERR_BAD_PAGES), (dict(bad_page=10 ** 6), kda.KDA_ERR_BAD_PAGES)])
@pytest.mark.parametrize("new", [[1, 1], [40, 60]])
def test_malformed_batches_are_reported(change, code, new):
    b = batch(new, [39, 39], 16, 2, 4, 64, I8, seed=31)
    if "bad_page" in change:
        b["table"][1][1] = change["bad_page"]
    else:
        b |= change
        if new[0] > 1 and "cu" in change:
            b["cu"] = [x * 30 for x in b["cu"]]
    st = status()
    call(b, dev_status=st)
    assert st.item() == code


def test_max_new_too_small_is_reported():
    b = batch([1, 5], [9, 9], 16, 2, 4, 64, I8, seed=37)
    st = status()
    call(b, max_new=4, dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_SEQLENS


def test_pool_past_32_bits():
    # a pool of over 4 GiB each, the request's pages at its end
    H, page, d, num = 8, 128, 128, 34000
    b = batch([1, 20], [300, 700], page, H, 2, d, I8, seed=41)
    used = b["kc"].shape[0]
    kc, vc = (torch.empty(num, H, page, d, dtype=I8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(num, H, device="cuda") for _ in range(2))
    for big, name in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
        big[num - used:] = b[name].cuda()
    tab = ints(b["table"])
    tab = torch.where(tab >= 0, tab + num - used, tab)
    out, lse = pkg.cache_attend(b["q"].cuda(), ints(b["cu"]), ints(b["kv"]), tab, kc, vc, ks, vs)
    check(b, out, lse)
    # and the append reaches it
    x = torch.randn(4, H, d).to(torch.bfloat16)
    pkg.cache_append(x.cuda(), x.cuda(), ints([[0, 4, num - 1, 0]]), kc, vc, ks, vs)
    wc, ws = plain.append(x, [[0, 4, 0, 0]], torch.zeros(1, H, page, d, dtype=I8), torch.zeros(1, H))
    assert torch.equal(kc[num - 1, :, :4].cpu().double(), wc[0, :, :4])
    assert torch.equal(vs[num - 1].cpu().double(), ws[0])


def test_long_context_single_token():
    b = batch([1, 1], [70000, 31], 128, 1, 8, 64, I8, seed=43)
    out, lse = call(b, max_new=1)
    check(b, out, lse)


def test_whole_step_in_a_graph():
    # plan, append and attention captured once, replayed after the inputs change
    page, H, G, d, R, width, num = 16, 2, 4, 64, 4, 8, 40
    new, ctx = ints([1] * R), ints([0, 15, 16, 40])
    table, stack = pool_state([0, 15, 16, 40], width, page, num - 6, 3)
    tab, free, left = ints(table), ints(stack + [-1] * (num - len(stack))), ints([len(stack)])
    kc, ks = fresh_pool(num, H, page, d, F8)
    vc, vs = fresh_pool(num, H, page, d, F8)
    x = torch.randn(60, H, d).to(torch.bfloat16).cuda()
    for r, n in enumerate([0, 15, 16, 40]):
        runs = [[i, min(page, n - i), table[r][i // page], 0] for i in range(0, n, page)]
        if runs:
            pkg.cache_append(x, -x, ints(runs), kc, vc, ks, vs)
    k, v = (torch.randn(R, H, d).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(R, H * G, d).to(torch.bfloat16).cuda()

    def step():
        p = pkg.page_plan(new, ctx, tab, free, left, R, page)
        pkg.cache_append(k, v, p.runs, kc, vc, ks, vs)
        return p, pkg.cache_attend(q, p.cu_seqlens, p.kv_lens, tab, kc, vc, ks, vs, max_new=1)
    saved = [t.clone() for t in (tab, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]

    def restore():
        for t, s in zip((tab, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), saved):
            t.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, (out, lse) = step()
    for seed in range(2):
        torch.manual_seed(seed)
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape).to(torch.bfloat16))
        restore()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        restore()
        want = step()[1]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        b = dict(q=q.cpu(), cu=p.cu_seqlens.tolist(), kv=p.kv_lens.tolist(), table=tab.tolist(),
                 kc=kc.cpu(), vc=vc.cpu(), ks=ks.cpu(), vs=vs.cpu())
        check(b, *got)
