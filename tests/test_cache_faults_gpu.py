"""Faulty tables, lengths and statuses of the paged 8-bit cache: what is found on
the device is reported and leaves nothing half done."""
import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests.test_cache_gpu import ints, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("row,col", [(0, 0), (0, 2), (2, 1)])
def test_release_refuses_pages_outside_the_pool(bad, row, col):
    # a faulty page must not reach the free stack, from where a plan would hand it out
    table = [[0, 1, 2], [3, -1, -1], [4, 5, -1]]
    table[row][col] = bad
    tab, lens = ints(table), ints([40, 16, 17])
    free, left = ints([6, 7] + [-1] * 6), ints([2])
    st = status()
    pkg.page_release(ints([1, 0, 1]), lens, tab, free, left, 16, dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_PAGES
    assert tab.tolist() == table and lens.tolist() == [40, 16, 17]
    assert left.item() == 2 and free.tolist() == [6, 7] + [-1] * 6
    # the other requests still leave
    pkg.page_release(ints([int(r != row) for r in range(3)]), lens, tab, free, left, 16, dev_status=st)
    assert st.item() == 0
    held = [(40, 3), (16, 1), (17, 2)]
    assert left.item() == 2 + sum(n for r, (_, n) in enumerate(held) if r != row)
    assert lens.tolist() == [t if r == row else 0 for r, (t, _) in enumerate(held)]
    assert all(0 <= x < 8 for x in free[:left.item()].tolist())


def test_release_of_a_request_without_pages_reads_no_table():
    tab, lens = ints([[-7, -7], [9, -7]]), ints([0, 3])
    free, left = ints([0, 1, 2, 3]), ints([4])
    st = status()
    pkg.page_release(ints([1, 0]), lens, tab, free, left, 16, dev_status=st)
    assert st.item() == 0 and left.item() == 4 and tab.tolist() == [[-7, -7], [9, -7]]


def attend(cu, kv, T, max_new):
    H, page, d = 2, 16, 64
    c = torch.zeros(4, H, page, d, dtype=torch.int8, device="cuda")
    s = torch.ones(4, H, device="cuda")
    q = torch.ones(T, 2 * H, d, device="cuda").to(torch.bfloat16)
    st = status()
    table = ints([[i % 4, 1] for i in range(len(kv))])
    pkg.cache_attend(q, ints(cu), ints(kv), table, c, c.clone(), s, s.clone(), max_new=max_new,
                     dev_status=st)
    return st.item()


@pytest.mark.parametrize("cu,kv,T,max_new,code", [
    ([0, 1, 1], [5, 3], 1, 0, kda.KDA_ERR_BAD_SEQLENS),    # a request with more than max_new tokens
    ([0, 3, 5], [5, 3], 5, 0, kda.KDA_ERR_BAD_SEQLENS),
    ([0, 0, 0], [5, 33], 4, 0, kda.KDA_ERR_BAD_SEQLENS),   # past the table
    ([0, 0, 0], [-1, 3], 4, 0, kda.KDA_ERR_BAD_SEQLENS),
    ([0, 0, -1], [5, 3], 4, 0, kda.KDA_ERR_BAD_SEQLENS),
    ([0, 0, 0], [5, 32], 4, 0, 0),                         # rows of no request: nothing to do
    ([0, 0, 1], [5, 3], 0, 1, kda.KDA_ERR_BAD_SEQLENS),    # more tokens than rows
    ([0, 0, 0], [5, 40], 0, 0, kda.KDA_ERR_BAD_SEQLENS),
    ([0, 0, 0], [5, 3], 0, 0, 0),
    ([0] * 3001, [7] * 2999 + [-2], 0, 0, kda.KDA_ERR_BAD_SEQLENS),
])
def test_steps_without_tokens_are_checked_too(cu, kv, T, max_new, code):
    assert attend(cu, kv, T, max_new) == code


@pytest.mark.parametrize("run,code", [([0, 1, 0, 0], kda.KDA_ERR_BAD_PAGES), ([0, 0, 0, 0], 0),
                                      ([0, -1, 0, 0], kda.KDA_ERR_BAD_PAGES)])
def test_runs_of_an_append_without_rows_are_checked_too(run, code):
    c = torch.full((2, 1, 16, 64), 3, dtype=torch.int8, device="cuda")
    s = torch.ones(2, 1, device="cuda")
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    st = status()
    v, vs = c.clone(), s.clone()
    pkg.cache_append(x, x, ints([run, [0, 0, 0, 0]]), c, v, s, vs, dev_status=st)
    assert st.item() == code
    assert (c == 3).all() and (v == 3).all() and (s == 1).all() and (vs == 1).all()


@pytest.mark.parametrize("bad", ["cpu", "int64", "empty", "float"])
def test_a_status_that_is_no_int32_on_the_device_is_refused(bad):
    # a kernel would write to the host's address, or past the element
    st = {"cpu": torch.zeros(1, dtype=torch.int32),
          "int64": torch.zeros(1, dtype=torch.int64, device="cuda"),
          "empty": torch.zeros(0, dtype=torch.int32, device="cuda"),
          "float": torch.zeros(1, device="cuda")}[bad]
    one, lens = ints([1]), ints([0])
    tab, free, left = ints([[-1, -1]]), ints([0, 1]), ints([2])
    c = torch.zeros(2, 1, 16, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(2, 1, device="cuda")
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for f, a in ((pkg.page_plan, (one, lens, tab, free, left, 1, 16)),
                 (pkg.page_release, (one, lens, tab, free, left, 16)),
                 (pkg.cache_append, (x, x, ints([[0, 1, 0, 0]]), c, c.clone(), s, s.clone())),
                 (pkg.cache_attend, (x, ints([0, 1]), one, ints([[0, 1]]), c, c.clone(), s, s.clone()))):
        with pytest.raises(ValueError, match="dev_status"):
            f(*a, dev_status=st)
    assert left.item() == 2 and (tab == -1).all() and (c == 0).all() and (s == 0).all()
