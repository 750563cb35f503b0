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
