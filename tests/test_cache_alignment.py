"""Pointers of the paged 8-bit cache's entry points that are not aligned to
their elements are refused before anything is queued (a kernel would fault on
them).  CPU only: the addresses are made up."""
import pytest

from gated_delta_rule_32_gb300 import kda
from tests.test_cache_abi import A, _append, _attn, _plan, _release, lib  # noqa: F401


@pytest.mark.parametrize("call,name,at", [
    (c, n, i + 1) for c, ns in (
        (_plan, "new_lens ctx_lens block_table free_pages free_count cu_seqlens kv_lens slots "
                "positions runs free_count_out dev_status"),
        (_release, "release kv_lens block_table free_pages free_count dev_status"),
        (_append, "k v runs k_codes v_codes k_scale v_scale dev_status"),
        (_attn, "q cu_seqlens kv_lens block_table k_codes v_codes k_scale v_scale out lse dev_status"))
    for i, n in enumerate(ns.split())])
@pytest.mark.parametrize("off", [1, 2])
def test_misaligned_pointers(call, name, at, off):
    # (addresses of their own, far from the others')
    assert call(**{name: (40 + at) * A + off}) == kda.KDA_ERR_MISALIGNED
