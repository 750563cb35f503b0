"""Waits of the tensor-core kernel of linear attention answer for a whole warp:
what follows them (tensor memory's loads and stores, shuffles, products) is not
defined for a part of one, and where a wait gives up some threads may have seen
its phase and others not.  Checked in the source: it shows in no result until
it does.  CPU only."""
import os
import re

import gated_delta_rule_32_gb300

CSRC = os.path.join(os.path.dirname(gated_delta_rule_32_gb300.__file__), "csrc")


def kernel():
    with open(os.path.join(CSRC, "kda_linear_tile.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text[text.index("kda_linear_tile_kernel("):text.index("kda_linear_scan_kernel(")]


def test_waits_are_voted_on():
    body = kernel()
    assert len(re.findall(r"\bwait\(&bars\.", body)) > 10
    calls = re.findall(r"(\S*\s*\S*)bounded_wait\(", body)
    assert calls == ["__all_sync(~0u, "], calls


def test_nothing_but_the_copies_ends_waits_for_itself():
    # (behind each of the two is only the block's own barrier)
    body = kernel()
    others = re.findall(r"mbar_(?:try_)?wait\(&bars\.(\w+)", body)
    assert sorted(others) == ["drain", "qk_full", "v_full"]
