"""Barriers that two CTAs share order memory between them only with the cluster
as their scope; the default scope is one CTA.  Checked in the source: a missing
scope shows in no result until it does.  CPU only."""
import glob
import os
import re

import gated_delta_rule_32_gb300

CSRC = os.path.join(os.path.dirname(gated_delta_rule_32_gb300.__file__), "csrc")


def instructions(name):
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for found in re.findall(r"%s[\w.:]*" % re.escape(name), f.read()):
                yield os.path.basename(path), found


def test_arrivals_at_another_cta_have_the_cluster_as_scope():
    remote = [(f, x) for f, x in instructions("mbarrier.arrive.") if "shared::cluster" in x]
    assert remote
    for f, x in remote:
        assert ".release.cluster." in x or ".relaxed.cluster." in x, (f, x)


def test_the_kernel_of_cta_pairs_waits_with_a_scope():
    waits = [x for f, x in instructions("mbarrier.try_wait.") if f == "kda_cache_tile.cu"]
    assert any(".acquire.cluster." in x for x in waits)
    for x in waits:
        assert re.search(r"\.(acquire|relaxed)\.(cta|cluster)\.", x), x


def test_the_kernel_of_cta_pairs_hands_operands_over_with_a_release():
    # what generic writes put into shared memory for the other CTA's products
    # needs more than execution order: one release to the cluster on its way
    with open(os.path.join(CSRC, "kda_cache_tile.cu")) as f:
        assert "mbarrier.arrive.release.cluster.shared::cluster" in f.read()
