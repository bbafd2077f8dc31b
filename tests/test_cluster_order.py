"""Blocks of a cluster tell one another through mbarriers that shared memory has been written. What such a
report orders must hold at cluster scope: an mbarrier arrival without a scope has the block's own, and
orders nothing for a thread of another block. Read from the sources (a wrong order does not show in a
run on hardware that happens to keep it)."""
import glob
import os
import re

from tests._util import ROOT


def sources():
    for path in sorted(glob.glob(os.path.join(ROOT, "weight_quantized_gemm_gb300", "csrc", "*.cu*"))):
        yield os.path.basename(path), re.sub(r"//[^\n]*", "", open(path).read())


def test_arrivals_at_other_blocks_name_the_cluster_scope():
    seen = 0
    for name, src in sources():
        for ins in re.findall(r"mbarrier\.arrive[\w.:]*", src):
            if "shared::cluster" in ins:
                seen += 1
                assert ".cluster.shared::cluster" in ins, f"{name}: {ins}"
    assert seen


def test_scales_are_released_to_the_cluster_before_they_are_reported():
    src = dict(sources())["group_gemm.cuh"]
    assert re.search(r"fence\.release\.sync_restrict::shared::cta\.cluster|mbarrier\.arrive\.release\.cluster\.shared::cluster", src)
    reports = re.findall(r"([^\n;{]*[;{])\s*(peer_arrive\(lead\(full\(s\)\)\))", src)
    assert reports
    for before, _ in reports:
        assert "release_shared()" in before


def test_waits_for_other_blocks_acquire_at_cluster_scope():
    src = dict(sources())["group_gemm.cuh"]
    waits = re.findall(r"mbarrier\.(?:try|test)_wait[\w.:]*", src)
    assert waits and all("acquire.cluster" in w for w in waits)
