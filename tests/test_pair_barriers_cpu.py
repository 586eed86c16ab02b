"""Barriers that a pair of blocks shares: by the memory model an arrival or a wait whose scope is one block orders nothing
between two, so every one that names another block's barrier, and every wait, has cluster scope in the source."""

import os
import re

from combine_get_layout_02_b200 import build as cbuild

with open(os.path.join(cbuild.CSRC, "matmul_mxfp4.cu")) as f:
    SOURCE = f.read()


def _asm(op):
    return re.findall(r'"[^"]*?(mbarrier\.' + op + r'[^ "]*) ', SOURCE)


def test_arrivals_at_another_blocks_barrier_have_cluster_scope():
    remote = [i for i in _asm("arrive") if ".shared::cluster" in i]
    assert remote and all(re.search(r"\.(relaxed|release)\.cluster\.shared::cluster", i) for i in remote), remote


def test_waits_have_cluster_scope():
    waits = _asm("try_wait") + _asm("test_wait")
    assert len(waits) >= 2 and all(re.search(r"\.(relaxed|acquire)\.cluster\.", i) for i in waits), waits


def test_relaxed_operations_stand_with_their_fences():
    """What passes through shared memory: a release fence before the arrival, an acquire fence after a wait or a test."""
    body = re.search(r"void bar_arrive_smem\(.*?\n}", SOURCE, re.S).group()
    assert body.index("fence.release.sync_restrict::shared::cta.cluster") < body.index("mbarrier.arrive.relaxed.cluster")
    wait = re.search(r"bool bar_wait\(.*?\n}", SOURCE, re.S).group()
    assert wait.index("fence_acquire_smem();") < wait.index("return true;") and wait.count("return true;") == 1
    assert "fence.acquire.sync_restrict::shared::cluster.cluster" in SOURCE
    assert re.search(r"= bar_test\([^;]*;\s*fence_acquire_smem\(\);", SOURCE)
    assert re.search(r"fence_proxy_async\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) bar_arrive_smem\(", SOURCE)
