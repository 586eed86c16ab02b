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


def _arrivals_left(fills, slots, tail):
    """Arrivals at one block's ring that nothing in it has waited for when the role that fills it leaves: fill n waits for
    the release of fill n - slots, the tail for those of `slots` fills more.  Each release is an arrival from the pair's
    first block, which may still be under way."""
    seen = {n - slots for n in range(fills + (slots if tail else 0)) if n >= slots}
    return set(range(fills)) - seen


def test_a_ring_without_a_tail_leaves_arrivals_under_way():
    for fills in range(0, 30):
        for slots in (2, 3, 4, 12):
            assert len(_arrivals_left(fills, slots, False)) == min(fills, slots)
            assert not _arrivals_left(fills, slots, True)


def test_no_block_leaves_before_the_last_arrivals_of_its_rings():
    """The roles that fill a ring wait as if to go round it once more: the stages' ring (s_empty) and the scales' (s_sffree)."""
    for ring, slots, place in (("s_empty", "p.stages", "s"), ("s_sffree", "p.chunks", "ch")):
        tail = rf"if \(ok && warp == \d && lane < {re.escape(slots)}\) (?:ok = )?bar_wait\(smem_u32\(&{ring}\[lane\]\), lane < {place} \? phase : phase \^ 1,"
        assert re.search(tail, SOURCE), ring


def test_whichever_role_gives_up_both_blocks_wait_for_what_is_under_way():
    """A wait that runs out is told to both blocks; behind the barrier that all roles of both have reached, before TMEM is
    freed and any of them leaves, copies and arrivals get time to land."""
    kernel = SOURCE[SOURCE.index("matmul_mxfp4_kernel(const __grid_constant__"):]
    end = kernel[kernel.rindex("cluster_sync();"):kernel.index("tcgen05.dealloc")]
    assert re.search(r"if \(\*abort\)\s*for \(const long long start = clock64\(\); clock64\(\) - start < kLandCycles;\)", end)
    assert not re.search(r"\breturn\b", kernel[kernel.index("Tiles tile;"):kernel.index("tcgen05.dealloc")].split("const auto chunk_at")[0])
    gives_up = re.search(r"void give_up\(.*?\n}", SOURCE, re.S).group()
    assert "*abort = 1;" in gives_up and "st.shared::cluster" in gives_up and "cluster_rank() ^ 1" in gives_up
    wait = re.search(r"bool bar_wait\(.*?\n}", SOURCE, re.S).group()
    assert "give_up(abort" in wait and "*abort = 1" not in wait
