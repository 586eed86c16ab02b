"""What the BF16 product's source must say where a run cannot show it (barriers that a pair of blocks shares), and the
polynomial in its normal distribution function against math.erfc."""

import math
import os
import re

import ctypes as C
import numpy as np
import pytest

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild

with open(os.path.join(cbuild.CSRC, "matmul_bf16.cu")) as f:
    SOURCE = f.read()
with open(os.path.join(cbuild.CSRC, "matmul_bf16.cuh")) as f:
    HEADER = f.read()


def _asm(op):
    return re.findall(r'"[^"]*?(mbarrier\.' + op + r'[^ "]*) ', SOURCE)


def test_arrivals_and_waits_across_blocks_have_cluster_scope():
    remote = [i for i in _asm("arrive") if ".shared::cluster" in i]
    assert remote and all(re.search(r"\.(relaxed|release)\.cluster\.shared::cluster", i) for i in remote), remote
    waits = _asm("try_wait") + _asm("test_wait")
    assert len(waits) >= 2 and all(re.search(r"\.(relaxed|acquire)\.cluster\.", i) for i in waits), waits


def test_relaxed_operations_stand_with_their_fences():
    body = re.search(r"void bar_arrive_smem\(.*?\n}", SOURCE, re.S).group()
    assert body.index("fence.release.sync_restrict::shared::cta.cluster") < body.index("mbarrier.arrive.relaxed.cluster")
    wait = re.search(r"bool bar_wait\(.*?\n}", SOURCE, re.S).group()
    assert wait.index("fence_acquire_smem();") < wait.index("return true;") and wait.count("return true;") == 1
    assert re.search(r"= bar_test\([^;]*;\s*fence_acquire_smem\(\);", SOURCE)
    # zeroed rows: written, fenced for the tensor core's proxy, then announced to the first block
    assert re.search(r"make_uint4\(0, 0, 0, 0\);\s*fence_proxy_async\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) bar_arrive_smem\(in_block", SOURCE)


def test_no_block_leaves_before_what_is_under_way_has_landed():
    assert re.search(r"if \(ok && warp == 0 && lane < p\.stages\) bar_wait\(smem_u32\(&s_empty\[lane\]\), lane < s \? phase : phase \^ 1,", SOURCE)
    kernel = SOURCE[SOURCE.index("matmul_bf16_kernel(const __grid_constant__"):]
    end = kernel[kernel.rindex("cluster_sync();"):kernel.index("tcgen05.dealloc")]
    assert re.search(r"if \(\*abort\)\s*for \(const long long start = clock64\(\); clock64\(\) - start < kLandCycles;\)", end)
    assert not re.search(r"\breturn\b", kernel[kernel.index("Tiles<MODE> tile;"):kernel.index("tcgen05.dealloc")])
    gives_up = re.search(r"void give_up\(.*?\n}", SOURCE, re.S).group()
    assert "*abort = 1;" in gives_up and "st.shared::cluster" in gives_up and "cluster_rank() ^ 1" in gives_up


def test_no_load_is_multicast():
    assert not [i for i in re.findall(r'"(cp\.async\.bulk[^ "]*)', SOURCE) if "multicast" in i]


def test_normal_distribution_polynomial():
    """binary32 as the kernel computes it, but for the approximate reciprocal and exponential (two steps each)."""
    body = re.search(r"float normal_cdf\(float z.*?\n}", HEADER, re.S).group()
    coef = [float(v) for v in re.findall(r"(?:p = |t, )(-?[0-9.]+)f", body)]
    c = float(re.search(r"fmaf\(([0-9.]+)f, fabsf", body).group(1))
    assert len(coef) == 7
    z = np.concatenate([np.linspace(-6, 6, 24001), np.linspace(-37, 37, 2001)]).astype(np.float32)
    t = np.float32(1) / (np.float32(1) + np.float32(c) * np.abs(z))
    with np.errstate(under="ignore"):
        bell = np.exp2(np.float32(-0.72134752) * z * z).astype(np.float32)
        p = np.full_like(z, np.float32(coef[0]))
        for v in coef[1:]:
            p = p * t + np.float32(v)
        half = p * t * bell
    got = np.where(z > 0, 1 - half, half).astype(np.float64)
    ref = np.array([0.5 * math.erfc(-float(v) / math.sqrt(2)) for v in z])
    near = np.abs(z) <= 6
    assert (np.abs(got - ref)[near] <= 4e-6 * ref[near]).all()      # the exponent's rounding: 18 * 1.44 * 2^-24 * ln 2 and the fit's 6.4e-7
    assert (np.abs(got - ref) <= 5e-7).all()


@pytest.mark.parametrize("bad,code", [
    (dict(what=3), cgl.EINVAL), (dict(what=-1), cgl.EINVAL), (dict(f=12), cgl.EINVAL), (dict(k=4), cgl.EINVAL), (dict(rows=0), cgl.EINVAL),
    (dict(rows=2 ** 21), cgl.EINVAL), (dict(wait=-1), cgl.EINVAL), (dict(x=None), cgl.EINVAL), (dict(st=None), cgl.EINVAL), (dict(x=0x10008), cgl.EALIGN),
    (dict(out=0x10008), cgl.EALIGN)])
def test_selftest_refusals(bad, code):
    P = 0x10000
    a = dict(dict(what=0, x=P, rows=8, y=P, f=64, k=64, out=P, wait=0, st=P), **bad)
    fn = cgl.lib().cgl_selftest_matmul_bf16_timeout
    p, i, q = C.c_void_p, C.c_int, C.c_int64
    fn.argtypes, fn.restype = [i, p, q, p, i, i, p, q, p, p], C.c_int
    assert fn(a["what"], a["x"], a["rows"], a["y"], a["f"], a["k"], a["out"], a["wait"], a["st"], None) == code
