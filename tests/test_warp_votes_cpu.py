"""Which lanes take part in a warp-wide operation is fixed by the code, never by which lanes happen to be active: two
reads of the active mask may differ, and lanes behind a branch need not have come together again."""

import glob
import os
import re

from combine_get_layout_02_b200 import build as cbuild


def test_no_kernel_asks_which_lanes_are_active():
    found = []
    for path in sorted(glob.glob(os.path.join(cbuild.CSRC, "*.cu*"))):
        with open(path) as f:
            for i, line in enumerate(f, 1):
                if re.search(r"__activemask|%lanemask|\bactivemask\.b32", line):
                    found.append(f"{os.path.basename(path)}:{i}: {line.strip()}")
    assert found == []
