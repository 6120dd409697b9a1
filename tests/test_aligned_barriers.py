"""Warp-aligned cluster barriers stand behind a warp barrier (read from the sources; no GPU needed).

barrier.cluster.*.aligned is defined only where all lanes of a warp execute it together.  A kernel whose lanes took
different branches before it may hang or leave its cluster early, so nothing here runs one: the sources are read.
"""
from __future__ import annotations

import os
import re

from rmsnorm_qknorm_b200 import build as qbuild


def sources():
    for name in sorted(os.listdir(qbuild.CSRC)):
        with open(os.path.join(qbuild.CSRC, name)) as f:
            yield name, re.sub(r"//[^\n]*", "", f.read())


def test_every_cluster_barrier_follows_a_warp_barrier():
    seen = 0
    for name, text in sources():
        for m in re.finditer(r'asm volatile\("barrier\.cluster\.\w+', text):
            assert text[:m.start()].rstrip().endswith("__syncwarp();"), f"{name}: {text[m.start(): m.start() + 60]}"
            seen += 1
        body = re.sub(r'asm volatile\("barrier\.cluster[^;]*;[^;]*;[^;]*;', "", text)
        assert "barrier.cluster" not in body, name
    assert seen == 1


def test_lanes_meet_before_the_barriers_behind_finish():
    # rows::finish returns per lane for features behind the last; what follows a call up to the next barrier
    text = dict(sources())["linear_rows.cuh"]
    tail = text[text.rindex("finish<"):]
    assert re.match(r"finish<[^;]*;\s*__syncwarp\(\);", tail)
