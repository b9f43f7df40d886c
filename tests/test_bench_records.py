"""bench.py reports a recorded DRAM figure only while the code that it was taken on is unchanged: every source that a
kernel is made of has to be in the record's list."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "combine_router_top_gb300", "csrc")


def included(name, seen):
    seen.add(name)
    with open(os.path.join(CSRC, name)) as fh:
        for inc in re.findall(r'^\s*#include "([^"]+)"', fh.read(), re.M):
            if inc not in seen and os.path.exists(os.path.join(CSRC, inc)):
                included(inc, seen)
    return seen


def test_the_records_hash_covers_every_source_of_the_kernel():
    for kernel, files in bench.TRAFFIC_SOURCES.items():
        assert included(files[0], set()) == set(files), kernel
