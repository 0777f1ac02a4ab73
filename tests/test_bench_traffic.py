"""The benchmark's recorded HBM traffic belongs to the kernels' code (no GPU)."""

import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "fp8_tensor_scaled_amd",
                    "csrc")


def local_sources(name, seen):
    """name and every file of the folder that it includes, directly or not."""
    if name in seen or not os.path.exists(os.path.join(CSRC, name)):
        return seen
    seen.add(name)
    with open(os.path.join(CSRC, name), encoding="utf-8") as fh:
        for inc in re.findall(r'^#include "([^"]+)"', fh.read(), re.M):
            local_sources(inc, seen)
    return seen


def test_key_covers_the_device_code():
    device = set()
    for name in local_sources("gemm_tiled.hip", set()):
        with open(os.path.join(CSRC, name), encoding="utf-8") as fh:
            if re.search(r"__device__|__global__", fh.read()):
                device.add(name)
    assert device == set(bench.PMC_SOURCES)


def test_recorded_traffic_is_of_this_code():
    """After a change to that code take the counters again and record its key."""
    for kernel in bench.PMC_TRAFFIC:
        assert bench.pmc_traffic(kernel), kernel
