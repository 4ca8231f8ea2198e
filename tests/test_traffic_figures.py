"""The committed DRAM traffic figures belong to the sources that are there."""
import json
import os

import pytest

import bench


def _kernels():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        return json.load(f)["kernels"]


@pytest.mark.parametrize("kernel", sorted(_kernels()))
def test_traffic_of_a_kernel_is_that_of_its_sources(kernel):
    # (a change to a kernel's sources voids its figure: take it again with the commands in the file)
    assert bench.ncu_traffic(kernel) == _kernels()[kernel]["dram_bytes_per_launch"]
