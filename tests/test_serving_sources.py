"""What the serving kernels' sources have to keep to and no run shows: no GPU needed."""
import os
import re

from block_sparse_long_tcgen05_b200 import build as msa_build

CSRC = os.path.join(msa_build.HERE, "csrc")


def test_results_of_a_kernel_before_are_not_read_as_read_only():
    """A decode's kernels start while the one before them still runs, so what one of them writes (ids, block
    maxima, parts, arrivals) is not read-only for the lifetime of the next: __ldg's path is not defined for it."""
    found = 0
    for name in ("paged.cuh", "paged_small.cuh", "prefix_scan.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for read in re.findall(r"__ldg\(([^;]*);", text):
            found += 1
            assert not re.search(r"block_ids|maxima|parts|arrived", read), f"{name}: __ldg({read}"
    assert found > 0
