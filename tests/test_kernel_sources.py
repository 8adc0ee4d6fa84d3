"""The sums that profiles carry cover every source of their kernels."""

import glob
import os

import bench


def test_sums_cover_the_block():
    csrc = os.path.join(bench.ROOT, "token_routing_amd", "csrc")
    own = {os.path.basename(f) for p in ("block_*", "pack*") for f in glob.glob(os.path.join(csrc, p))}
    assert own and own <= set(bench.KERNEL_SOURCES["block"])
    assert bench.kernel_source_sha("block") != bench.kernel_source_sha("fwd")


def test_labels():
    assert bench.kernel_source_sha("dX") == bench.kernel_source_sha("groups")
    assert bench.kernel_source_sha("combine") == bench.kernel_source_sha("combine_bwd")
    assert len({bench.kernel_source_sha(x) for x in (None, "fwd", "combine", "route", "block")}) == 5
