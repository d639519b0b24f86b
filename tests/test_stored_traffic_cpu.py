"""The committed DRAM figure of a decode-attention call belongs to the committed kernel sources, so
that the bench can report it."""

import json
import os

import bench


def test_the_stored_figure_is_for_these_sources():
    with open(os.path.join(bench.ROOT, "profiles", "attn_traffic.json")) as f:
        t = json.load(f)
    assert t["kernel_rev"] == bench.kernel_revision()
    assert t["dram_bytes_per_launch"] == sum(t["parts"].values())
    assert bench.stored_traffic(t["workload"]) == t["dram_bytes_per_launch"]
