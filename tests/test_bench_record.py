"""The bench's DRAM figure of the attention kernel stands only while the kernel's sources
are those of its committed capture: a change to them needs a capture of its own."""
import dataclasses

import bench
from clustered_sparse_attention_b200 import synth


def test_attention_traffic_is_of_the_current_sources():
    w = synth.WORKLOADS["wan720p"]
    traffic = bench.attend_traffic(w)
    assert traffic is not None, "the attention kernel's sources changed since its capture"
    assert traffic == 5 * bench.attend_traffic(dataclasses.replace(w, H=w.H // 5))
