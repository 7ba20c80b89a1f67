"""The bench line's DRAM traffic belongs to the Newton-Schulz sources that it was measured on."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "muon_adamw_hybrid_grad_gb300", "csrc")


def included(name, seen):
    """The file and what it includes of its own folder."""
    path = os.path.join(CSRC, name)
    if name in seen or not os.path.exists(path):
        return seen
    seen.add(name)
    with open(path) as fh:
        for other in re.findall(r'^#include "([^"]+)"', fh.read(), re.M):
            included(other, seen)
    return seen


def test_traffic_is_tied_to_every_source_of_its_kernel():
    assert set(bench.NS_SOURCES) == included("ns_tc.cu", set())


def test_traffic_is_null_once_a_source_changes(monkeypatch):
    monkeypatch.setitem(bench.NS_TRAFFIC, "sources_sha256", "0" * 64)
    assert bench.ns_traffic_per_launch("full_vla") is None
