"""The sources that a recorded capture of a kernel's DRAM traffic is valid for."""

import json
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "long_context_decode_c4a_b200", "csrc")


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_every_included_header_counts(kernel):
    seen, todo = set(), [bench.KERNEL_SOURCES[kernel][0]]
    while todo:
        f = todo.pop()
        if f not in seen and os.path.exists(os.path.join(CSRC, f)):   # (the public header has no code)
            seen.add(f)
            with open(os.path.join(CSRC, f), encoding="utf-8") as fh:
                todo += re.findall(r'#include "([^"]+)"', fh.read())
    assert seen == set(bench.KERNEL_SOURCES[kernel])


def test_a_record_holds_only_for_its_sources(monkeypatch):
    with open(os.path.join(bench.ROOT, "profiles", "dram_traffic.json")) as f:
        records = json.load(f)
    for key, r in records.items():
        kernel, workload = key.split("@")
        files = bench.KERNEL_SOURCES[kernel]
        monkeypatch.setattr(bench, "kernel_hash", lambda fs: r["source_hash"])
        assert bench.traffic_for(kernel, workload, files) == r["bytes_per_launch"]
        monkeypatch.setattr(bench, "kernel_hash", lambda fs: "another")
        assert bench.traffic_for(kernel, workload, files) is None
