"""The sources that bench.py's stored counter results are tied to: all that a kernel's device code comes from, or an
edit would leave stale counters passing as current."""
import os
import re

import pytest

import bench

# declarations of the C ABI and of host functions: no device code
HOST_ONLY = {"gfg.h", "gfg_internal.h"}


def closure(path):
    """A source and the headers of its folder that it includes, by any number of steps."""
    seen, todo = set(), [path]
    while todo:
        p = todo.pop()
        if p in seen:
            continue
        seen.add(p)
        with open(p) as f:
            names = re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M)
        todo += [os.path.join(os.path.dirname(p), n) for n in names if n not in HOST_ONLY]
    return seen


@pytest.mark.parametrize("sources,roots", [(bench.KERNEL_SRC, ("gfg_gemm.hip", "gfg_gemm256.hip")), (bench.QUANT_SRC, ("gfg_quant.hip",))])
def test_hash_covers_every_included_header(sources, roots):
    want = set().union(*(closure(os.path.join(bench._CSRC, r)) for r in roots))
    assert want == set(sources)


def test_every_source_changes_the_hash(tmp_path):
    copies = []
    for p in bench.KERNEL_SRC:
        with open(p) as f:
            text = f.read()
        c = tmp_path / os.path.basename(p)
        c.write_text(text)
        copies.append(str(c))
    before = bench.kernel_source_hash(copies)
    for c in copies:
        with open(c) as f:
            text = f.read()
        with open(c, "w") as f:
            f.write(text + "\nint one_more;\n")
        assert bench.kernel_source_hash(copies) != before, c
        with open(c, "w") as f:
            f.write(text + "\n// a comment\n")
        assert bench.kernel_source_hash(copies) == before, c
        with open(c, "w") as f:
            f.write(text)


def test_stored_traffic_belongs_to_the_sources():
    """The GEMM workloads' stored counter results are reported: they were taken on these sources."""
    from fp8_block_scaled_amd import workloads as wl
    folder = os.path.join(bench.ROOT, "profiles")
    names = [n[len("traffic_"):-len(".json")] for n in os.listdir(folder)
             if n.startswith("traffic_") and not n.startswith("traffic_quant_")]
    assert bench.DEFAULT_WORKLOAD in names
    assert [n for n in names if bench.traffic_from_profile(wl.workload(n)) is None] == []
