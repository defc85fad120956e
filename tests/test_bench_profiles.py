"""The recorded captures (profiles/) against the sources they were taken on: the
benchmark reports a recorded figure only while these match, so a stale record
shows up there as a missing one."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench():
    sys.path.insert(0, ROOT)
    import bench
    return bench


def _records(name):
    with open(os.path.join(ROOT, "profiles", name)) as f:
        return [line.split() for line in f if line.strip() and not line.startswith("#")]


@pytest.mark.parametrize("name,source", [("single_launch.txt", 2), ("traffic.txt", 4)])
def test_recorded_captures_are_of_the_present_sources(name, source):
    bench = _bench()
    stale = [r[0] for r in _records(name) if bench.source_digest(os.path.join(ROOT, r[source])) != r[source + 1]]
    assert not stale, "captured on other sources: %s" % ", ".join(stale)


def test_every_recorded_single_launch_is_reported():
    bench = _bench()
    for r in _records("single_launch.txt"):
        assert bench.profiled_single_us(r[0]) == float(r[1])


def test_a_kernels_header_counts_as_its_source(tmp_path):
    # sources joined by "+", each from the first one's root: a change in any of them changes the digest
    bench = _bench()
    (tmp_path / "csrc").mkdir()
    for f in ("csrc/a.cu", "csrc/a.cuh"):
        (tmp_path / f).write_text(f)
    alone, both = str(tmp_path / "csrc/a.cu"), "%s+%s" % (tmp_path / "csrc/a.cu", tmp_path / "csrc/a.cuh")
    before = bench.source_digest(alone), bench.source_digest(both)
    assert before[0] != before[1]
    (tmp_path / "csrc/a.cuh").write_text("changed")
    assert bench.source_digest(alone) == before[0] and bench.source_digest(both) != before[1]


def test_the_groupnorms_records_cover_their_header():
    for name, source in (("single_launch.txt", 2), ("traffic.txt", 4)):
        for r in _records(name):
            if r[0].startswith("gn_"):
                assert "tb_groupnorm.cuh" in r[source], r[0]
