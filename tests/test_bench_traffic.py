"""The bench line's measured DRAM traffic belongs to the code in this tree."""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.TRAFFIC))
def test_captures_are_of_the_code_as_it_is(kernel):
    t = bench.TRAFFIC[kernel]
    assert t["sha256"] == bench.sources_sha256(t["sources"])
    for key, entry in t["bytes_per_launch"].items():
        assert bench.traffic_of(kernel, key) == (entry["bytes"], entry["how"])


def test_only_code_counts(tmp_path):
    a, b, c = (str(tmp_path / n) for n in "abc")
    open(a, "w").write("int f() { return 1; }  // one\n")
    open(b, "w").write("/* f,\n   f */ int f()\n{ return  1; }")
    open(c, "w").write("int f() { return 2; }  // one\n")
    hashes = [bench.sources_sha256([p]) for p in (a, b, c)]
    assert hashes[0] == hashes[1] != hashes[2]
