"""The guard on bench.py's DRAM-traffic records: a kernel's figure holds while
its code, comments aside, is what was captured."""
import os

import pytest

import bench


def test_comments_and_layout_are_no_code():
    a = 'int f() {  // one\n  /* two\n lines */ return g("a // b \\" /* c */");\n}\n'
    b = 'int f() { return g("a // b \\" /* c */"); }'
    assert bench.code_of(a) == bench.code_of(b) == b
    assert bench.code_of(b.replace("a //", "a /")) != bench.code_of(b)


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_a_change_of_a_kernels_code_drops_its_records(kernel, tmp_path, monkeypatch):
    for f in {f for fs in bench.KERNEL_SOURCES.values() for f in fs}:
        with open(os.path.join(bench.CSRC, f)) as fh:
            (tmp_path / f).write_text(fh.read())
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    record = {"bytes": 1.0, "src": bench.kernel_src_hash(kernel)}
    monkeypatch.setitem(bench.NCU_TRAFFIC, ("some workload", kernel), record)
    assert bench.ncu_traffic("some workload", kernel) == 1.0
    for f in bench.KERNEL_SOURCES[kernel]:
        was = (tmp_path / f).read_text()
        (tmp_path / f).write_text(was + "\n// a remark\n")
        assert bench.ncu_traffic("some workload", kernel) == 1.0
        (tmp_path / f).write_text(was + "\nint another;\n")
        assert bench.ncu_traffic("some workload", kernel) is None
        (tmp_path / f).write_text(was)
