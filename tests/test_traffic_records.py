"""The benchmark's records of measured DRAM traffic hold for the code that they were taken on (CPU)."""
import json
import os

import pytest

import bench

WORKLOADS = [w for w in bench.WORKLOADS.values() if w.traffic_file]


def _hash(tmp_path, monkeypatch, text):
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "a.cu").write_text(text)
    return bench.src_hash(["a.cu"])


def test_comments_and_spacing_do_not_count(tmp_path, monkeypatch):
    code = "int f(int a) {\n  return a + 1;\n}\n"
    want = _hash(tmp_path, monkeypatch, code)
    for same in ("// what f does\n" + code, code.replace("a + 1;", "a + 1;  // one more"), code.replace("\n", "\n\n"),
                 "/* two\n lines */" + code):
        assert _hash(tmp_path, monkeypatch, same) == want
    for other in (code.replace("1", "2"), code.replace("a + 1", "a - 1"), code + "int g;\n"):
        assert _hash(tmp_path, monkeypatch, other) != want


@pytest.mark.parametrize("wl", WORKLOADS, ids=lambda w: w.name)
def test_the_launch_code_counts(wl):
    names = [os.path.basename(s) for s in wl.sources]
    assert {"bl_common.cuh", "bl_host.cuh", "bl_api.cu"} <= set(names) and len(names) > 3
    assert all(os.path.exists(os.path.join(bench.ROOT, s)) for s in wl.sources)


@pytest.mark.parametrize("wl", WORKLOADS, ids=lambda w: w.name)
def test_a_record_of_other_code_is_left_out(wl, tmp_path, monkeypatch):
    with open(os.path.join(bench.ROOT, "profiles", wl.traffic_file)) as f:
        record = json.load(f)
    assert record.get("dram_bytes_per_launch", record.get("dram_bytes_per_step")) > 0
    monkeypatch.setattr(bench, "src_hash", lambda sources: "of other code")
    assert wl().traffic() is None
    monkeypatch.setattr(bench, "src_hash", lambda sources: record["src_hash"])
    assert wl().traffic() > 0
