"""The counter records of the bench name the sources that they were taken on."""
import json
import os
import shutil

import pytest

import bench


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the kernel sources and the records; bench looks there."""
    for part in (("lossless_kv_cache_scalar_amd", "csrc"), ("profiles",)):
        shutil.copytree(os.path.join(bench.ROOT, *part), tmp_path.joinpath(*part))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path


def records(tree):
    return sorted(p for p in os.listdir(tree / "profiles") if p.startswith("traffic_"))


def test_records_are_current(tree):
    assert records(tree)
    for name in records(tree):
        rec = json.loads((tree / "profiles" / name).read_text())
        assert bench.counter_record(rec["kernel"], rec["workload"]) == rec, name


@pytest.mark.parametrize("source", ["skv_api.hip", "skv_decode.hip", "skv_encode.hip", "skv_internal.hpp", "skv_model.hip"])
def test_a_change_to_the_coder_sets_its_records_aside(tree, source):
    """Its kernels, and the file that sets their grids and the layout of their workspace."""
    path = tree / "lossless_kv_cache_scalar_amd" / "csrc" / source
    path.write_text(path.read_text() + "\n// changed\n")
    for name in records(tree):
        rec = json.loads((tree / "profiles" / name).read_text())
        assert bench.counter_record(rec["kernel"], rec["workload"]) is None, name


@pytest.mark.parametrize("source", ["skv_pages.hip", "skv_pages.hpp", "skv_attend.hip", "skv_status.hip"])
def test_other_calls_leave_them_current(tree, source):
    before = bench.csrc_hash()
    path = tree / "lossless_kv_cache_scalar_amd" / "csrc" / source
    path.write_text(path.read_text() + "\n// changed\n")
    assert bench.csrc_hash() == before
