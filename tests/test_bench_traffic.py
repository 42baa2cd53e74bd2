"""bench.py takes a recorded DRAM traffic only while the kernel's source and the headers it includes are
those of the capture (CPU only)."""

import json
import os
import shutil

import pytest

import bench

CSRC = os.path.join("int4_blockwise_quantised_b200", "csrc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    source = os.path.join(CSRC, "attn_prefill.cu")
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(
        {"attn_prefill": {"dram_bytes_per_launch": 123, "source": source, "source_sha": bench.source_sha(source)}}))
    return tmp_path / CSRC


def test_traffic_of_unchanged_sources(tree):
    assert bench.traffic_for("attn_prefill") == 123
    (tree / "vv_internal.h").write_text("// host side\n")
    (tree / "logits.cu").write_text("// another kernel\n")
    assert bench.traffic_for("attn_prefill") == 123


@pytest.mark.parametrize("name", ["attn_prefill.cu", "attn_prefill.h", "attn_tc.cuh", "vv_device.cuh"])
def test_traffic_is_dropped_when_a_source_changes(tree, name):
    with open(tree / name, "a") as f:
        f.write("// changed\n")
    assert bench.traffic_for("attn_prefill") is None


def test_committed_captures_name_commands_and_existing_sources():
    for d in json.load(open(os.path.join(bench.ROOT, "profiles", "traffic.json"))).values():
        assert os.path.exists(os.path.join(bench.ROOT, d["source"])) and d["dram_bytes_per_launch"] > 0
        assert d["command"].startswith("ncu ") and "<" not in d["command"]
