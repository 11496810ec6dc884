"""The recorded DRAM traffic of the bench line: which changes of the sources drop it (no GPU needed)."""
import json
import os
import shutil

import pytest

import bench

CSRC = os.path.join("mamba_selective_state_causal_b200", "csrc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources with a record of 42 bytes per token for each recorded kernel, taken from them."""
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        d = json.load(f)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    for r in d.values():
        r.update(dram_bytes_per_token=42.0, code_sha256_16=bench.code_digest(str(tmp_path / r["source"])))
    os.makedirs(tmp_path / "profiles")
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(d))
    return tmp_path / CSRC


def _edit(path, old, new):
    text = path.read_text()
    assert old in text
    path.write_text(text.replace(old, new, 1))


KERNELS = ("chunk_output_tc", "bwd_chunk_grad_tc")


def test_recorded_for_both_kernels(tree):
    assert [bench.recorded_traffic(k) for k in KERNELS] == [42.0, 42.0]
    assert bench.recorded_traffic("no_such_kernel") is None


def test_comments_and_spaces_keep_it(tree):
    for f in ("scan_tc.cu", "scan_bwd.cu", "scan_tc_util.cuh", "tc_ptx.cuh"):
        _edit(tree / f, "\n", "   // of no consequence\n\n/* nor\n this */\n")
    assert [bench.recorded_traffic(k) for k in KERNELS] == [42.0, 42.0]


@pytest.mark.parametrize("f,lost", [
    ("scan_tc.cu", ("chunk_output_tc",)), ("scan_bwd.cu", ("bwd_chunk_grad_tc",)), ("scan_tc_util.cuh", ("chunk_output_tc",)),
    ("tc_ptx.cuh", KERNELS), ("ssd_common.cuh", KERNELS), ("decode.cu", ()),
])
def test_a_change_of_the_code_drops_it(tree, f, lost):
    """Of the kernel's file or of a header that it includes, and of no other."""
    _edit(tree / f, "namespace ssd {", "namespace ssd {\nconstexpr int kOther = 1;")
    for k in KERNELS:
        assert bench.recorded_traffic(k) == (None if k in lost else 42.0), k
