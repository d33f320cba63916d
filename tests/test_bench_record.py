"""The hash that dates the recorded DRAM traffic covers the recorded kernels and what they include."""
import os
import shutil

import bench

CSRC = os.path.join("kimi_delta_attention_03_gb300", "csrc")


def _copy(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path / CSRC


def test_other_headers_do_not_date_the_record(tmp_path, monkeypatch):
    here = bench.kernel_source_hash()
    csrc = _copy(tmp_path, monkeypatch)
    assert bench.kernel_source_hash() == here
    (csrc / "kda_unrelated.cuh").write_text("// nothing includes this\n")
    assert bench.kernel_source_hash() == here


def test_included_headers_do(tmp_path, monkeypatch):
    here = bench.kernel_source_hash()
    csrc = _copy(tmp_path, monkeypatch)
    for name in ("kda_sm100.cuh", "kda_common.cuh", "kda_prologue.cuh", "kda_decode.cu"):
        old = (csrc / name).read_text()
        (csrc / name).write_text(old + "\n")
        assert bench.kernel_source_hash() != here, name
        (csrc / name).write_text(old)
