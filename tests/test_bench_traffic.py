"""The benchmark's DRAM-traffic records belong to the sources of the kernels they were captured on: those and the
headers they include, not the files of other operators."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join("rwkv_wkv_recurrence_b200", "csrc")


@pytest.fixture
def csrc(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path / CSRC


def _hashes():
    return {k: bench._kernel_source_hash(k) for k in bench._TRAFFIC_SOURCES}


def test_other_operators_do_not_touch_the_records(csrc):
    before = _hashes()
    (csrc / "another.cuh").write_text("// a header of another operator\n")
    (csrc / "another.cu").write_text('#include "another.cuh"\n')
    for name in ("api_mixer.cu", "conv.cu", "mixer.h", "mixer_common.cuh", "norm.cu", "scan_bwd.cu", "scan_common.cuh",
                 "scan_fwd.cu", "scan_plan.h", "scan_step.cu"):
        with open(csrc / name, "a") as f:
            f.write("// changed\n")
    assert _hashes() == before


def test_the_kernels_own_sources_do(csrc):
    before = _hashes()
    with open(csrc / "wkv5_step.cu", "a") as f:
        f.write("// changed\n")
    assert {k for k, v in _hashes().items() if v != before[k]} == {"wkv5_step_kernel", "wkv5_step_kernel/finch"}
    for name in ("launch.h", "wkv_common.cuh"):
        now = _hashes()
        with open(csrc / name, "a") as f:
            f.write("// changed\n")
        assert all(v != now[k] for k, v in _hashes().items()), name
