"""The compiler's figures are found for the kernels that run by default, and for every tile of
the sweep."""
import json
import os

import pytest

import gemv_fp16_amd as gf
from gemv_fp16_amd import resources


def test_names_of_the_report(tmp_path):
    cfg = {"block_m": 64, "block_n": 64, "block_k": 64, "stages": 3, "threads": 256, "schedule": 0}
    name = resources.gemm_kernel_name(cfg).replace(">(gf::GemmArgs)", ", gf::GemmArgs>(gf::GemmArgs)")
    path = tmp_path / "report.json"
    path.write_text(json.dumps({"_Z1": {"name": name, "scratch_bytes": 4}, "_Z2": {"name": "void gf::other<1>(int)"}}))
    report = resources.load(str(path))
    assert resources.gemm(cfg, report=report) == {"name": name, "scratch_bytes": 4}
    assert "void gf::other<1>(int)" in report


def test_default_kernels_are_in_the_report():
    if not os.path.exists(resources.RESOURCES):
        pytest.skip("the library was built elsewhere")
    assert "not in the report" not in resources.defaults_table()
    known = [resources.gemm(c) for c, there in gf.gemm_configs() if there]
    assert known and all(known)
