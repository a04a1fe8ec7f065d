"""The index arithmetic of rows grouped by expert (csrc/grouped.hpp) compiled for
the host (tests/helpers/grouped_index_main.cpp): the expert of every unit, and no
place outside the tensors, whatever the offsets."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_offsets_of_any_kind_stay_inside_the_tensors(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    # a header of that name that declares nothing: the intrinsics are the test's
    os.makedirs(tmp_path / "hip")
    (tmp_path / "hip" / "hip_runtime.h").write_text("")
    exe = str(tmp_path / "index")
    build = subprocess.run(["g++", "-std=c++17", "-O2", "-I", str(tmp_path), "-I",
                            os.path.join(ROOT, "fp4_precision_gemms_amd", "csrc"),
                            os.path.join(ROOT, "tests", "helpers", "grouped_index_main.cpp"), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout
