"""The kernel that fp4_gemm_grouped takes, from its host code against stub
launchers (tests/helpers/abi_grouped_rule_main.cpp); no GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def test_which_kernel_a_grouped_product_takes(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("g++ or the HIP headers not available")
    exe = str(tmp_path / "rule")
    csrc = os.path.join(ROOT, "fp4_precision_gemms_amd", "csrc")
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                            "-I", os.path.join(ROOT, "include"), "-I", csrc,
                            os.path.join(ROOT, "tests", "helpers", "abi_grouped_rule_main.cpp"),
                            os.path.join(csrc, "fp4_abi_ops.cpp"), "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout
