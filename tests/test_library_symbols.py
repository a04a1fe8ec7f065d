"""The C names that libfp4.so exports: the ABI's, and no helper that another
library's function of the same name could take the place of."""
import os
import re
import shutil
import subprocess

import pytest

import fp4_precision_gemms_amd as F


def test_exported_c_names_are_the_abi():
    if not os.path.exists(F.LIB_PATH) or shutil.which("nm") is None:
        pytest.skip("libfp4.so not built or nm not available")
    out = subprocess.run(["nm", "-D", "--defined-only", F.LIB_PATH], capture_output=True, text=True, check=True).stdout
    names = {l.split()[2] for l in out.splitlines() if l.split()[1] == "T" and not l.split()[2].startswith("_")}
    header = os.path.join(os.path.dirname(os.path.dirname(F.LIB_PATH)), "include", "fp4.h")
    with open(header) as f:
        declared = set(re.findall(r"\b((?:nv)?fp4_\w+)\(", f.read()))
    assert names == names & declared, sorted(names - declared)
    assert "fp4_gemm_grouped" in names
