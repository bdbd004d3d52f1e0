"""CPU check of the LDS layouts of the matrix-core kernel's gated form, with
the kernel's own index functions compiled for the host."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_glu_layouts(tmp_path):
    hipcc = "/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else shutil.which("hipcc")
    if hipcc is None:
        pytest.skip("hipcc not available")
    exe = tmp_path / "glu_layout_check"
    subprocess.check_call([hipcc, "-O1", "-std=c++17", os.path.join(HERE, "glu_layout_check.hip"),
                           "-o", str(exe)], stderr=subprocess.DEVNULL)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    print(res.stdout)
    assert res.returncode == 0, res.stdout
