"""What importing the package brings in."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_loads_neither_torch_nor_the_library():
    """The build and the report tools import the package without tensors: torch
    (seconds on a cold start, and not needed to build) comes with the first
    call that takes one, the library with the first call."""
    code = ("import sys, roofline_sgemm_f32_amd as rs; from roofline_sgemm_f32_amd import binding; "
            "assert 'torch' not in sys.modules, 'torch'; assert binding._lib is None, 'library'; "
            "assert rs.ACTIVATIONS['silu'] == 0")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
