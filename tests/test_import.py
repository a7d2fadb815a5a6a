"""CPU-only: the C bindings need no torch; the operators that do are found on first use."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "dense_fp32_matrix_08_gb300"


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_bindings_work_without_torch():
    r = run(f"""
import sys
sys.modules["torch"] = None  # any import of it fails
import {PACKAGE} as sg
from {PACKAGE} import *
assert sgemm_f32_version() == sg.sgemm_f32_version()
assert sg.sgemm_f32(-1, 4, 4, 1.0, None, 4, None, 4, 0.0, None, 4, 0) == -1
assert sg.lib.f8_gemm_with(None) == -1 and sg.lib.ns_orthogonalize_workspace_size(-1, 1, 1, None) == -1
assert sg.F8_EXPORTED and NS_EXPORTED
try:
    sg.f8_quantize
except ImportError:
    pass
else:
    raise AssertionError("f8_quantize without torch")
""")
    assert r.returncode == 0, r.stderr


def test_operators_are_found():
    r = run(f"""
import sys
import {PACKAGE} as sg
assert "torch" not in sys.modules
names = {{"f8_quantize", "f8_quantize_pair", "f8_matmul", "f8_gemm_status", "orthogonalize",
         "ns_orthogonalize_workspace_size", "ns_orthogonalize_status"}}
assert names <= set(dir(sg)) and names <= set(sg.__all__)
from {PACKAGE} import orthogonalize
from {PACKAGE} import *
assert all(callable(getattr(sg, n)) for n in names)
assert f8_matmul is sg.f8.f8_matmul and orthogonalize is sg.newton_schulz.orthogonalize
assert not hasattr(sg, "f9_matmul")
""")
    assert r.returncode == 0, r.stderr
