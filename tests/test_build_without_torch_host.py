"""The library builds and loads where torch is not installed (CPU only): torch is
for device memory and streams in Python, and for the C++ side of decode.py's calls,
which is left out there; a C caller needs neither."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_binding_is_left_out_without_torch(detfold_lib, tmp_path):
    out = str(tmp_path / "_bind.so")
    text = """
import sys
sys.modules["torch"] = None  # as if it were not installed
from deterministic_fixed_order_amd import _build
import deterministic_fixed_order_amd as detfold
detfold.load()
assert _build.build_binding(sys.argv[1]) is None
print("left out")
"""
    res = subprocess.run([sys.executable, "-c", text, out], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0, res.stderr[-3000:]
    assert res.stdout.strip().endswith("left out") and "torch" in res.stdout
    assert not os.path.exists(out)
