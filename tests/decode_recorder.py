"""The decode step's checks and planning with recorded launches (``tests/c/decode_recorder.cpp``):
an accepted call returns 0 and touches no device, whatever its addresses."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session")
def recorder(tmp_path_factory):
    from deterministic_fixed_order_amd import _build
    from deterministic_fixed_order_amd import decode as d
    out = str(tmp_path_factory.mktemp("recorder") / "librecorder.so")
    subprocess.run([_build.hipcc()] + _build.common_flags() + ["-I", _build.CSRC, "-shared",
                   os.path.join(_build.CSRC, "decode.cpp"), os.path.join(_build.CSRC, "plan.cpp"),
                   os.path.join(ROOT, "tests", "c", "decode_recorder.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    d.bind(lib)
    return lib
