"""Checks on the gfx950 assembly of the decode-step operators (CPU only): no packed
float32 arithmetic, no writes through the scalar data cache, subnormals kept, the
products on the matrix units, the cache's bytes in wide loads, and nothing of a
main loop in scratch memory."""
import glob
import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_isa import SCALAR_WRITE, _kernels

PACKED = re.compile(r"^\s*(v_pk_fma_f32|v_pk_add_f32|v_pk_mul_f32)\b", re.M)


@pytest.fixture(scope="module")
def isa(tmp_path_factory):
    from deterministic_fixed_order_amd import _build

    root = str(tmp_path_factory.mktemp("isa"))

    def one(src):
        out = os.path.join(root, os.path.basename(src).replace(".", "_"))
        _build.save_temps(out, src)
        files = glob.glob(os.path.join(out, "*gfx950*.s"))
        assert files, "no gfx950 assembly produced"
        return os.path.basename(src), "\n".join(open(f).read() for f in files)
    with ThreadPoolExecutor(max_workers=5) as pool:
        return dict(pool.map(one, _build.DECODE_KERNELS))


def test_no_packed_float32_and_no_scalar_writes(isa):
    for name, text in isa.items():
        assert not PACKED.findall(text), name
        assert not SCALAR_WRITE.findall(text), name


def test_f32_denormals_kept(isa):
    for name, text in isa.items():
        modes = re.findall(r"\.amdhsa_float_denorm_mode_32\s+(\d+)", text)
        assert modes and set(modes) == {"3"}, name


def test_products_are_on_the_matrix_units(isa):
    for name, ops in (("attend_bf16.hip", {"v_mfma_f32_16x16x32_bf16", "v_mfma_f32_16x16x4_f32"}),
                      ("attend_f16.hip", {"v_mfma_f32_16x16x32_f16", "v_mfma_f32_16x16x4_f32", "v_mfma_f32_16x16x32_bf16"}),
                      ("attend_f32.hip", {"v_mfma_f32_16x16x4_f32", "v_mfma_f32_16x16x32_bf16"})):
        assert set(re.findall(r"v_mfma_\w+", isa[name])) == ops, name


def test_scratch(isa):
    """Heads of at most 128 hold everything in registers; above, a few words."""
    for name, text in isa.items():
        for kernel, block in _kernels(text):
            private = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1))
            assert private <= (16 if "Li256E" in kernel else 0), "%s: %d bytes" % (kernel, private)
