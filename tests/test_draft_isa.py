"""Checks on the gfx950 assembly of the drafted step's operators (CPU only): no packed
float32 arithmetic, no writes through the scalar data cache, subnormals kept, the
products on the matrix units, and nothing of a hot loop in scratch memory."""
import glob
import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_decode_isa import PACKED
from test_isa import SCALAR_WRITE, _kernels


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
        return dict(pool.map(one, _build.DRAFT_KERNELS))


def test_no_packed_float32_and_no_scalar_writes(isa):
    for name, text in isa.items():
        assert not PACKED.findall(text), name
        assert not SCALAR_WRITE.findall(text), name


def test_f32_denormals_kept(isa):
    for name, text in isa.items():
        modes = re.findall(r"\.amdhsa_float_denorm_mode_32\s+(\d+)", text)
        assert modes and set(modes) == {"3"}, name


def test_products_are_on_the_matrix_units(isa):
    for name, ops in (("tree_bf16.hip", {"v_mfma_f32_16x16x32_bf16", "v_mfma_f32_16x16x4_f32"}),
                      ("tree_f16.hip", {"v_mfma_f32_16x16x32_f16", "v_mfma_f32_16x16x4_f32", "v_mfma_f32_16x16x32_bf16"}),
                      ("tree_f32.hip", {"v_mfma_f32_16x16x4_f32", "v_mfma_f32_16x16x32_bf16"})):
        assert set(re.findall(r"v_mfma_\w+", isa[name])) == ops, name


def test_scratch(isa):
    """Heads of at most 128 hold everything in registers, but for a few words of float16 to float32 in small pages;
    above, some more."""
    for name, text in isa.items():
        for kernel, block in _kernels(text):
            private = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1))
            most = 128 if "Li256E" in kernel else 32 if "IDF16_Li1ELi2ELi128ELb0E" in kernel else 0
            assert private <= most, "%s: %d bytes" % (kernel, private)
