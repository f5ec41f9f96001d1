"""Build step for ``libdetfold.so`` (hipcc, gfx950 only).

Sources (``csrc/``): fold_kernels.hip (the fold's device code and launches),
plan.cpp (host-only planning and argument checks), detfold.cpp (call sequences
and the C ABI), internal.h (their shared declarations); of the decode-step
operators cache_kernels.hip and attend_kernels.hip (device code and launches),
attend_f32.hip, attend_f16.hip and attend_bf16.hip (the instances of
attend_kernel.h), decode.cpp (checks, planning and the C ABI), decode.h,
decode_check.h and decode_device.h; of the drafted step's tree_kernels.hip and
page_kernels.hip (device code and launches), tree_f32.hip, tree_f16.hip and
tree_bf16.hip (the instances of tree_kernel.h), draft.cpp (checks, planning and
the C ABI) and draft.h; and bind.cpp, the C++ side of both modules' calls, a library
of its own.
exports.map limits the exported symbols to the C ABI of include/detfold.h.

The .hip files are compiled in two passes, so that device-only flags reach
the device compiler only: the device pass writes the gfx950 code object
bundle, and the host pass embeds it (clang's ``-fcuda-include-gpubinary``,
the step the one-command HIP build performs internally).  Both passes of a
file share one compilation-unit id, so host and device agree on the names of
any ``__device__`` variable.  The .cpp files hold no device code.  The files
are compiled side by side.

Flags that fix the fold's bits:
  -ffp-contract=off                 no fused multiply-add anywhere
  -fno-fast-math                    no reassociation of the add chain
  -fno-gpu-flush-denormals-to-zero  binary32 subnormals kept (the gfx9 default,
                                    stated; device pass)
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                    no packed FP32 instructions; every add is a
                                    plain v_add_f32 (device pass)

``source_digest()`` is the sha256 of every input of the build (sources,
header, export map and the flags); ``build_library`` writes it beside the
library, and ``is_current()`` compares it, so that a library built from
other sources is rebuilt rather than run.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
KERNELS = os.path.join(CSRC, "fold_kernels.hip")
HOST_SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "detfold.cpp")]
SOURCES = [KERNELS] + HOST_SOURCES
INTERNAL_HEADER = os.path.join(CSRC, "internal.h")
DECODE_KERNELS = [os.path.join(CSRC, f) for f in ("cache_kernels.hip", "attend_kernels.hip", "attend_f32.hip",
                                                     "attend_f16.hip", "attend_bf16.hip")]
DRAFT_KERNELS = [os.path.join(CSRC, f) for f in ("tree_kernels.hip", "page_kernels.hip", "tree_f32.hip", "tree_f16.hip",
                                                     "tree_bf16.hip")]
DRAFT_SOURCES = DRAFT_KERNELS + [os.path.join(CSRC, f) for f in ("draft.cpp", "draft.h", "tree_kernel.h")]
DECODE_SOURCES = DECODE_KERNELS + [os.path.join(CSRC, f) for f in ("decode.cpp", "decode.h", "decode_check.h", "decode_device.h",
                                                                 "attend_kernel.h", "bind.cpp")]
BINDING = os.path.join(CSRC, "bind.cpp")
EXPORTS_MAP = os.path.join(CSRC, "exports.map")
HEADER = os.path.join(ROOT, "include", "detfold.h")
LIB = os.path.join(PKG, "libdetfold.so")
BINDING_LIB = os.path.join(PKG, "_bind.so")
DIGEST = LIB + ".sha256"
ARCH = "gfx950"


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def common_flags() -> list[str]:
    return [
        "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
        "-ffp-contract=off", "-fno-fast-math",
        "-Wall", "-Wextra", "-Wno-unused-parameter",
        "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    ]


def device_flags() -> list[str]:
    return ["-fno-gpu-flush-denormals-to-zero",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def link_flags() -> list[str]:
    return ["--offload-arch=" + ARCH, "-shared", "-fPIC", "-Wl,--version-script=" + EXPORTS_MAP]


def source_digest() -> str:
    h = hashlib.sha256()
    for path in SOURCES + DECODE_SOURCES + DRAFT_SOURCES + [INTERNAL_HEADER, EXPORTS_MAP, HEADER]:
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode() + b"\0" + f.read() + b"\0")
    h.update("\0".join(common_flags() + device_flags() + link_flags()).encode())
    return h.hexdigest()


def is_current(lib: str = LIB) -> bool:
    """Whether ``lib`` exists and was built from the sources as they are now."""
    try:
        with open(lib + ".sha256") as f:
            return os.path.exists(lib) and f.read().strip() == source_digest()
    except OSError:
        return False


def _run(cmd: list[str], cwd: str | None = None) -> None:
    subprocess.run(cmd, check=True, cwd=cwd)


def _stem(path: str) -> str:
    return os.path.splitext(os.path.basename(path))[0]


def _cuid(path: str) -> str:
    return "-cuid=detfold_" + _stem(path)


def _device_pass(src: str, work: str, extra: list[str], temps: bool = False) -> str:
    bundle = os.path.join(work, _stem(src) + ".hipfb")
    cmd = [hipcc(), "--cuda-device-only", _cuid(src)] + common_flags() + device_flags() + extra
    if temps:
        cmd.append("-save-temps=obj")
    _run(cmd + ["-c", src, "-o", bundle], cwd=work)
    return bundle


def _kernel_object(src: str, work: str, extra: list[str]) -> str:
    bundle = _device_pass(src, work, extra)
    obj = os.path.join(work, _stem(src) + ".o")
    _run([hipcc(), "--cuda-host-only", _cuid(src)] + common_flags() + extra +
         ["-Xclang", "-fcuda-include-gpubinary", "-Xclang", bundle, "-c", src, "-o", obj])
    return obj


def _host_object(src: str, work: str, extra: list[str]) -> str:
    obj = os.path.join(work, _stem(src) + ".o")
    _run([hipcc()] + common_flags() + extra + ["-c", src, "-o", obj])
    return obj


def _objects(work: str, extra: list[str]) -> list[str]:
    kernels = DRAFT_KERNELS[::-1] + DECODE_KERNELS[::-1] + [KERNELS]
    hosts = HOST_SOURCES + [s for s in DECODE_SOURCES + DRAFT_SOURCES if s.endswith(".cpp") and s != BINDING]
    with ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as pool:
        jobs = [pool.submit(_kernel_object, s, work, extra) for s in kernels]
        jobs += [pool.submit(_host_object, s, work, extra) for s in hosts]
        return [j.result() for j in jobs]


def build_library(out: str = LIB, extra: list[str] | None = None) -> str:
    """Compile the sources into ``out`` (atomically replaced) and record the
    source digest beside it (only for the default flags)."""
    extra = extra or []
    work = tempfile.mkdtemp(prefix="detfold_build_")
    try:
        objs = _objects(work, extra)
        tmp = out + ".tmp%d" % os.getpid()
        _run([hipcc()] + link_flags() + ["-o", tmp] + objs)
        os.replace(tmp, out)
    finally:
        shutil.rmtree(work, ignore_errors=True)
    digest = out + ".sha256"
    if extra:
        if os.path.exists(digest):
            os.remove(digest)
    else:
        with open(digest, "w") as f:
            f.write(source_digest() + "\n")
    return out


def build_binding(out: str = BINDING_LIB) -> str | None:
    """Compile bind.cpp, the C++ side of decode.py's calls (host code only),
    against the installed torch.  It holds the digest of the sources, so that
    it is never used beside a library of other ones.  Without torch there are no
    such calls, and nothing is built."""
    import sysconfig

    try:
        import torch
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        print("torch is not installed: %s, the C++ side of decode.py, is not built" % os.path.basename(out))
        return None
    from torch.utils import cpp_extension
    tmp = out + ".tmp%d" % os.getpid()
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
             '-DDETFOLD_BUILT_FROM="%s"' % source_digest(),
             "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"]]
    for path in cpp_extension.include_paths():
        flags += ["-isystem", path]
    _run(["g++"] + flags + [BINDING, "-o", tmp, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
                            "-lc10", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, out)
    return out


def save_temps(outdir: str, src: str | None = None) -> None:
    """Keep the gfx950 assembly of a file's device pass (for reading our own
    ISA); the fold's unless another is named."""
    os.makedirs(outdir, exist_ok=True)
    _device_pass(src or KERNELS, outdir, [], temps=True)


if __name__ == "__main__":
    print(build_library())
    print(build_binding())
