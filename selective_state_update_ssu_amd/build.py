"""Compile the HIP sources into the in-tree shared library `_lib/libssu_amd.so`.

Every translation unit is compiled for gfx950 only, in parallel, then linked into
one shared library that exports the C ABI of include/ssu.h, include/ssd.h and
include/layer.h. Packed-fp32 VALU instructions are disabled for the device code.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIBRARY = os.path.join(LIB_DIR, "libssu_amd.so")
# Streaming reference kernels used by the benchmark only (bandwidth ceilings and
# counter calibration); not part of the SSU library.
STREAM_LIBRARY = os.path.join(LIB_DIR, "libssu_stream.so")
STREAM_SOURCES = ["stream_ceiling.hip"]

# Python side of include/layer.h: host code against torch's headers, linked to the library.
BINDING = os.path.join(LIB_DIR, "_layer_binding.so")
BINDING_SOURCE = "layer_binding.cpp"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("HIP_CXX", "/opt/rocm/llvm/bin/clang++")
ARCH = "gfx950"
SOURCES = ["ssu_api.hip", "ssu_kernels_f32.hip", "ssu_kernels_f16.hip", "ssu_kernels_bf16.hip",
           "ring_trackers.hip", "ssd_api.hip", "ssd_kernels_bf16.hip", "ssd_kernels_f16.hip",
           "layer_conv.hip", "layer_scan_api.hip", "layer_scan_f32.hip", "layer_scan_f16.hip",
           "layer_scan_bf16.hip", "layer_cache.hip"]
CXXFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    # hipcc's host pass does not know the device-only target feature; that note is noise.
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if noise not in l and "warning generated" not in l
                    and "warnings generated" not in l and l.strip())
    return msg


def _binding_flags():
    import sysconfig

    import torch
    import torch.utils.cpp_extension as ext
    include = ext.include_paths() + [sysconfig.get_paths()["include"], "/opt/rocm/include"]
    return ["-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f"-I{INCLUDE}", *[f"-isystem{p}" for p in include]]


def _compile(cmd, src):
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    return obj, _run([*cmd, "-c", os.path.join(CSRC, src), "-o", obj])


def _link_binding(obj):
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run([CXX, "-shared", "-fPIC", "-o", BINDING + ".tmp", obj,
          f"-L{LIB_DIR}", "-l:" + os.path.basename(LIBRARY), "-Wl,-rpath,$ORIGIN",
          f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"])
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False) -> str:
    """Compile every source and link the library; returns its path. The Python binding comes
    after it and needs torch and its headers: without torch the library is built alone."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    sources = SOURCES + STREAM_SOURCES
    try:
        import torch  # noqa: F401
    except ImportError:
        torch = None
    with ThreadPoolExecutor(max_workers=min(len(sources) + 1, os.cpu_count() or 1)) as ex:
        jobs = {s: ex.submit(_compile, [HIPCC, *CXXFLAGS], s) for s in sources}
        if torch is not None:
            jobs[BINDING_SOURCE] = ex.submit(lambda: _compile([CXX, *_binding_flags()],
                                                              BINDING_SOURCE))
    objs = {s: jobs[s].result() for s in sources}
    for lib, srcs in ((LIBRARY, SOURCES), (STREAM_LIBRARY, STREAM_SOURCES)):
        tmp = lib + ".tmp"
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp,
              *[objs[s][0] for s in srcs]])
        os.replace(tmp, lib)
    if torch is not None:
        objs[BINDING_SOURCE] = jobs[BINDING_SOURCE].result()
        _link_binding(objs[BINDING_SOURCE][0])
    else:
        print(f"torch is not importable: {BINDING} is not built", file=sys.stderr)
    for _, msg in objs.values():
        if msg and verbose:
            print(msg, file=sys.stderr)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
