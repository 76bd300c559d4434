"""Build librr.so (the HIP library behind include/rr.h) for gfx950, in-tree."""
from __future__ import annotations

import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BLOCK = os.path.join(HERE, "csrc_block")  # a block's operators between two collectives
LIB = os.path.join(HERE, "librr.so")
# the Python module that marshals the usual calls of a block's operators; links librr.so
BINDING_SOURCE = os.path.join(BLOCK, "blk_binding.cpp")
BINDING = os.path.join(HERE, "_block.so")
# one translation unit per kernel family (the in-place ring: one per element
# type), and the host side with the C ABI
SOURCES = [os.path.join(CSRC, f) for f in
           ("rr_ring_i32.hip", "rr_ring_f32.hip", "rr_ring_bf16.hip", "rr_ring_f16.hip",
            "rr_staged_kernel.hip", "rr_aux_kernels.hip", "rr_api.hip")]
SOURCES += [os.path.join(BLOCK, f) for f in ("blk_expert.hip", "blk_norm.hip", "blk_norm_f32.hip",
                                                "blk_norm_bf16.hip", "blk_norm_f16.hip", "blk_linear.hip",
                                                "blk_gemm_bf16.hip", "blk_gemm_f16.hip")]
HEADERS = [os.path.join(CSRC, "rr_device.hpp"), os.path.join(CSRC, "rr_kernels.hpp"),
           os.path.join(CSRC, "rr_ring_kernel.hpp"), os.path.join(BLOCK, "blk_common.hpp"),
           os.path.join(BLOCK, "blk_gemm.hpp"), os.path.join(BLOCK, "blk_norm.hpp"),
           os.path.join(ROOT, "include", "rr.h")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 instructions stay off: hipcc would form them from plain float code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def declared_functions() -> list[str]:
    """The functions include/rr.h declares: the library's whole dynamic interface."""
    with open(os.path.join(ROOT, "include", "rr.h")) as fh:
        text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
    decl = re.compile(r"^(?:const\s+)?\w+[\s*]+(\w+)\s*\(", re.M)
    return sorted(set(decl.findall(text)))


def _version_script(path: str) -> str:
    """Export the declared functions only; kernel handles and helpers stay local."""
    with open(path, "w") as fh:
        fh.write("{\n  global:\n")
        fh.writelines("    %s;\n" % name for name in declared_functions())
        fh.write("  local: *;\n};\n")
    return path


def build(force: bool = True, verbose: bool = False) -> str:
    """Compile every HIP source (in parallel) and link ring_allreduce_amd/librr.so."""
    newest = max(os.path.getmtime(p) for p in SOURCES + HEADERS + [BINDING_SOURCE])
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in (LIB, BINDING)):
        return LIB
    include = ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", BLOCK]
    with tempfile.TemporaryDirectory(prefix="rr_build_") as tmpdir:
        objects = [os.path.join(tmpdir, os.path.basename(src) + ".o") for src in SOURCES]

        def compile_one(job):
            src, obj = job
            cmd = [HIPCC, *FLAGS, *include, "-c", "-o", obj, src]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)

        with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
            list(pool.map(compile_one, zip(SOURCES, objects)))
        tmp = LIB + ".tmp%d" % os.getpid()
        script = _version_script(os.path.join(tmpdir, "exports.map"))
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC",
               "-Wl,--version-script=" + script, "-o", tmp, *objects]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """Compile and link the module ring_allreduce_amd._block against librr.so and torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [os.path.join(ROOT, "include"), *cpp_extension.include_paths(),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include")]
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-DUSE_ROCM=1",
           "-D__HIP_PLATFORM_AMD__=1",         # host code: what hipcc defines for device code
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           *("-I" + p for p in includes), "-x", "c++", BINDING_SOURCE, "-o", tmp,
           "-L" + HERE, "-lrr", "-L" + torch_lib, "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True))
