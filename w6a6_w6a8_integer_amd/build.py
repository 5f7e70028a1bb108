"""Build libflexq.so (the gfx950 HIP kernels behind include/flexq.h) in-tree with hipcc,
and _serve.so, the Python binding of the decoding-step calls, with the host compiler."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libflexq.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["api.hip", "pack_quant.hip", "gemm_decode.hip", "gemm_prefill.hip", "group_dots.hip",
           "peaks.hip", "gemm_prefill_ws.hip", "serve_api.hip", "serve_gemv.hip",
           "serve_cache.hip", "serve_attention.hip", "serve_kv4_cache.hip",
           "serve_kv4_attention.hip", "serve_lora.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # no packed fp32 VALU ops in generated code; the host pass warns and ignores it
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in ordinary VGPRs: the fused dequant reads every one with the VALU,
    # and results parked in AGPRs would cost a copy each
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    # the quantizers and the fused dequant need exact IEEE binary32
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-mcode-object-version=5",
    "-I", os.path.join(ROOT, "include"),
]


BINDING = os.path.join(PKG, "_serve.so")


class NoBinding(Exception):
    """What the binding needs and this host lacks."""


def binding_command(out: str) -> list[str]:
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        raise NoBinding(f"torch cannot be imported ({e})") from e

    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        raise NoBinding(f"there is no host compiler {cxx}")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [*cpp_extension.include_paths("cuda"), sysconfig.get_paths()["include"]]
    for header in ("torch/csrc/autograd/python_variable.h", "c10/hip/HIPStream.h", "Python.h"):
        if not any(os.path.exists(os.path.join(p, header)) for p in include):
            raise NoBinding(f"there is no {header}")
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            # what torch's own headers ask for on ROCm
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-isystem{p}" for p in include), os.path.join(CSRC, "serve_binding.cpp"),
            f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip",
            f"-Wl,-rpath,{lib}", "-o", out]


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Builds both.  The library needs hipcc alone: where the host lacks what the binding
    needs, it is left out (the calls that need it say so), and where the binding does not
    compile, the library is there before the error is raised."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs, procs = [], []
    try:
        cmd = binding_command(BINDING + ".tmp")
    except NoBinding as e:
        binding = None
        print(f"{os.path.basename(BINDING)} is not built: {e}", file=sys.stderr)
    else:
        if verbose:
            print(" ".join(cmd), flush=True)
        binding = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        procs.append(("serve_binding.cpp", binding))
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # hipcc's host pass does not know the packed-fp32 feature; drop that notice
        lines = [l for l in text.splitlines() if "packed-fp32-ops" not in l]
        if lines and (verbose or p.returncode):
            print(f"[{src}]\n" + "\n".join(lines), file=sys.stderr)
        if p.returncode:
            failed.append(src)
    if set(failed) - {"serve_binding.cpp"}:
        raise RuntimeError(f"the compiler failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    if os.path.exists(BINDING):
        os.remove(BINDING)  # none is left that was built for another library
    os.replace(tmp, LIB)
    if failed:
        raise RuntimeError(f"the compiler failed for {failed}; {LIB} is built")
    if binding is not None:
        os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
