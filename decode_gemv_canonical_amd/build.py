"""Build libuw.so in-tree: hipcc for the gfx950 kernels, g++ for the host C++ (no
library beyond the HIP runtime is linked); and _uw_torch.so, the C++ side of
the Python binding (torch's headers and libraries, g++), where torch is there:
C callers need libuw.so alone.

    python decode_gemv_canonical_amd/build.py

(run as a file: importing the package would first load the library being
rebuilt)
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libuw.so")
BINDING = os.path.join(CSRC, "binding", "uw_torch.cpp")
TORCH_LIB = os.path.join(LIBDIR, "_uw_torch.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
ARCH = "gfx950"

HIPCC_FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
               # packed fp32 instructions are kept out of every kernel
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall", "-Wno-unused-function"]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", "-Wall", "-Wextra",
             "-Wno-unused-parameter"]


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l and l.strip())
    if verbose and err:
        print(err, file=sys.stderr)


def _binding_command(out: str) -> list[str] | None:
    # torch is found without importing it; its import takes longer than this compile
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return None
    torch_dir = torch.submodule_search_locations[0]
    inc = os.path.join(torch_dir, "include")
    return ["g++", *CXX_FLAGS, "-DUSE_ROCM", "-shared", "-Wno-sign-compare", f"-isystem{inc}",
            f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-I{sysconfig.get_paths()['include']}",
            BINDING, "-o", out, f"-L{os.path.join(torch_dir, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    jobs = []
    objs = []
    for name in sorted(os.listdir(CSRC)):
        src = os.path.join(CSRC, name)
        obj = os.path.join(BUILD, name + ".o")
        if name.endswith(".hip"):
            jobs.append([os.path.join(ROCM, "bin", "hipcc"), *HIPCC_FLAGS, "-c", src, "-o", obj])
        elif name.endswith(".cpp"):
            jobs.append(["g++", *CXX_FLAGS, "-c", src, "-o", obj])
        else:
            continue
        objs.append(obj)
    binding = _binding_command(TORCH_LIB + ".tmp")
    if binding:
        jobs.append(binding)
    else:
        print("torch is not installed: libuw.so is built without the Python binding's _uw_torch.so", file=sys.stderr)
    with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        list(ex.map(lambda c: _run(c, verbose), jobs))
    tmp = LIB + ".tmp"
    _run([os.path.join(ROCM, "bin", "hipcc"), "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs,
          "-lpthread"], verbose)
    os.replace(tmp, LIB)
    if binding:
        os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
