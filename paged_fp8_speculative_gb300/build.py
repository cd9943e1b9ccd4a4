"""Build libmtpattn.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

Every ``csrc/*.cu`` file compiles to an object in parallel, then one link makes
``paged_fp8_speculative_gb300/libmtpattn.so``; beside them g++ compiles ``csrc/binding.cpp``, the
compiled part of the Python binding, linked to that library.  The library needs neither PyTorch nor
Python's headers: it is linked first, and is there for C programs where the binding cannot be built
(which is an error all the same).  Run as ``python -m paged_fp8_speculative_gb300.build`` or through
``__graft_entry__.build()``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmtpattn.so")
# with the interpreter's own suffix, so that no other version of Python takes it for its own
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmtpattn.so")


def _torch_dir() -> str:
    """PyTorch's folder, without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found: the Python binding is compiled against it")
    return list(spec.submodule_search_locations)[0]


def binding_commands():
    """g++ command lines: compile csrc/binding.cpp, link it."""
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "binding.o")
    includes = [os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{d}" for d in includes], "-c",
                os.path.join(CSRC, "binding.cpp"), "-o", obj]
    link = ["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L", PKG, "-lmtpattn",
            "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build(verbose: bool = False, extra_flags=(), lib_path: str = LIB) -> str:
    """Compile every csrc/*.cu and link ``lib_path``.  ``extra_flags`` (e.g. the test-only
    -DMTPATTN_WAIT_CYCLES / -DMTPATTN_TEST_STALL of the wait-limit test) go to every nvcc;
    such builds use their own object folder and library path."""
    obj_dir = BUILD if lib_path == LIB else os.path.join(BUILD, os.path.splitext(
        os.path.basename(lib_path))[0])
    os.makedirs(obj_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cc = nvcc()
    procs = []
    objs = []
    for src in srcs:
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    product = lib_path == LIB
    binding, no_binding = None, ""
    if product:
        try:
            compile_binding, link_binding = binding_commands()
            if verbose:
                print(" ".join(compile_binding), flush=True)
            binding = subprocess.Popen(compile_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        except (RuntimeError, OSError) as e:         # no PyTorch, no g++
            no_binding = str(e)

    def ended(pr) -> bool:
        out, _ = pr.communicate()
        if pr.returncode != 0 or (verbose and out):
            sys.stdout.write(out.decode(errors="replace"))
        return pr.returncode == 0

    failed = [src for src, pr in procs if not ended(pr)]
    if binding and not ended(binding):
        no_binding = "compiling csrc/binding.cpp failed"
    if failed:
        raise RuntimeError(f"compiling failed for {failed}")
    tmp = lib_path + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, lib_path)
    if product:
        if not no_binding and subprocess.call(link_binding) != 0:
            no_binding = "linking it failed"
        if no_binding:
            raise RuntimeError(f"{os.path.basename(lib_path)} is built, the Python binding is not: {no_binding}")
        os.replace(BINDING + ".tmp", BINDING)
        untagged = os.path.join(PKG, "_binding.so")  # what builds made before the name had a suffix
        if os.path.exists(untagged):
            os.remove(untagged)
    return lib_path


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
