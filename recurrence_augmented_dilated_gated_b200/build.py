"""Build librat.so (every CUDA source under csrc/) for sm_100a with nvcc, and
_binding.so (csrc/binding.cpp, the Python binding's native part) with g++.

Both are built in-tree, next to this file, so they ship with the package.
_binding.so only makes calls shorter on the host: without it the package does
the same checks in Python, so a failed g++ is a warning.
"""
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "librat.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_STAMP = os.path.join(HERE, "_binding.stamp")   # what BINDING was built for
BUILD_DIR = os.path.join(ROOT, "_build")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def start_binding(out):
    """Start the compilation of the binding's native part against the installed torch."""
    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-DRAT_BUILT_FOR=\"%s\"" % binding_target(), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, BINDING_SOURCE, "-o", out]
    for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += ["-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        warnings.warn("%s: calls take their checks in Python" % e)
        return None


def binding_target():
    """The torch and the Python whose headers the binding's native part is compiled against."""
    import torch

    return "torch %s %s %s" % (torch.__version__, sysconfig.get_config_var("SOABI"), torch._C._GLIBCXX_USE_CXX11_ABI)


def binding_up_to_date():
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP) as f:
        if f.read() != binding_target():
            return False
    return os.path.getmtime(BINDING) >= os.path.getmtime(BINDING_SOURCE)


def finish_binding(proc, tmp):
    out, _ = proc.communicate()
    if proc.returncode:
        sys.stderr.write(out.decode())
        warnings.warn("g++ failed for %s: calls take their checks in Python" % BINDING_SOURCE)
        return
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP + ".tmp%d" % os.getpid(), "w") as f:
        f.write(binding_target())
    os.replace(f.name, BINDING_STAMP)


def build(force=False, verbose=False, ptxas_v=False):
    binding = None
    if force or not binding_up_to_date():
        tmp = BINDING + ".tmp%d" % os.getpid()
        binding = start_binding(tmp)
    lib = build_library(force, verbose, ptxas_v)
    if binding:
        finish_binding(binding, tmp)
    return lib


def build_library(force=False, verbose=False, ptxas_v=False):
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_v else []) + ["-dc" if False else "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_v or p.returncode):
            sys.stdout.write(out.decode())
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp%d" % os.getpid()
    link = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
    subprocess.check_call(link)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_v="--ptxas" in sys.argv))
