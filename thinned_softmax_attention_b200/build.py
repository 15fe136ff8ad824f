"""Build libthin_attn.so in-tree for sm_100a with nvcc, and the paged operators' Python binding with g++.

    python -m thinned_softmax_attention_b200.build [--force]
"""
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libthin_attn.so")
BINDING = os.path.join(HERE, "_paged.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "paged_binding.cpp")
BINDING_TORCH = os.path.join(ROOT, "_build", "paged_binding.torch")   # the torch that the binding was built against
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + glob.glob(os.path.join(HERE, "csrc", "*.h"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def newer(target, inputs):
    """Whether the target exists and none of its inputs has changed since."""
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in inputs + [__file__])


def library_up_to_date():
    return newer(LIB, sources() + headers())


def torch_version():
    from importlib.metadata import version
    return version("torch")


def binding_up_to_date():
    try:
        built_against = open(BINDING_TORCH).read()
    except OSError:
        return False
    return built_against == torch_version() and newer(BINDING, [BINDING_SOURCE, os.path.join(ROOT, "include", "thin_attn.h")])


def up_to_date():
    return library_up_to_date() and binding_up_to_date()


def build_binding():
    """_paged.so against the installed torch (its C++ ABI and libraries)."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(os.environ.get("NVCC", "nvcc"))))), "include")
    tmp = BINDING + ".tmp"
    # nvcc's host compiler, whose C++ library is torch's too (a compiler that links its own statically is not)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                           "-isystem", os.path.join(base, "include"),
                           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-I", os.path.join(ROOT, "include"),
                           BINDING_SOURCE, "-o", tmp, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
                           "-ltorch", "-ltorch_python"])
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_TORCH), exist_ok=True)
    with open(BINDING_TORCH, "w") as f:
        f.write(torch_version())


def build(force=False, verbose=False):
    # the library needs nvcc alone: it is built first, whatever the binding lacks
    if force or not library_up_to_date():
        build_library(verbose)
    if force or not binding_up_to_date():
        build_binding()
    return LIB


def build_library(verbose=False):
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
               "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp"
    subprocess.check_call([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
                           "-Xcompiler", "-fPIC", "-cudart", "static"])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
