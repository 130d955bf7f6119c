"""Build libpkv.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and
_marshal.so (the Python binding's argument checks) with the host compiler.

    python -m paged_kv_flight_b200.build [--force] [--ptxas-v]
"""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpkv.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cc")
MARSHAL = os.path.join(HERE, "_marshal.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-warn-spills",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "pkv.h"), os.path.join(ROOT, "include", "pkv_pages.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def marshal_stamp() -> str:
    """What a built module depends on besides its source: it has torch's and
    CPython's layouts compiled in."""
    import torch

    return f"torch {torch.__version__}, abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {sysconfig.get_config_var('SOABI')}"


def marshal_current(stamp: str) -> bool:
    if not os.path.exists(MARSHAL) or os.path.getmtime(MARSHAL) < os.path.getmtime(MARSHAL_SRC):
        return False
    with open(MARSHAL, "rb") as f:
        return b"\0" + stamp.encode() + b"\0" in f.read()


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """The binding's extension module, against the installed torch's headers.
    pkv.py does its work in Python where it is missing, so that a host without
    a C++ compiler or those headers still has the library; a module that could
    not be built again is removed."""
    try:
        import torch

        stamp = marshal_stamp()
        if not force and marshal_current(stamp):
            return MARSHAL
        base = os.path.dirname(torch.__file__)
        inc, new = os.path.join(base, "include"), f"{MARSHAL}.{os.getpid()}.so"
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DPKV_STAMP="{stamp}"', "-isystem",
               inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-I",
               sysconfig.get_paths()["include"], "-o", new, MARSHAL_SRC, "-L", os.path.join(base, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10"]
        if verbose:
            print(" ".join(cmd))
        try:
            subprocess.run(cmd, check=True)
            os.replace(new, MARSHAL)
        finally:
            if os.path.exists(new):
                os.remove(new)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        print(f"_marshal.so not built ({e}): the binding's checks stay in Python", file=sys.stderr)
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or needs_build() or extra:
        nvcc = os.environ.get("NVCC", "nvcc")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB, *sources()]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force="--force" in sys.argv, verbose=True, extra=extra))
