"""Builds libvsl.so (the C-ABI library) in-tree with nvcc for sm_100a, the
Python side of its shortest calls (_binding.so, g++ against torch's headers),
and the test library tests/libvsl_test.so (the same objects plus the test-only
probes of tests/csrc/vsl_test_probes.cu; never part of libvsl.so)."""
import os
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libvsl.so")
BINDING_SRC = os.path.join(CSRC, "vsl_binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
TEST_SRC = os.path.join(ROOT, "tests", "csrc", "vsl_test_probes.cu")
TEST_LIB_PATH = os.path.join(ROOT, "tests", "libvsl_test.so")
SOURCES = ["vsl_api.cu", "vsl_gemm.cu", "vsl_sample.cu", "vsl_verify.cu", "vsl_processed.cu", "vsl_tiles.cu",
           "vsl_adapters.cu", "vsl_scores.cu", "vsl_preference.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def needs_build():
    built = (LIB_PATH, TEST_LIB_PATH, BINDING_PATH)
    if not all(os.path.exists(p) for p in built):
        return True
    t = min(os.path.getmtime(p) for p in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps += [os.path.join(ROOT, "include", "vsl.h"), TEST_SRC]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _compile(src, obj, verbose):
    cmd = [_nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)


def _link(objs, path):
    tmp = path + ".tmp"
    subprocess.run([_nvcc(), "-shared", *ARCH, "-o", tmp, *objs], check=True)
    os.replace(tmp, path)


def _build_binding(verbose):
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[x for p in include for x in ("-isystem", p)],
           BINDING_SRC, "-o", tmp, "-L" + PKG_DIR, "-l:libvsl.so", "-L" + os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING_PATH)


def build(force=False, verbose=False):
    """Compile every CUDA source, link libvsl.so next to this file (and the test library), and compile the binding."""
    if not force and not needs_build():
        return LIB_PATH
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        _compile(os.path.join(CSRC, src), obj, verbose)
        objs.append(obj)
    _link(objs, LIB_PATH)
    _build_binding(verbose)
    probe = os.path.join(objdir, "vsl_test_probes.o")
    _compile(TEST_SRC, probe, verbose)
    _link(objs + [probe], TEST_LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB_PATH)
