"""Build in-tree: libgemmrelu.so with nvcc for sm_103a (one translation unit), and beside it the
CPython extension _serving that hands torch tensors to it (g++, torch's headers; left out where
there is no torch, which the library itself does not need)."""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(CSRC, "gemm_relu_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("gemm_relu_kernels.cuh", "gemm_relu_splitk.cuh", "gemm_relu_2sm.cuh", "gemm_relu_gemv.cuh", "flash_attention.cuh", "sm103.cuh", "gemm_relu_stage.cuh",
                                                 "flash_attention_window.cuh", "flash_attention_window_api.cuh",
                                                 "kv_cache.cuh", "kv_attention.cuh", "kv_ragged.cuh", "kv_cache_api.cuh",
                                                 "rotary.cuh", "rotary_api.cuh", "cross_step.cuh")] + [
    os.path.join(INCLUDE, f) for f in ("gemm_relu.h", "flash_attention.h", "kv_cache.h", "rotary.h")]
LIB = os.path.join(PKG, "libgemmrelu.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


BINDING_SRC = os.path.join(CSRC, "serving_binding.cpp")
BINDING = os.path.join(PKG, "_serving" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_DEPS = [BINDING_SRC] + [os.path.join(INCLUDE, f) for f in
                                ("gemm_relu.h", "flash_attention.h", "kv_cache.h", "rotary.h")]


def _stale(target, deps):
    return not os.path.exists(target) or any(
        os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _has_torch():
    try:
        return importlib.util.find_spec("torch") is not None
    except ValueError:   # a placeholder in sys.modules
        return False


def needs_build():
    return _stale(LIB, DEPS) or (_has_torch() and _stale(BINDING, BINDING_DEPS))


def build_binding():
    import torch
    root = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wextra",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_path("include"), "-isystem", os.path.join(cuda, "include"),
           "-o", BINDING, BINDING_SRC, f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.run(cmd, check=True)
    return BINDING


def build(verbose=False, extra=()):
    """Compile both at the same time, the library alone without torch."""
    failed = []

    def binding():
        try:
            build_binding()
        except Exception as e:   # raised again below, in the caller's thread
            failed.append(e)
    side = threading.Thread(target=binding)
    if _has_torch():
        side.start()
    else:
        print("no torch: the serving operators' extension is not built", file=sys.stderr)
    try:
        cmd = [nvcc(), *NVCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", *extra, "-o", LIB, *SOURCES]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    finally:
        if side.ident is not None:
            side.join()
    if failed:
        raise failed[0]
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
