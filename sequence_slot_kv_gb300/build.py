"""Build libslotkv.so in place for sm_103a.

The translation units compile in parallel (one per head dim for the decode
and the tensor-core prefill kernels and their scored forms, the request-length
kernels, the host side, the allocation-free entry point), then link into
``sequence_slot_kv_gb300/libslotkv.so``.
"""
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libslotkv.so")
CALL = os.path.join(HERE, "_slotkv_call.so")  # the compiled calls of the Python binding
OBJDIR = os.path.join(HERE, "_build")
SOURCES = ["slotkv.cu", "decode_attn_hd64.cu", "decode_attn_hd128.cu", "decode_attn_hd256.cu",
           "noalloc.cu", "prefill_tc_hd64.cu", "prefill_tc_hd128.cu", "scored_decode_hd64.cu",
           "scored_decode_hd128.cu", "scored_decode_hd256.cu", "scored_prefill_hd64.cu",
           "scored_prefill_hd128.cu", "maps.cu"]
DEPS = ["params.h", "maps.h", "score_rule.cuh", "decode_attn.cuh", "decode_small.cuh",
        "prefill_tc.cuh", "tc_ops.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE] + ARCH


def _cuda_home():
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _stale(out, srcs):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in srcs)


def _call_flags():
    """Compile and link flags of the compiled calls, from the installed torch
    (found without importing it) and Python; None where their headers are
    missing, and the binding then makes the calls through ctypes alone."""
    spec = importlib.util.find_spec("torch")
    inc = sysconfig.get_paths()["include"]
    if spec is None or not os.path.exists(os.path.join(inc, "Python.h")):
        return None
    root = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(root, "include", "torch", "csrc", "autograd",
                                       "python_variable.h")):
        return None
    lib = os.path.join(root, "lib")
    cflags = ["-O2", "-std=c++17", "-fPIC", "-I", inc, "-I", os.path.join(root, "include"),
              "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
              "-I", os.path.join(_cuda_home(), "include")]
    ldflags = ["-L" + HERE, "-lslotkv", "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-lc10_cuda", "-Wl,-rpath,$ORIGIN:" + lib]
    return cflags, ldflags


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _call_stamp(flags):
    """What the compiled calls are made for beside their own sources: the torch
    and the Python whose headers they were compiled with."""
    spec = importlib.util.find_spec("torch")
    torch_version = _read(os.path.join(spec.submodule_search_locations[0], "version.py"))
    return repr((flags, torch_version, sys.version))


def build(force=False, verbose_ptxas=False):
    os.makedirs(OBJDIR, exist_ok=True)
    header = os.path.join(INCLUDE, "slotkv.h")
    deps = [os.path.join(CSRC, d) for d in DEPS] + [header]
    procs, objs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path] + deps):
            cmd = ["nvcc"] + NVCC_FLAGS + ["-c", path, "-o", obj]
            if verbose_ptxas:
                cmd += ["-Xptxas", "-v"]
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    flags = _call_flags()
    call_src, call_obj = os.path.join(CSRC, "call.cpp"), os.path.join(OBJDIR, "call.o")
    stamp_file = os.path.join(OBJDIR, "call.stamp")
    call_stale = False
    if flags is None:
        print("no headers of Python or torch: the compiled calls are not built")
        if os.path.exists(CALL):  # made for other headers, maybe other C declarations
            os.remove(CALL)
    else:
        stamp = _call_stamp(flags)
        call_stale = (force or _stale(call_obj, [call_src, header]) or
                      _read(stamp_file) != stamp)
    if call_stale:
        procs.append(("call.cpp", subprocess.Popen(
            ["g++"] + flags[0] + ["-c", call_src, "-o", call_obj], stdout=subprocess.PIPE,
            stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if verbose_ptxas or pr.returncode != 0:
            sys.stdout.write(out)
        if pr.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    if force or _stale(LIB, objs):
        cuda_lib = os.path.join(_cuda_home(), "lib64")
        cmd = ["nvcc", "-shared", "-o", LIB] + objs + ARCH + [
            "-cudart", "shared", "-Xlinker", "-rpath=" + cuda_lib]
        subprocess.run(cmd, check=True)
    if flags is not None and (call_stale or _stale(CALL, [call_obj, LIB])):
        subprocess.run(["g++", "-shared", "-o", CALL, call_obj] + flags[1], check=True)
        with open(stamp_file, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
