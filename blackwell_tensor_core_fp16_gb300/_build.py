"""Build step for libgemm_f16.so (nvcc, sm_103a only) and the Python module _decode.so that links to
it (g++); in-tree output."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import tempfile

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
HEADERS = [os.path.join(ROOT, "include", h) for h in ("gemm_f16.h", "gdn.h", "decode.h")]
# translation units, compiled in parallel
SOURCES = ["gemm_f16.cu", "gdn.cu", "decode.cu", "gdn_step.cu", "qk_norm_rope.cu",
           "paged_attention.cu"]
LIB_PATH = os.path.join(PKG_DIR, "libgemm_f16.so")
# the CPython module of the decode-step operators' torch entry points, linked to the library
BINDING = "decode_binding.cpp"
BINDING_PATH = os.path.join(PKG_DIR, "_decode.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "-shared",
]


def _nvcc() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    for cand in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgemm_f16.so")


def _sources():
    srcs = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    return srcs + HEADERS


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return any(os.path.getmtime(s) > t for s in _sources())


def _binding_commands(obj: str, out: str):
    """g++ commands that compile and link the binding against this Python and this torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *(x for i in include for x in ("-isystem", i)),
                "-c", "-o", obj, os.path.join(CSRC, BINDING)]
    link = ["g++", "-shared", "-o", out, obj, "-L" + os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
            "-L" + PKG_DIR, "-l:libgemm_f16.so", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the sources (in parallel) and link libgemm_f16.so next to this file."""
    if not force and not is_stale():
        return LIB_PATH
    tag = f"tmp{os.getpid()}"
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(PKG_DIR, f".{os.path.splitext(src)[0]}.{tag}.o")
        cmd = [_nvcc(), *compile_flags, "-c", "-o", obj, os.path.join(CSRC, src)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                      text=True))
        objs.append(obj)
    binding_obj = os.path.join(PKG_DIR, f".decode_binding.{tag}.o")
    binding_tmp = BINDING_PATH + "." + tag
    binding_compile, binding_link = _binding_commands(binding_obj, binding_tmp)
    procs.append(subprocess.Popen(binding_compile, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                  text=True))
    errors, logs = [], []
    for p in procs:
        out, err = p.communicate()
        logs.append(out + err)
        if p.returncode != 0:
            errors.append(f"{p.args[0]} failed ({p.returncode}):\n{out}\n{err}")
    try:
        if errors:
            raise RuntimeError("\n".join(errors))
        tmp = LIB_PATH + "." + tag
        res = subprocess.run([_nvcc(), *NVCC_FLAGS, "-o", tmp, *objs], capture_output=True,
                             text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc link failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
        res = subprocess.run(binding_link, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"g++ link failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
        os.replace(binding_tmp, BINDING_PATH)
    finally:
        for obj in (*objs, binding_obj):
            if os.path.exists(obj):
                os.unlink(obj)
    if verbose:
        print("".join(logs))
    return LIB_PATH


def ptxas_report() -> dict:
    """Resource usage ptxas reports for every function of the library (nvcc -Xptxas -v): per
    mangled name, its stack frame, spill stores and spill loads in bytes, and, for kernels, the
    registers per thread.  Compiles into a temporary directory; the library is left as it is."""
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]
    funcs: dict = {}
    with tempfile.TemporaryDirectory() as tmp:
        procs = []
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.splitext(src)[0] + ".o")
            cmd = [_nvcc(), "-Xptxas=-v", *compile_flags, "-c", "-o", obj,
                   os.path.join(CSRC, src)]
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
        for src, p in procs:
            out, _ = p.communicate()
            if p.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src} ({p.returncode}):\n{out}")
            current = None
            for line in out.splitlines():
                m = re.search(r"Function properties for (\S+)", line)
                if m:
                    current = funcs.setdefault(m.group(1), {"source": src})
                    continue
                m = re.search(r"Compiling entry function '([^']+)'", line)
                if m:
                    current = funcs.setdefault(m.group(1), {"source": src})
                    current["entry"] = True
                    continue
                m = re.search(r"(\d+) bytes stack frame, (\d+) bytes spill stores, "
                              r"(\d+) bytes spill loads", line)
                if m and current is not None:
                    current.update(stack=int(m.group(1)), spill_stores=int(m.group(2)),
                                   spill_loads=int(m.group(3)))
                    continue
                m = re.search(r"Used (\d+) registers", line)
                if m and current is not None:
                    current["registers"] = int(m.group(1))
    return funcs
