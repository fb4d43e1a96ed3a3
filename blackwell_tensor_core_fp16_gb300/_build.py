"""Build step for libgemm_f16.so (nvcc, sm_103a only) and the Python module _decode.so that links to
it (g++, where torch is installed); in-tree output."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
HEADERS = [os.path.join(ROOT, "include", h) for h in ("gemm_f16.h", "gdn.h", "decode.h")]
# translation units, compiled in parallel
SOURCES = ["gemm_f16.cu", "gdn.cu", "decode.cu", "gdn_step.cu", "qk_norm_rope.cu",
           "paged_attention.cu", "cache_fp8.cu", "paged_attention_fp8.cu", "linear_w4.cu"]
LIB_PATH = os.path.join(PKG_DIR, "libgemm_f16.so")
# the CPython module of the decode-step operators' torch entry points, linked to the library, and
# beside it the Python and torch that it was compiled for
BINDING = "decode_binding.cpp"
BINDING_PATH = os.path.join(PKG_DIR, "_decode.so")
BINDING_ABI = BINDING_PATH + ".abi"

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


def _stale(path: str, sources) -> bool:
    return not os.path.exists(path) or \
        any(os.path.getmtime(s) > os.path.getmtime(path) for s in sources)


def binding_abi():
    """The Python and torch that the binding is compiled for; None without torch, where there is no
    binding.  (Does not import torch, which takes seconds.)"""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "of no version"
    return f"{sysconfig.get_config_var('SOABI')}, torch {version}"


def _binding_stale() -> bool:
    abi = binding_abi()
    if abi is None:
        return False
    try:
        with open(BINDING_ABI) as f:
            made_for = f.read()
    except OSError:
        made_for = None
    return made_for != abi or _stale(BINDING_PATH, _sources())


def is_stale() -> bool:
    return _stale(LIB_PATH, _sources()) or _binding_stale()


def _binding_commands(obj: str, out: str):
    """g++ commands that compile and link the binding against this Python and this torch."""
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
    """Compile the sources (in parallel) and link libgemm_f16.so next to this file, and _decode.so
    where there is a torch to compile it for.  A binding that does not compile leaves the
    library usable: a RuntimeWarning says why, and the operators that need it raise."""
    if not force and not is_stale():
        return LIB_PATH
    tag = f"tmp{os.getpid()}"
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]
    library = force or _stale(LIB_PATH, _sources())
    abi = binding_abi()
    commands, objs = [], []
    for src in SOURCES if library else ():
        obj = os.path.join(PKG_DIR, f".{os.path.splitext(src)[0]}.{tag}.o")
        cmd = [_nvcc(), *compile_flags, "-c", "-o", obj, os.path.join(CSRC, src)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        commands.append(cmd)
        objs.append(obj)
    binding_obj = os.path.join(PKG_DIR, f".decode_binding.{tag}.o")
    tmp, binding_tmp = LIB_PATH + "." + tag, BINDING_PATH + "." + tag
    made, logs = (*objs, binding_obj, tmp, binding_tmp), []

    def run(cmd):
        """(what went wrong, or None) of a command."""
        try:
            p = subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:
            return f"{cmd[0]}: {e}"
        logs.append(p.stdout + p.stderr)
        return f"{cmd[0]} failed ({p.returncode}):\n{p.stdout}\n{p.stderr}" if p.returncode else None

    def compile_binding():
        """(what went wrong or None, the command that links)."""
        try:
            compile_, link = _binding_commands(binding_obj, binding_tmp)
        except (ImportError, OSError, RuntimeError) as e:
            return str(e), None
        return run(compile_), link

    try:
        with ThreadPoolExecutor(len(commands) + 1) as pool:
            binding = pool.submit(compile_binding) if abi is not None else None
            errors = [e for e in pool.map(run, commands) if e]
        if not errors and library:
            errors = [e for e in [run([_nvcc(), *NVCC_FLAGS, "-o", tmp, *objs])] if e]
        if errors:
            raise RuntimeError("\n".join(errors))
        if library:
            os.replace(tmp, LIB_PATH)
        if binding is not None:
            error, link = binding.result()
            error = error or run(link)
            if error:
                warnings.warn(f"{BINDING_PATH} is not built: {error}", RuntimeWarning)
            else:
                os.replace(binding_tmp, BINDING_PATH)
                with open(BINDING_ABI, "w") as f:
                    f.write(abi)
    finally:
        for path in made:
            if os.path.exists(path):
                os.unlink(path)
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
