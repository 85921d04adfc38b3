"""Build libnf.so in-tree: every csrc/*.cu compiled for sm_103a in parallel,
then linked into row_normalization_inner_gb300/libnf.so; and _tensors.so, the
native part of the token-side operators' tensor helpers (csrc/tensors.cpp,
against the installed Python, PyTorch and libnf.so).  libnf.so needs neither
Python nor PyTorch and is linked first; without PyTorch it is all that is
built.

    python -m row_normalization_inner_gb300.build [--force] [--ptxas-table]

Objects and the ptxas resource report (registers, spills, shared memory per
kernel) go to _build/ at the repository root; --ptxas-table prints that
report as a markdown table, one row per kernel instantiation.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnf.so")
TENSORS_SRC = os.path.join(CSRC, "tensors.cpp")
TENSORS = os.path.join(PKG, "_tensors.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-Xptxas", "-v", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _older(out, deps) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(p) > os.path.getmtime(out) for p in deps)


def _lib_stale() -> bool:
    return _older(LIB, _sources() + _headers())


def _abi() -> str:
    """What the helpers are compiled against, beside their sources: an upgrade
    of Python or PyTorch changes no file of this tree."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = ""
    return f"{sys.implementation.cache_tag} torch {version} {_torch_dir()}"


def _abi_file() -> str:
    return os.path.join(BUILD, "tensors.abi")


def _tensors_stale() -> bool:
    if _older(TENSORS, [TENSORS_SRC] + _headers()) or not os.path.exists(_abi_file()):
        return True
    with open(_abi_file()) as f:
        return f.read() != _abi()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _compile_tensors() -> str:
    import sysconfig
    obj = os.path.join(BUILD, "tensors.o")
    torch_inc = os.path.join(_torch_dir(), "include")
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", TENSORS_SRC, "-o", obj, "-isystem", torch_inc, "-isystem",
           os.path.join(torch_inc, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", cuda_inc]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {TENSORS_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd, out):
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _link_lib(results):
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (_, log), src in zip(results, _sources()):
            f.write(f"==== {os.path.basename(src)}\n{log}\n")
    _link([_nvcc()] + ARCH + ["-shared"] + [o for o, _ in results], LIB)


def _link_tensors(obj):
    torch_lib = os.path.join(_torch_dir(), "lib")
    _link(["g++", "-shared", obj, "-L", PKG, "-l:libnf.so", "-Wl,-rpath,$ORIGIN", "-L", torch_lib,
           f"-Wl,-rpath,{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], TENSORS)
    with open(_abi_file(), "w") as f:
        f.write(_abi())


def build(force: bool = False, verbose: bool = False) -> str:
    have_torch = _torch_dir() is not None
    if not have_torch and verbose:
        print("PyTorch is not installed: libnf.so alone is built, without the tensor helpers", file=sys.stderr)
    lib, tensors = force or _lib_stale(), have_torch and (force or _tensors_stale())
    if not lib and not tensors:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if lib else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        obj = ex.submit(_compile_tensors) if tensors else None
        results = list(ex.map(_compile, srcs))
        if lib:
            _link_lib(results)
        if tensors:
            _link_tensors(obj.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


def _demangle(names):
    try:
        r = subprocess.run(["c++filt"], input="\n".join(names), capture_output=True, text=True,
                           check=True)
        out = r.stdout.splitlines()
        if len(out) == len(names):
            return out
    except (OSError, subprocess.CalledProcessError):
        pass
    return names


def ptxas_table() -> str:
    """The ptxas report of the last build as a markdown table: per kernel
    instantiation its registers per thread, spill stores / loads, stack
    frame and static shared memory (dynamic shared memory is set at launch
    and is not in this report)."""
    import re
    path = os.path.join(BUILD, "ptxas.log")
    with open(path) as f:
        text = f.read()
    rows, src = [], None
    cur = None
    for line in text.splitlines():
        m = re.match(r"==== (\S+)", line)
        if m:
            src = m.group(1)
            continue
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            cur = {"src": src, "name": m.group(1), "regs": "", "spill_st": "0", "spill_ld": "0",
                   "stack": "0", "smem": "0"}
            rows.append(cur)
            continue
        if cur is None:
            continue
        m = re.search(r"(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m:
            cur["stack"], cur["spill_st"], cur["spill_ld"] = m.groups()
        m = re.search(r"Used (\d+) registers", line)
        if m:
            cur["regs"] = m.group(1)
            m2 = re.search(r"(\d+) bytes smem", line)
            if m2:
                cur["smem"] = m2.group(1)
    names = _demangle([r["name"] for r in rows])
    out = ["| file | kernel | registers | spill stores / loads (B) | stack (B) | static smem (B) |",
           "|---|---|---|---|---|---|"]
    for r, n in sorted(zip(rows, names), key=lambda t: (t[0]["src"] or "", t[1])):
        n = n.replace("(anonymous namespace)::", "").replace("nf::", "")
        n = re.sub(r"\([^()]*\)$", "", n)
        n = re.sub(r"^void ", "", n)
        out.append(f"| {r['src']} | `{n}` | {r['regs']} | {r['spill_st']} / {r['spill_ld']} | "
                   f"{r['stack']} | {r['smem']} |")
    return "\n".join(out)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    if "--ptxas-table" in sys.argv:
        print(ptxas_table())
