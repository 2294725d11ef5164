"""Build the CUDA library libattn_gb300.so in-tree with nvcc (sm_103a only).

    python -m attn_fwd_02_gb300.build [--verbose-ptxas]

Each translation unit under csrc/ compiles in parallel to an object file under
_build/, then nvcc links them into attn_fwd_02_gb300/libattn_gb300.so with the
CUDA runtime linked statically (the library loads without a GPU present).
g++ also compiles csrc/fastcall.cpp, the binding's compiled argument marshalling, against the
installed torch, into a file named by that torch's and this Python's versions; where that is
not possible (no Python or torch headers), the binding marshals in Python alone, with the
same results.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
OUT = os.path.join(HERE, "libattn_gb300.so")
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden,-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
SOURCES = ["abi.cu", "prefill.cu", "prefill_scoremod.cu", "decode.cu", "kvcache.cu", "backward.cu", "backward_scoremod.cu", "append_rope.cu",
           "decode_scoremod.cu", "decode_shared.cu"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime(src: str) -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(ROOT, "include", "attn_gb300.h"))
    files.append(src)
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, verbose_ptxas: bool) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= _deps_mtime(path):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", path, "-o", obj + ".tmp"]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def fastcall_path(torch_version: str) -> str:
    """The compiled marshalling for one torch (its full version) and this Python: one built for others is not found."""
    return os.path.join(HERE, f"_fastcall-{torch_version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _installed_torch() -> tuple[str, str]:
    """Folder and full version of the installed torch, which is not imported ('' without one)."""
    spec = importlib.util.find_spec("torch")
    folder = spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else ""
    try:
        with open(os.path.join(folder, "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)['\"]", f.read(), re.M)
    except OSError:
        found = None
    return folder, found.group(1) if found else ""


def _compile_fastcall() -> str | None:
    header = os.path.join(ROOT, "include", "attn_gb300.h")
    torch, version = _installed_torch()
    if not version:
        sys.stderr.write("fastcall.cpp was not compiled (the binding marshals in Python): no torch\n")
        return None
    out = fastcall_path(version)
    if os.path.exists(out) and os.path.getmtime(out) >= max(map(os.path.getmtime, (FAST_SRC, header))):
        return out
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = [os.path.dirname(header), os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f'-DATTN_TORCH_VERSION="{version}"',
           *(f"-I{i}" for i in inc), FAST_SRC, "-o", tmp, "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stderr if r.returncode else ""
    except OSError as e:
        why = str(e)
    if why:
        sys.stderr.write(f"fastcall.cpp was not compiled (the binding marshals in Python):\n{why[-2000:]}\n")
        return None
    os.replace(tmp, out)
    return out


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD, f))
        for f in os.listdir(HERE):
            if f.startswith("_fastcall") and f.endswith(".so"):
                os.remove(os.path.join(HERE, f))
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = ex.submit(_compile_fastcall)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
        fast.result()
    if os.path.exists(OUT) and os.path.getmtime(OUT) >= max(os.path.getmtime(o) for o in objs) and not force:
        return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args()
    print(build(verbose_ptxas=args.verbose_ptxas, force=args.force))
