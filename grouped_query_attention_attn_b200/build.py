"""Build libgqa.so in-tree with nvcc for sm_100a.

    python -m grouped_query_attention_attn_b200.build [--force] [--verbose]

Each .cu under csrc/ is compiled to an object in _build/ (in parallel), then
linked into grouped_query_attention_attn_b200/libgqa.so.  csrc/torch_binding.cpp
becomes the CPython extension _torch_binding.so (g++, torch's headers).  Objects
are rebuilt when their source or any header changed, the extension also when torch or
Python did.
"""

import argparse
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgqa.so")
TORCH_BINDING = os.path.join(PKG, "_torch_binding.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC,-O2,-Wall", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _compile(src, force, verbose, extra):
    obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj, ""
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stderr}")
    return obj, (res.stderr if verbose else "")


def torch_binding_target():
    """The torch and Python whose binary interfaces the torch binding is compiled against."""
    import torch
    return (f"torch {torch.__version__}, CXX11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('EXT_SUFFIX')}")


def torch_binding_fits():
    """Whether the present binding was built for torch_binding_target(): it holds that string."""
    try:
        with open(TORCH_BINDING, "rb") as f:
            return b"<" + torch_binding_target().encode() + b">" in f.read()
    except OSError:
        return False


def _build_torch_binding(force):
    src = os.path.join(CSRC, "torch_binding.cpp")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "gqa.h")))
    if not force and torch_binding_fits() and os.path.getmtime(TORCH_BINDING) >= newest:
        return
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    tmp = TORCH_BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DGQA_BUILT_FOR="<{torch_binding_target()}>"', *(f"-I{d}" for d in inc), src, "-o", tmp,
           f"-L{os.path.join(root, 'lib')}",
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_binding.cpp:\n{res.stderr}")
    os.replace(tmp, TORCH_BINDING)


def build_library(force=False, verbose=False, extra_flags=()):
    """Compile every CUDA source for sm_100a and link libgqa.so (returns its path), and
    build the torch binding, which needs torch and g++: without either the library is
    built alone, and what is missing is said on stderr."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = _sources()
    extra = list(extra_flags)
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, force, verbose, extra), srcs))
    objs = [o for o, _ in results]
    for _, log in results:
        if log:
            sys.stderr.write(log)
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, LIB)
    missing = [what for what, there in (("torch", importlib.util.find_spec("torch")), ("g++", shutil.which("g++")))
               if not there]
    if missing:
        sys.stderr.write(f"the torch binding is not built: no {' and no '.join(missing)}\n")
    else:
        _build_torch_binding(force)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    a = ap.parse_args()
    print(build_library(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
