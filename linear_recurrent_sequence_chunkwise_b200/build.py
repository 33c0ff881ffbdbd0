"""Build step of the CUDA library: compiles every ``csrc/*.cu`` for sm_100a
into ``libretention.so`` and ``csrc/binding.cpp`` into ``_binding-torch<version>.so``
next to this file (in-tree, so they travel with the source tree).  Run as ``python linear_recurrent_sequence_chunkwise_b200/build.py`` (by path:
importing the package loads the library this script builds)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libretention.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(HERE, "csrc")]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + \
        glob.glob(os.path.join(HERE, "csrc", "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, jobs: int = 8) -> str:
    """Compile (in parallel, one object per source) and link the shared library."""
    binding = _start_binding(force)
    if not force and not _stale():
        _finish_binding(binding)
        return LIB
    objdir = os.path.join(ROOT, "_build", "obj")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        if len(procs) >= jobs:
            _wait(procs.pop(0), verbose)
    for p in procs:
        _wait(p, verbose)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    _finish_binding(binding)
    return LIB


def binding_path() -> str:
    """The Python binding is built against one torch, whose version its name carries:
    another torch finds none and builds its own."""
    import torch
    return os.path.join(HERE, f"_binding-torch{torch.__version__}.so")


def _start_binding(force: bool):
    """Start compiling the Python binding of the short calls (g++, against torch's headers)."""
    src, header = os.path.join(HERE, "csrc", "binding.cpp"), os.path.join(ROOT, "include", "retention.h")
    binding = binding_path()
    if not force and os.path.exists(binding) and os.path.getmtime(binding) > max(map(os.path.getmtime, (src, header))):
        return None
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths("cuda"), sysconfig.get_path("include"), os.path.join(ROOT, "include")]
    obj = os.path.join(ROOT, "_build", "obj", "binding.o")
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *["-I" + i for i in inc], "-c", src, "-o", obj]
    return obj, os.path.join(os.path.dirname(torch.__file__), "lib"), \
        subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish_binding(job):
    if job is None:
        return
    obj, torch_lib, p = job
    _wait(("binding.cpp", p), False)
    tmp = binding_path() + f".tmp{os.getpid()}"
    # the library next to it; torch's own are loaded by the time it is imported
    subprocess.check_call(["g++", "-shared", obj, "-o", tmp, "-L" + HERE, "-l:libretention.so", "-L" + torch_lib, "-ltorch_python",
                           "-ltorch_cuda", "-lc10_cuda", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, binding_path())


def _wait(item, verbose):
    src, p = item
    out, _ = p.communicate()
    text = out.decode(errors="replace")
    if p.returncode != 0:
        sys.stderr.write(text)
        raise RuntimeError(f"compiling {os.path.basename(src)} failed")
    if verbose and text.strip():
        sys.stderr.write(f"--- {os.path.basename(src)}\n{text}")


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
