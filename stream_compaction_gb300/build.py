"""Build libsc_gb300.so in-tree with nvcc (sm_103a only), and the binding of the
sequence operators to torch tensors with the host compiler.

Each .cu translation unit is compiled in parallel into _build/, then linked
into stream_compaction_gb300/libsc_gb300.so (CUDA runtime linked statically);
sc_bind.cpp becomes stream_compaction_gb300/_seqbind.so on top of it.
Run ``python -m stream_compaction_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsc_gb300.so")
BIND = os.path.join(HERE, "_seqbind.so")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsc_gb300.so")


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(ROOT, "include", h) for h in ("sc_scan.h", "sc_seq.h")]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    newest = _deps_mtime()
    return all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BIND))


def _bind_commands(cc: str):
    """Compile and link commands of the binding (paths from the installed torch, without importing it)."""
    import importlib.util
    import sysconfig
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(cc)))
    obj = os.path.join(BUILD, "sc_bind.o")
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    gxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    compile_ = [gxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=1", "-c",
                os.path.join(CSRC, "sc_bind.cpp"), "-o", obj]
    for d in include:
        compile_ += ["-isystem", d]
    lib = os.path.join(torch_dir, "lib")
    tmp = BIND + ".tmp.%d" % os.getpid()
    link = [gxx, "-shared", "-o", tmp, obj, LIB, "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return compile_, link, tmp


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = list(NVCC_FLAGS) + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(BUILD, src[:-3] + ".o")
        cmd = [cc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    bind_compile, bind_link, bind_tmp = _bind_commands(cc)

    def compile_bind():
        r = subprocess.run(bind_compile, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("the binding's compilation failed:\n%s\n%s" % (r.stdout, r.stderr))

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        binding = ex.submit(compile_bind)
        results = list(ex.map(compile_one, srcs))
        binding.result()
    if verbose:
        for (obj, log) in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-cudart", "static", "-Xlinker",
                                                                           "-soname=libsc_gb300.so"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    r = subprocess.run(bind_link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding's link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(bind_tmp, BIND)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
