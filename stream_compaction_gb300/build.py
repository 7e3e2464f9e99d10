"""Build libsc_gb300.so in-tree with nvcc (sm_103a only), and the binding of the
sequence operators to torch tensors with the host compiler.

Each .cu translation unit is compiled in parallel into _build/, then linked
into stream_compaction_gb300/libsc_gb300.so (CUDA runtime linked statically);
sc_bind.cpp becomes stream_compaction_gb300/_seqbind.so on top of it.  The
library needs nvcc alone: it is linked whatever becomes of the binding, which
is left out where torch is not installed and raises where it does not build.
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


def _newest(names):
    files = [os.path.join(CSRC, f) for f in names]
    files += [os.path.join(ROOT, "include", h) for h in ("sc_scan.h", "sc_seq.h")]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _library_up_to_date() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(f for f in os.listdir(CSRC) if f != "sc_bind.cpp")


def _torch_dir():
    """Folder of the installed torch (which is not imported), or None."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_up_to_date() -> bool:
    """Newer than its sources and than the installed torch, whose headers and libraries it is built on."""
    if not os.path.exists(BIND):
        return False
    version = os.path.join(_torch_dir() or "", "version.py")
    built = os.path.getmtime(BIND)
    return built >= _newest(["sc_bind.cpp"]) and not (os.path.exists(version) and os.path.getmtime(version) > built)


def up_to_date() -> bool:
    """Whether there is nothing to build: the library and, where torch is, the binding."""
    return _library_up_to_date() and (_torch_dir() is None or _binding_up_to_date())


def _bind_commands(cc: str, torch_dir: str):
    """Compile and link commands of the binding."""
    import sysconfig
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
    link = [gxx, "-shared", "-o", tmp, obj, LIB, "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return compile_, link, tmp


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    torch_dir = _torch_dir()
    commands = _bind_commands(cc, torch_dir) if torch_dir and (force or not _binding_up_to_date()) else None
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside the library's compilation
        binding = ex.submit(_run, commands[0], "the binding's compilation") if commands else None
        if force or not _library_up_to_date():
            _build_library(cc, verbose, extra_flags)
        if binding:
            binding.result()
    if commands:
        _run(commands[1], "the binding's link")
        os.replace(commands[2], BIND)
    elif not torch_dir:
        sys.stderr.write("torch is not installed: the sequence operators' binding to its tensors is not built\n")
    return LIB


def _run(command, what: str) -> str:
    try:
        r = subprocess.run(command, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError("%s failed: %s" % (what, e)) from e
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, r.stdout, r.stderr))
    return r.stderr


def _build_library(cc: str, verbose: bool, extra_flags) -> None:
    flags = list(NVCC_FLAGS) + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(BUILD, src[:-3] + ".o")
        cmd = [cc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, "nvcc on %s" % src)

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for (obj, log) in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-cudart", "static", "-Xlinker",
                                                                           "-soname=libsc_gb300.so"]
    _run(cmd, "link")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
