"""Kernels whose wait for a bulk copy runs out, in CTAs that a test names: the library's own
sources, compiled with a probe that says that nothing came."""
import ctypes
import os
import subprocess

SOURCE = r"""
#include <cuda_runtime.h>
#define mbar_try_wait_sleep really_wait
#include "sc_tma.cuh"
#undef mbar_try_wait_sleep
namespace scg {
// CTA 1: the team (of TEAM threads) 2 never sees its copies; CTA 3: none of an odd phase.
// (Giving up takes a million probes, long after the copies have come.)
__device__ __forceinline__ bool mbar_try_wait_sleep(uint32_t bar, uint32_t parity, uint32_t) {
    const bool ok = really_wait(bar, parity, 20);
    const bool late = (blockIdx.x == 1 && threadIdx.x / TEAM == 2) || (blockIdx.x == 3 && parity == 1);
    return ok && !late;
}
}  // namespace scg
#include "FILE"
namespace scg {
void count_launches(int) {}
long long seq_sms() { return 152; }
}  // namespace scg
MORE
"""


def build(folder, file, more, team):
    """A ctypes library of `file` from the library's sources and the entry points `more`."""
    from stream_compaction_gb300 import build as b
    src, lib = os.path.join(folder, "late.cu"), os.path.join(folder, "late.so")
    with open(src, "w") as f:
        f.write(SOURCE.replace("FILE", file).replace("MORE", more).replace("TEAM", str(team)))
    subprocess.run([b.nvcc()] + b.NVCC_FLAGS + ["-I" + b.CSRC, "-shared", src, "-o", lib], check=True)
    return ctypes.CDLL(lib)
