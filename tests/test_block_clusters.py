"""Where the device holds no cluster of 16 CTAs, launches take 8: the host side of the two
kernels that ask for 16, compiled with CUDA calls that the test makes up."""
import os
import subprocess

import pytest

FAKES = r"""
#include <cstdio>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

static int asked = 0, launched = 0, device = 0, room[3] = {1, 1, 1};
static bool broken = false;
static unsigned cluster = 0, grid = 0;
static cudaError_t last = cudaSuccess;
static cudaError_t fake_occupancy(int* n, const void*, const cudaLaunchConfig_t* c) {
    ++asked;
    if (c->attrs[0].val.clusterDim.x != c->gridDim.x && c->gridDim.x % c->attrs[0].val.clusterDim.x) return cudaErrorInvalidValue;
    if (broken) return last = cudaErrorUnknown;
    *n = room[device];
    return cudaSuccess;
}
static cudaError_t fake_launch(const cudaLaunchConfig_t* c) {
    ++launched;
    cluster = c->attrs[0].val.clusterDim.x;
    grid = c->gridDim.x;
    return cluster > 8 && (room[device] == 0 || broken) ? last = cudaErrorInvalidClusterSize : cudaSuccess;
}
#define cudaFuncSetAttribute(...) cudaSuccess
#define cudaGetDevice(p) (*(p) = device, cudaSuccess)
#define cudaGetLastError() (last = cudaSuccess)
#define cudaOccupancyMaxActiveClusters(n, k, c) fake_occupancy(n, k, c)
#define cudaLaunchKernelEx(c, ...) fake_launch(c)
#define cudaLaunchKernelExC(c, ...) fake_launch(c)
#include "FILE"
namespace scg {
void count_launches(int) {}
long long seq_sms() { return 152; }
}  // namespace scg

static int wrong = 0;
static void expect(bool ok, const char* what) { if (!ok) printf("%s: cluster %u grid %u asked %d last %d\n", what, cluster, grid, asked, (int)last), ++wrong; }
int main() {
    auto run = [](int ctas) {
        launched = 0;
        const cudaError_t e = CALL;
        return e == cudaSuccess && launched == 1 && last == cudaSuccess;
    };
    expect(run(16) && cluster == 16 && asked == 1, "there is room");
    expect(run(16) && cluster == 16 && asked == 1, "asked once");
    expect(run(8) && cluster == 8 && asked == 1, "8 need not be asked for");
    device = 1;
    room[1] = 0;
    expect(run(16) && cluster == 8 && grid % 8 == 0 && asked == 2, "no room on another device");
    expect(run(16) && cluster == 8 && asked == 2, "asked once there, too");
    device = 0;
    expect(run(16) && cluster == 16, "the first one still has room");
    device = 2;
    broken = true;
    expect(run(16) && cluster == 8, "the question fails");
    return wrong != 0;
}
"""
SORT = "scg::launch_expert_sort(nullptr, 0, ctas * 1024ll, 100, nullptr, nullptr, nullptr, nullptr)"
GATED = ("scg::go<float, 1, false, true, 8, false>(scg::GatedParams{}, scg::GatedMaps{}, %s, 3, ctas, nullptr)")


@pytest.mark.parametrize("source,call", [("sc_experts.cu", SORT), ("sc_gated.cuh", GATED % "false"), ("sc_gated.cuh", GATED % "true")])
def test_sixteen_only_where_they_fit(source, call, tmp_path):
    from stream_compaction_gb300 import build
    src, exe = tmp_path / "clusters.cu", tmp_path / "clusters"
    src.write_text(FAKES.replace("FILE", source).replace("CALL", call))
    subprocess.run([build.nvcc()] + build.ARCH + ["-std=c++17", "-O0", "-Xptxas", "-O0", "-I" + build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    made = subprocess.run([str(exe)], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout
