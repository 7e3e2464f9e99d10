"""A launch that fails is reported by its own call, and by no later one: the host side of
the block operators, compiled with launchers and CUDA calls that the test makes up."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKES = r"""
#include <cstdio>
#include "sc_block_api.cu"

static cudaError_t last = cudaSuccess;  // as the runtime keeps it
static bool fail = false;
extern "C" cudaError_t cudaGetLastError() { cudaError_t e = last; last = cudaSuccess; return e; }
static cudaError_t made() {  // what a call that launches something returns
    if (fail) last = cudaErrorInvalidClusterSize;
    return fail ? last : cudaGetLastError();
}
extern "C" cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return fail ? last = cudaErrorInvalidValue : cudaSuccess; }
extern "C" cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) {
    return fail ? last = cudaErrorInvalidValue : cudaSuccess;
}
namespace scg {
sc_status seq_scratch(cudaStream_t, size_t, unsigned char** p) { static unsigned char b; *p = &b; return SC_OK; }
size_t seq_scratch_total(size_t n) { return n; }
size_t norm_grad_scratch(long long, long long) { return 256; }
cudaError_t launch_gated(int, const GatedParams&, cudaStream_t) { return made(); }
cudaError_t launch_gated_grad(int, const GatedParams&, cudaStream_t) { return made(); }
cudaError_t launch_gated_step(int, const GatedParams&, cudaStream_t) { return made(); }
cudaError_t launch_norm(int, NormParams, cudaStream_t) { return made(); }
cudaError_t launch_norm_grad(int, NormParams, cudaStream_t) { return made(); }
cudaError_t launch_expert_sort(const void*, int, long long, int, int32_t*, int32_t*, int64_t*, cudaStream_t) { return made(); }
cudaError_t launch_expert_gather(int, const ExpertParams&, cudaStream_t) { return made(); }
cudaError_t launch_expert_combine(int, const ExpertParams&, cudaStream_t) { return made(); }
cudaError_t launch_expert_combine_grad(int, const ExpertParams&, cudaStream_t) { return made(); }
}  // namespace scg

template <class T = void> static T* at(size_t n) { return reinterpret_cast<T*>(n << 16); }  // never followed

int main() {
    sc_gated_desc g{}, none{}, one{};
    g.batch = 2, g.length = 8, g.channels = 16, g.x = at(1), g.gate = at(2);
    g.x_batch = g.gate_batch = 128, g.x_token = g.gate_token = 16, g.dtype = SC_F32;
    none = one = g;
    none.length = 0;
    one.length = 1;
    sc_norm_desc n{};
    n.batch = 2, n.length = 8, n.channels = 16, n.x = at(1), n.x_batch = 128, n.x_token = 16, n.dtype = n.wtype = SC_F32;
    n.weight = at(9);
    sc_norm_desc nothing = n;
    nothing.length = 0;
    sc_expert_desc e{};
    e.dtype = e.wtype = SC_F32, e.tokens = 4, e.choices = 2, e.dim = 8, e.experts = 3;
    e.place = at<int32_t>(10), e.offsets = at<int64_t>(11), e.weights = at(12);
    auto calls = [&](int i) -> sc_status {
        switch (i) {
        case 0: return sc_gated_scan(&g, at(3), 128, 16, nullptr, nullptr, 0);
        case 1: return sc_gated_scan(&none, nullptr, 0, 0, at<float>(4), nullptr, 0);  // zeros
        case 2: return sc_gated_scan_grad(&g, at(3), 128, 16, at<float>(4), nullptr, at(5), at(6), nullptr, 0);
        case 3: return sc_gated_scan_step(&one, at<float>(4), 2, nullptr, at(3), 16, 0);
        case 4: return sc_layer_norm(&n, at(3), 128, 16, nullptr, 0, 0, nullptr, 0);
        case 5: return sc_layer_norm_grad(&n, at(3), 128, 16, nullptr, 0, 0, at<float>(4), at(5), at<float>(6), nullptr, 0);
        case 6: return sc_layer_norm_grad(&nothing, at(3), 128, 16, nullptr, 0, 0, at<float>(4), at(5), at<float>(6), nullptr, 0);
        case 7: return sc_expert_sort(at(1), 0, 8, 3, at<int32_t>(2), at<int32_t>(3), at<int64_t>(4), 0);
        case 8: return sc_expert_gather(&e, at(1), 8, at(2), 8, 0);
        case 9: return sc_expert_gather_grad(&e, at(2), 8, at(1), 8, 0);
        case 10: return sc_expert_combine(&e, at(2), 8, at(1), 8, 0);
        default: return sc_expert_combine_grad(&e, at(1), 8, at(2), 8, at(3), 8, at(4), 0);
        }
    };
    int wrong = 0;
    for (int i = 0; i < 12; ++i)
        for (int next = 0; next < 12; ++next) {
            fail = true;
            const sc_status bad = calls(i);
            fail = false;
            const sc_status good = calls(next);
            if (bad != SC_ERR_CUDA || good != SC_OK || last != cudaSuccess) printf("%d then %d: %d %d\n", i, next, bad, good), ++wrong;
            last = cudaSuccess;
        }
    return wrong != 0;
}
"""


def test_an_error_does_not_stay_behind(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    from stream_compaction_gb300 import build
    toolkit = os.path.dirname(os.path.dirname(build.nvcc()))
    src, exe = tmp_path / "errors.cpp", tmp_path / "errors"
    src.write_text(FAKES)
    subprocess.run([gxx, "-std=c++17", "-I" + os.path.join(build.CSRC), "-I" + os.path.join(toolkit, "include"), str(src),
                    "-o", str(exe)], check=True)
    made = subprocess.run([str(exe)], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout
