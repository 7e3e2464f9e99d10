"""A wait that runs out makes NaN of what it was for, and of nothing else."""
import ctypes

import pytest
import torch

import late_copies
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _p(t):
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


NORM = r"""
extern "C" int late_norm(int grad, long long rows, long long channels, const void* x, const void* residual, void* y, void* sum,
                         float* saved, const void* dy, const void* dsum, void* dx, float* partials) {
    scg::NormParams p{};
    p.eps = 1e-5f;
    p.rows = p.length = (uint32_t)rows;
    p.channels = channels;
    p.vec = p.dense = p.params_f32 = 1;
    p.x = x, p.residual = residual, p.y = y, p.sum = sum, p.saved = saved;
    p.dy = dy, p.dsum = dsum, p.dx = dx, p.partials = partials;
    p.dweight = p.dbias = partials;
    p.x_token = p.residual_token = p.y_token = p.sum_token = p.dy_token = p.dsum_token = channels;
    const cudaError_t e = scg::go<float, scg::kRing, 32, 2>(p, grad != 0, nullptr);
    return e != cudaSuccess ? (int)e : (int)cudaDeviceSynchronize();
}
"""


def test_norm(tmp_path):
    """256 channels: a warp a row, 8 rows a turn of a CTA, 8 stages of a ring at most."""
    lib = late_copies.build(str(tmp_path), "sc_norm.cuh", NORM, 32)
    channels, turns = 256, 20
    rows = 3 * SMS * 8 * turns - 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy, ds = (torch.randn(rows, channels, generator=gen, device="cuda") for _ in range(4))
    saved = sc.layer_norm_saved(x)
    y, s = sc.layer_norm(x, residual=r, saved=saved)
    want = sc.layer_norm_grad(dy, s, saved=saved, dsum=ds)["x"]
    torch.cuda.synchronize()
    row = torch.arange(rows, device="cuda")
    for resident, grad in ((3, False), (2, True)):
        cta, turn, team = row // 8 % (resident * SMS), row // 8 // (resident * SMS), row % 8
        gone = (cta == 1) & (team == 2)
        here = ~gone & (cta != 3)
        got = torch.zeros(rows, channels, device="cuda")
        if not grad:
            total, stat = torch.zeros_like(got), torch.zeros(rows, 2, device="cuda")
            assert lib.late_norm(0, ctypes.c_longlong(rows), ctypes.c_longlong(channels), _p(x), _p(r), _p(got), _p(total), _p(stat), None,
                                 None, None, None) == 0
            checks = ((got, y), (total, s), (stat, saved))
        else:
            partials = torch.zeros(resident * SMS, 2, channels, device="cuda")
            assert lib.late_norm(1, ctypes.c_longlong(rows), ctypes.c_longlong(channels), _p(s), None, None, None, _p(saved), _p(dy), _p(ds),
                                 _p(got), _p(partials)) == 0
            checks = ((got, want),)
            nan = partials.isnan()
            assert nan[[1, 3]].all() and not nan[[0, 2] + list(range(4, resident * SMS))].any()
        for a, b in checks:
            assert a[gone].isnan().all() and torch.equal(a[here], b[here])
            # CTA 3 goes well until its ring's second way round, and not at all from there on
            for t in range(8):
                mine = a[(cta == 3) & (team == t)].isnan()
                assert (mine.all(1) == mine.any(1)).all()
                bad = mine.any(1).nonzero().flatten().tolist()
                assert 1 < bad[0] <= 8 and bad == list(range(bad[0], len(mine)))
