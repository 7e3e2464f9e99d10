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


GATED = r"""
extern "C" int late_gated(int grad, long long batch, long long length, long long channels, const void* x, const void* gate,
                          const uint8_t* heads, void* y, float* final_state, float* saved, const void* dy, void* dx, void* dgate) {
    scg::GatedParams p{};
    p.sigmoid = 1, p.batch = batch, p.length = length, p.channels = channels;
    p.x = x, p.gate = gate, p.heads = heads, p.y = y, p.final_state = final_state, p.saved = saved;
    p.dy = dy, p.dx = dx, p.dgate = dgate;
    p.x_token = p.gate_token = p.y_token = p.dy_token = channels;
    p.x_batch = p.gate_batch = p.y_batch = p.dy_batch = length * channels;
    scg::GatedMaps maps{};
    if (!scg::maps_of<float, 1>(&maps, p, grad != 0)) return -1;
    const cudaError_t e = scg::go<float, 1, true, true, 4, true>(p, maps, grad != 0, batch * (channels / 32), 1, nullptr);
    return e != cudaSuccess ? (int)e : (int)cudaDeviceSynchronize();
}
"""


def test_gated(tmp_path):
    """Four warps a CTA, a tile of 16 tokens each, 32 channels; NaN goes on, and back, until a
    segment starts in a tile that came.  Forward three stages, gradient two, from the end."""
    lib = late_copies.build(str(tmp_path), "sc_gated.cuh", GATED, 32)
    batch, tiles, channels = 2, 43, 128
    length = 16 * tiles - 7
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, g, dy = (torch.randn(batch, length, channels, generator=gen, device="cuda") for _ in range(3))
    heads = torch.rand(batch, length, generator=gen, device="cuda") < 0.05
    saved, final = sc.gated_scan_saved(x), torch.empty(batch, channels, device="cuda")
    want = sc.gated_scan(x, g, heads=heads, saved=saved, final_state=final)
    grads = sc.gated_scan_grad(dy, x, g, heads=heads, saved=saved)
    y, dx, dg, end, kept = (torch.zeros_like(t) for t in (x, x, x, final, saved))
    torch.cuda.synchronize()
    n = [ctypes.c_longlong(v) for v in (batch, length, channels)]
    assert lib.late_gated(0, *n, _p(x), _p(g), _p(heads), _p(y), _p(end), _p(kept), None, None, None) == 0
    assert lib.late_gated(1, *n, _p(x), _p(g), _p(heads), None, None, _p(saved), _p(dy), _p(dx), _p(dg)) == 0
    cut = heads.cpu().tolist()
    for b in range(batch):
        for block in range(channels // 32):
            cta, cols = b * (channels // 32) + block, slice(32 * block, 32 * block + 32)
            lost = lambda i, ring: (cta == 1 and i % 4 == 2) or (cta == 3 and i // 4 // ring % 2 == 1)  # noqa: E731
            gone, state = [], False
            for t in range(length):
                bad = lost(t // 16, 3)
                state = bad or (state and not cut[b][t])
                gone.append(state)
            gone = torch.tensor(gone, device="cuda")
            assert gone.any() == (cta in (1, 3))
            assert torch.equal(y[b, ~gone, cols], want[b, ~gone, cols]) and y[b, gone, cols].isnan().all()
            if gone[-1]:
                assert end[b, cols].isnan().all()
            back, state = [], False
            for t in reversed(range(length)):
                bad = lost(tiles - 1 - t // 16, 2)
                back.append(bad or state)
                state = bad or (state and not cut[b][t])
            back = torch.tensor(back[::-1], device="cuda")
            for got, name in ((dx, "x"), (dg, "gate")):
                assert torch.equal(got[b, ~back, cols], grads[name][b, ~back, cols]) and got[b, back, cols].isnan().all(), name
