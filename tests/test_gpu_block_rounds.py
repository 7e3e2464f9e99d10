"""The gated recurrence where the last of several rounds has tiles for a few warps only:
whole tiles come and go by the copy engine, some rounds under way at once."""
import pytest
import torch

import block_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


# 4 warps of 4 x 4096 or 8 x 4096 channels, 5 and 16 rounds; 16 CTAs of 8 warps in a cluster, 5 rounds;
# the last round: one tile, one token of one, all but one of the tiles
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,length,channels", [(8, 16 * 17, 4096), (8, 16 * 16 + 1, 4096), (4, 16 * 63 - 5, 8192),
                                                   (1, 16 * (4 * 128 + 1), 64)])
def test_a_last_round_with_few_tiles(batch, length, channels, dtype):
    gen = torch.Generator(device="cuda").manual_seed(length)
    x, g, dy = (torch.randn(batch, length, channels, generator=gen, device="cuda", dtype=torch.float32).to(dtype) for _ in range(3))
    dfinal = torch.randn(batch, channels, generator=gen, device="cuda")
    # copies beside the calls, so that results wait for the memory
    side, noise = torch.cuda.Stream(), torch.empty(2, 128 << 20, dtype=torch.uint8, device="cuda")

    def run():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                noise[0].copy_(noise[1])
        saved = sc.gated_scan_saved(x)
        y = sc.gated_scan(x, g, saved=saved)
        grads = sc.gated_scan_grad(dy, x, g, saved=saved, dfinal_state=dfinal)
        return y, grads["x"], grads["gate"]

    first = run()
    for _ in range(15):
        assert all(torch.equal(a, b) for a, b in zip(run(), first))
    part = slice(channels // 2, channels // 2 + 32)
    cut = [t[:2, :, part].contiguous().cpu() for t in (x, g, dy)]
    r = ref.gated(cut[0], cut[1], dy=cut[2], dfinal=dfinal[:2, part].cpu())
    for name, t in zip(("y", "dx", "dgate"), first):
        ref.check(name, t[:2, :, part].cpu(), r[name])
