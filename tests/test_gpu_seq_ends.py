"""Rows that end inside a tile of the scan's kernels: what lies past the end takes no part,
whatever the rates; and steps of size 0 leave a state as it is, bit by bit."""
import pytest
import torch

import seq_reference as ref
import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("states", [8, 16, 24, 64])
@pytest.mark.parametrize("length", [1, 3, 16, 17, 37, 395])
def test_rates_of_minus_infinity(length, states):
    """A = -infinity: such a state forgets everything at every token, exp(d A) = 0.  (By its
    definition the gradient by dt multiplies it by 0 and is NaN: not compared.)"""
    gen = torch.Generator().manual_seed(length * states)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    c = {"x": normal(2, length, 20), "dt": normal(2, length, 20), "A": -0.1 - normal(20, states).abs(),
         "B": normal(2, length, 1, states), "C": normal(2, length, 1, states), "D": normal(20), "z": normal(2, length, 20),
         "state": normal(2, 20, states)}
    c["A"][:, ::2] = -float("inf")
    dy, dfinal = normal(2, length, 20), normal(2, 20, states)
    r = ref.scan(**c, dy=dy, dfinal=dfinal)
    finite = {**c, "A": c["A"].clamp(min=-1e30)}  # the same decays, and sums of absolute values without infinity times 0
    m = ref.scan(**finite, dy=dy, dfinal=dfinal, sizes=True)
    d = {k: v.cuda() for k, v in c.items()}
    final, saved = torch.empty_like(d["state"]), sc.selective_scan_saved(d["x"], d["A"])
    y = sc.selective_scan(**d, final_state=final, saved=saved)
    ref.check("y", y, r["y"], m["y"], torch.float32, length, states + 1)
    ref.check("final", final, r["final"], m["final"], torch.float32, length, 0)
    g = sc.selective_scan_grad(dy.cuda(), **d, saved=saved, dfinal_state=dfinal.cuda())
    for k, of in (("x", "dx"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"), ("state", "dstate")):
        ref.check(k, g[k], r[of], m[of], torch.float32, length, 20)


@pytest.mark.parametrize("length", [1, 7, 16, 100, 3000])
def test_steps_of_size_zero_keep_the_state(length):
    gen = torch.Generator(device="cuda").manual_seed(length)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    zero = torch.zeros(2, length, 40, device="cuda")
    A, state, bc = -8 * torch.rand(40, 16, generator=gen, device="cuda"), normal(2, 40, 16), normal(2, length, 1, 16)
    final = torch.empty_like(state)
    sc.selective_scan(normal(2, length, 40), zero, A, bc, bc, softplus=False, state=state, final_state=final)
    assert torch.equal(final, state)
    saved = sc.selective_scan_saved(zero, A)
    sc.selective_scan(zero, zero, A, bc, bc, softplus=False, state=state, saved=saved)
    back = sc.selective_scan_grad(zero, zero, zero, A, bc, bc, softplus=False, state=state, saved=saved, dfinal_state=state)
    assert torch.equal(back["state"], state)
    pool = state.clone()
    sc.selective_scan_step(normal(2, 40), zero[:, 0], A, bc[:, 0], bc[:, 0], pool, softplus=False)
    assert torch.equal(pool, state)
