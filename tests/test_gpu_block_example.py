"""The gated expert model of examples/: it trains, its gradients are those of differences,
and its single-token form continues what its prompt form began."""
import os
import sys

import pytest
import torch

from gpu_helpers import ensure_lib

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples import gated_expert_model as example  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    torch.backends.cuda.matmul.allow_tf32 = False


def test_it_trains():
    losses = example.train(example.Model(), 3, rows=4, length=96)
    assert len(losses) == 3 and all(0 < v < 100 for v in losses)


def test_gradients_reach_every_parameter():
    model = example.Model()
    ids, heads = example.batch(torch.Generator(device="cuda").manual_seed(3), 4, 96, 64)
    weight = torch.randn(4, 96, 64, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    (model.logits(ids, heads) * weight).sum().backward()
    assert all(v.grad is not None and v.grad.isfinite().all() for v in model.p.values())
    # along the gradient of each of some parameters: a central difference.  The 24576 logits of up to 10 are each
    # off by some 1e-6 of that, their sum by 1.6e-3; over the 2e-3 between the points 0.8, of slopes of 100 and more.
    # 5 % leave room for a token whose router is at a tie and takes another expert.
    for name in ("tokens", "norm", "norm1.0", "to_xg.1", "gate_bias.0", "mix.1", "norm2.1", "up.0", "down.1"):
        v = model.p[name]
        direction = v.grad / v.grad.norm()

        def at(step):
            with torch.no_grad():
                keep = v.clone()
                v.add_(direction, alpha=step)
                out = (model.logits(ids, heads).double() * weight).sum().item()
                v.copy_(keep)
            return out

        slope = (at(1e-3) - at(-1e-3)) / 2e-3
        assert abs(slope - v.grad.norm().item()) <= 0.05 * v.grad.norm().item(), name


def test_tokens_continue_a_prompt():
    """Prompt and single tokens give the logits of the whole row: the same operators on other
    splits of the length, and torch's products of other shapes.  A token's router could take
    another expert only where two shares differ by less than the error."""
    model = example.Model()
    ids, _ = example.batch(torch.Generator(device="cuda").manual_seed(5), 3, 40, 64)
    with torch.no_grad():
        whole = model.logits(ids)
    pool = model.pool(6)
    slots = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    got = [model.prompt(ids[:, :17].contiguous(), pool)]
    for t in range(17, 40):
        got.append(model.token(ids[:, t].contiguous(), pool, slots)[:, None])
    assert torch.allclose(torch.cat(got, 1), whole, rtol=1e-3, atol=1e-3)
