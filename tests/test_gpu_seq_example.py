"""The sequence operators together, as examples/state_space_model.py uses them."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    ensure_lib()
    spec = importlib.util.spec_from_file_location("state_space_model", os.path.join(ROOT, "examples", "state_space_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss(example):
    model = example.Model()
    losses = example.train(model, 200)
    # log(64) = 4.16 is all that single tokens can give; within a document all but
    # the first period of 6 in 48 can be known: half of 4.16 needs the state
    assert losses[0] > 3.5 and sum(losses[-5:]) / 5 < 2.08, losses[::10]
    again = example.train(example.Model(), 5)
    assert again[0] == losses[0]  # the same inputs, the same bits


def test_tokens_continue_a_prompt(example):
    """Token by token from a prompt's states: the logits of the whole row."""
    model = example.Model(seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids, _ = example.batch(gen, 3, 40, 64)
    with torch.no_grad():
        whole = model.logits(ids, torch.zeros(3, 40, dtype=torch.bool, device="cuda"))
    pool = model.pool(5)
    first = model.prompt(ids[:, :17].contiguous(), pool)
    # float32 products in another order: 1e-5 of values of order 10
    assert torch.allclose(first, whole[:, :17], atol=2e-4, rtol=2e-4)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    for t in range(17, 40):
        assert torch.allclose(model.token(ids[:, t].contiguous(), pool, slots), whole[:, t], atol=2e-4, rtol=2e-4), t
    assert (pool["scan"][3:] == 0).all() and (pool["conv"][3:] == 0).all()
