"""A small language model of gated recurrences and experts on the library's block
operators: trained with their gradients, then continued token by token with their
single-token forms.

    python examples/gated_expert_model.py [--steps 200]

Each layer, on a residual stream: norm -> projection to (x, gate) -> gated_scan ->
projection, added to the stream -> norm -> a router's two experts of eight for every token
-> expert_gather -> an expert's two matrices -> expert_combine, added to the stream.  The
matrix products and the router's softmax are torch's; everything between them is the
library's.  The task: sequences of tokens that repeat with a period, several of them
packed into a row.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_gb300 as sc  # noqa: E402
from examples.state_space_model import batch  # noqa: E402


class Model:
    """The parameters, in float32, and the two ways through them."""

    def __init__(self, vocab=64, dim=64, channels=128, layers=2, experts=8, choices=2, hidden=128, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).requires_grad_()

        def ones(n):
            return torch.ones(n, device="cuda").requires_grad_()

        self.dim, self.channels, self.experts, self.choices = dim, channels, experts, choices
        self.p = {"tokens": normal(vocab, dim, scale=dim ** -0.5), "norm": ones(dim)}
        self.layers = []
        for n in range(layers):
            # gates that remember 2 to 200 tokens
            span = 2 * torch.exp(torch.rand(channels, generator=gen, device="cuda") * math.log(100))
            layer = {"norm1": ones(dim), "to_xg": normal(dim, 2 * channels, scale=dim ** -0.5),
                     "gate_bias": torch.log(span - 1).requires_grad_(), "mix": normal(channels, dim, scale=channels ** -0.5),
                     "norm2": ones(dim), "router": normal(dim, experts, scale=dim ** -0.5),
                     "up": normal(experts, dim, hidden, scale=dim ** -0.5),
                     "down": normal(experts, hidden, dim, scale=hidden ** -0.5)}
            self.layers.append(layer)
            self.p |= {"%s.%d" % (k, n): v for k, v in layer.items()}

    def _experts(self, p, y):
        """Every token (a row of y) through its experts."""
        share, chosen = torch.softmax(y @ p["router"], -1).topk(self.choices, -1)
        order = sc.expert_sort(chosen, self.experts)
        rows = sc.expert_gather(y, order)
        at = order.offsets.tolist()
        made = [torch.nn.functional.silu(rows[a:b] @ p["up"][e]) @ p["down"][e]
                for e, (a, b) in enumerate(zip(at, at[1:]))]
        return sc.expert_combine(torch.cat(made), order, share)

    def _layers(self, ids, mix):
        """Logits; mix(n, x, gate): the recurrence of layer n."""
        stream, add = sc.embed(ids, self.p["tokens"], math.sqrt(self.dim)), None
        for n, p in enumerate(self.layers):
            if add is None:
                y = sc.layer_norm(stream, p["norm1"], rms=True)
            else:
                y, stream = sc.layer_norm(add, p["norm1"], rms=True, residual=stream)
            x, gate = (y @ p["to_xg"]).chunk(2, -1)
            add = mix(n, x, gate + p["gate_bias"]) @ p["mix"]
            y, stream = sc.layer_norm(add, p["norm2"], rms=True, residual=stream)
            add = self._experts(p, y.flatten(0, -2)).view_as(y)
        return sc.layer_norm(add, self.p["norm"], rms=True, residual=stream)[0] @ self.p["tokens"].T

    def logits(self, ids, heads=None):
        """A batch of rows, packed sequences starting where heads is set."""
        return self._layers(ids, lambda n, x, gate: sc.gated_scan(x, gate, heads=heads))

    @torch.no_grad()
    def prompt(self, ids, pool):
        """Logits of a prompt without packing; its states into the first rows of the pool."""
        return self._layers(ids, lambda n, x, gate: sc.gated_scan(x, gate, final_state=pool[n][:len(ids)]))

    @torch.no_grad()
    def token(self, ids, pool, slots):
        """Logits of one more token for the sequences whose states lie in `slots`."""
        return self._layers(ids, lambda n, x, gate: sc.gated_scan_step(x, gate, pool[n], slots=slots))

    def pool(self, rows):
        return [torch.zeros(rows, self.channels, device="cuda") for _ in self.layers]


def train(model, steps, rows=16, length=192, rate=3e-3, seed=1, report=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    optimizer = torch.optim.Adam(list(model.p.values()), lr=rate)
    losses = []
    for step in range(steps):
        ids, heads = batch(gen, rows, length + 1, model.p["tokens"].shape[0])
        logits = model.logits(ids[:, :-1].contiguous(), heads[:, :-1].contiguous())
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), ids[:, 1:].flatten())
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if report and step % report == 0:
            print("step %4d  loss %.3f" % (step, loss.item()))
    return [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    model = Model()
    losses = train(model, args.steps, report=20)
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))
    # four prompts of two periods, continued greedily from their states
    ids, _ = batch(torch.Generator(device="cuda").manual_seed(2), 4, 36, 64)
    pool, slots = model.pool(4), torch.arange(4, dtype=torch.int32, device="cuda")
    token = model.prompt(ids[:, :24].contiguous(), pool)[:, -1].argmax(-1)
    made = [token]
    for _ in range(11):
        token = model.token(token, pool, slots).argmax(-1)
        made.append(token)
    print("continued right: %d of %d tokens" % (int((torch.stack(made, 1) == ids[:, 24:]).sum()), 4 * 12))


if __name__ == "__main__":
    main()
