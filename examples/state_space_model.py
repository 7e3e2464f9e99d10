"""A small state space language model on the library's sequence operators: trained
with their gradients, then continued token by token with their single-token forms.

    python examples/state_space_model.py [--steps 200]

One layer: tokens -> embed -> projection to (x, z) -> causal_conv -> projections to
dt, B, C -> selective_scan -> projection -> logits against the same embedding.  The
matrix products are torch's; everything between them is the library's.  The task:
sequences of tokens that repeat with a period, several of them packed into a row.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_gb300 as sc  # noqa: E402


class Model:
    """The parameters, in float32, and the two ways through them."""

    def __init__(self, vocab=64, dim=64, channels=128, states=16, rank=8, width=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).requires_grad_()

        self.dim, self.channels, self.states, self.rank, self.width = dim, channels, states, rank, width
        step = torch.exp(torch.rand(channels, generator=gen, device="cuda") * math.log(100) + math.log(1e-3))
        self.p = {
            "tokens": normal(vocab, dim, scale=dim ** -0.5),
            "to_xz": normal(dim, 2 * channels, scale=dim ** -0.5),
            "conv": normal(channels, width, scale=width ** -0.5),
            "conv_bias": torch.zeros(channels, device="cuda").requires_grad_(),
            "to_dt_bc": normal(channels, rank + 2 * states, scale=channels ** -0.5),
            "to_dt": normal(rank, channels, scale=rank ** -0.5),
            "dt_bias": (step + torch.log(-torch.expm1(-step))).requires_grad_(),
            "log_A": torch.log(torch.arange(1, states + 1, device="cuda").float().repeat(channels, 1)).requires_grad_(),
            "D": torch.ones(channels, device="cuda").requires_grad_(),
            "out": normal(channels, dim, scale=channels ** -0.5),
        }

    def _inner(self, u):
        """dt, B and C from the convolution's outputs."""
        p = self.p
        low, B, C = (u @ p["to_dt_bc"]).split([self.rank, self.states, self.states], -1)
        return low @ p["to_dt"], B.unsqueeze(-2), C.unsqueeze(-2)

    def logits(self, ids, heads):
        """A batch of rows, packed sequences starting where heads is set."""
        p = self.p
        h = sc.embed(ids, p["tokens"], math.sqrt(self.dim))
        x, z = (h @ p["to_xz"]).chunk(2, -1)
        u = sc.causal_conv(x, p["conv"], p["conv_bias"], heads=heads)
        dt, B, C = self._inner(u)
        y = sc.selective_scan(u, dt, -torch.exp(p["log_A"]), B, C, p["D"], z, p["dt_bias"], heads=heads)
        return (h + y @ p["out"]) @ p["tokens"].T

    @torch.no_grad()
    def prompt(self, ids, pool):
        """Logits of a prompt without packing; its states into the first rows of the pool."""
        p, n = self.p, ids.shape[0]
        h = sc.embed(ids, p["tokens"], math.sqrt(self.dim))
        x, z = (h @ p["to_xz"]).chunk(2, -1)
        u = sc.causal_conv(x, p["conv"], p["conv_bias"], final_state=pool["conv"][:n])
        dt, B, C = self._inner(u)
        y = sc.selective_scan(u, dt, -torch.exp(p["log_A"]), B, C, p["D"], z, p["dt_bias"], final_state=pool["scan"][:n])
        return (h + y @ p["out"]) @ p["tokens"].T

    @torch.no_grad()
    def token(self, ids, pool, slots):
        """Logits of one more token for the sequences whose states lie in `slots`."""
        p = self.p
        h = sc.embed(ids, p["tokens"], math.sqrt(self.dim))
        x, z = (h @ p["to_xz"]).chunk(2, -1)
        u = sc.causal_conv_step(x, pool["conv"], p["conv"], p["conv_bias"], slots=slots)
        dt, B, C = self._inner(u)
        y = sc.selective_scan_step(u, dt, -torch.exp(p["log_A"]), B, C, pool["scan"], p["D"], z, p["dt_bias"], slots=slots)
        return (h + y @ p["out"]) @ p["tokens"].T

    def pool(self, rows):
        return {"conv": torch.zeros(rows, self.width - 1, self.channels, device="cuda"),
                "scan": torch.zeros(rows, self.channels, self.states, device="cuda")}


def batch(gen, rows, length, vocab, period=6, document=48):
    """Rows of packed documents, each repeating its own `period` random tokens."""
    words = torch.randint(0, vocab, (rows, -(-length // document), period), generator=gen, device="cuda")
    t = torch.arange(length, device="cuda")
    ids = words[:, t // document, t % document % period]
    return ids, (t % document == 0).expand(rows, length).contiguous()


def train(model, steps, rows=16, length=192, rate=3e-3, seed=1, report=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params = list(model.p.values())
    optimizer = torch.optim.Adam(params, lr=rate)
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
    pool = model.pool(4)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    token = model.prompt(ids[:, :24].contiguous(), pool)[:, -1].argmax(-1)
    made = [token]
    for _ in range(11):
        token = model.token(token, pool, slots).argmax(-1)
        made.append(token)
    print("continued right: %d of %d tokens" % (int((torch.stack(made, 1) == ids[:, 24:]).sum()), 4 * 12))


if __name__ == "__main__":
    main()
