"""Trains a small recurrent sequence model with the library's operators and
lets it generate token by token.

The model: an embedding, gated linear recurrent layers (a projection to gate
logits and inputs, the recurrence, a gated output projection) and a linear
head.  The task: sequences over a small alphabet in which every symbol is
followed by a fixed successor, except that the marker 0 is followed by the
symbol that came before the previous marker, which the state has to remember.

- forward and backward through time: ``linear_recurrence`` (sigmoid form)
- the matrices' updates: momentum, then ``orthogonalize``, all matrices of one
  shape in one batch
- generation: ``linear_recurrence_step`` on a table of states

    python examples/recurrent_layer.py [--steps N] [--width D] [--seed S]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import triangular_solve_gb300 as tg  # noqa: E402

VOCAB = 16


def batch(rows: int, length: int, gen: torch.Generator) -> torch.Tensor:
    """Sequences of the task, (rows, length) of int64 on the CPU."""
    out = torch.empty(rows, length, dtype=torch.int64)
    successor = torch.arange(VOCAB)
    successor[1:] = torch.roll(torch.arange(1, VOCAB), 1)
    current = torch.randint(1, VOCAB, (rows,), generator=gen)
    before = torch.randint(1, VOCAB, (rows,), generator=gen)  # the symbol before the last marker
    for t in range(length):
        out[:, t] = current
        marker = (torch.rand(rows, generator=gen) < 0.2) & (current != 0)
        following = torch.where(current == 0, before, successor[current])
        before = torch.where(marker, current, before)
        current = torch.where(marker, torch.zeros_like(current), following)
    return out


class Layer(torch.nn.Module):
    """x + out(silu(o) * h), h the recurrence of (gate, input) = in(norm(x))."""

    def __init__(self, width: int):
        super().__init__()
        self.norm = torch.nn.LayerNorm(width)
        self.inner = torch.nn.Linear(width, 3 * width)
        self.out = torch.nn.Linear(width, width, bias=False)
        # channels that forget after 2 to 64 tokens, to begin with
        with torch.no_grad():
            self.inner.bias[:width] = torch.linspace(0.0, 4.0, width)

    def forward(self, x):
        gate, inputs, o = self.inner(self.norm(x)).chunk(3, dim=-1)  # strided views of one projection
        h, last = tg.linear_recurrence(gate, inputs, form="sigmoid")
        return x + self.out(torch.nn.functional.silu(o) * h), last

    def step(self, x, state, slots):
        gate, inputs, o = self.inner(self.norm(x)).chunk(3, dim=-1)
        h = tg.linear_recurrence_step(gate, inputs, state, form="sigmoid", slots=slots)
        return x + self.out(torch.nn.functional.silu(o) * h)


class Model(torch.nn.Module):
    def __init__(self, width: int, layers: int = 2):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, width)
        self.layers = torch.nn.ModuleList(Layer(width) for _ in range(layers))
        self.head = torch.nn.Linear(width, VOCAB)

    def forward(self, tokens):
        """Logits (rows, length, VOCAB) and the layers' last states."""
        x, states = self.embed(tokens), []
        for layer in self.layers:
            x, last = layer(x)
            states.append(last)
        return self.head(x), states

    def step(self, tokens, states, slots):
        x = self.embed(tokens)
        for layer, state in zip(self.layers, states):
            x = layer.step(x, state, slots)
        return self.head(x)


class OrthogonalisedMomentum:
    """Momentum whose direction is orthogonalised before it is applied, for
    matrices; the matrices of one shape go through one call."""

    def __init__(self, matrices, rate: float, momentum: float = 0.95):
        self.rate, self.momentum = rate, momentum
        self.groups = {}
        for p in matrices:
            self.groups.setdefault(tuple(p.shape), []).append(p)
        self.buffers = {s: torch.zeros(len(ps), *s, device=ps[0].device) for s, ps in self.groups.items()}

    @torch.no_grad()
    def step(self):
        for shape, ps in self.groups.items():
            grads, buf = torch.stack([p.grad for p in ps]), self.buffers[shape]
            buf.mul_(self.momentum).add_(grads)
            update = tg.orthogonalize(grads.add_(buf, alpha=self.momentum))
            scale = self.rate * max(1.0, shape[0] / shape[1]) ** 0.5
            for p, u in zip(ps, update.unbind()):
                p.sub_(u, alpha=scale)


def train(steps: int = 200, width: int = 128, rows: int = 32, length: int = 96, seed: int = 0, log=print):
    """Returns the trained model and the losses."""
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model(width).cuda()
    matrices = [p for layer in model.layers for p in (layer.inner.weight, layer.out.weight)]
    ids = {id(p) for p in matrices}
    rest = torch.optim.Adam([p for p in model.parameters() if id(p) not in ids], lr=3e-3)
    muon = OrthogonalisedMomentum(matrices, rate=0.02)
    losses = []
    for i in range(steps):
        tokens = batch(rows, length + 1, gen).cuda()
        logits, _ = model(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        model.zero_grad(set_to_none=True)
        loss.backward()
        rest.step()
        muon.step()
        losses.append(loss.item())
        if log and (i % 50 == 0 or i + 1 == steps):
            log(f"step {i:4d}  loss {losses[-1]:.4f}")
    return model, losses


@torch.no_grad()
def generate(model: Model, prompts: torch.Tensor, count: int) -> torch.Tensor:
    """Continues each prompt by `count` tokens, greedily: the prompt through the
    scan, then token by token out of a table of states."""
    rows = prompts.shape[0]
    logits, states = model(prompts)
    slots = torch.randperm(rows, device=prompts.device).to(torch.int32)  # any place in the table
    table = [torch.empty_like(s) for s in states]
    for t, s in zip(table, states):
        t[slots.long()] = s
    out = [logits[:, -1].argmax(-1)]
    for _ in range(count - 1):
        out.append(model.step(out[-1], table, slots).argmax(-1))
    return torch.stack(out, dim=1)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--width", type=int, default=128)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args()
    model, losses = train(a.steps, a.width, seed=a.seed)
    prompts = batch(4, 40, torch.Generator().manual_seed(a.seed + 1)).cuda()
    tokens = generate(model, prompts, 24)
    again = model(torch.cat([prompts, tokens[:, :-1]], 1))[0][:, prompts.shape[1] - 1:].argmax(-1)
    print("prompt ends ", prompts[0, -12:].tolist())
    print("continues   ", tokens[0].tolist())
    print(f"token by token and through the scan alike: {(again == tokens).float().mean().item():.0%}")


if __name__ == "__main__":
    main()
