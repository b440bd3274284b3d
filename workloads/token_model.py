"""A small token model trained with the library end to end: the embedding,
dropout and 4-bit linear layers of `layers` under ZeroAdam, N simulated
data-parallel ranks.

    python -m workloads.token_model            # a line per 20 steps

The task is synthetic: the next token is a fixed function of the current one.
A residual block of two 4-bit layers sits between the table and the output
layer; the padding token (0) takes part in neither the table's gradient nor
the loss.
"""
from __future__ import annotations

import math

import torch
import torch.nn.functional as F

import zero_sharded_optimizer_step_gb300 as z


class TokenModel:
    def __init__(self, vocab: int = 500, dim: int = 128, hidden: int = 512, p: float = 0.1,
                 dtype: torch.dtype = torch.bfloat16, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sigma):
            t = torch.randn(*shape, generator=g, device=device) * sigma
            return t.to(dtype).requires_grad_()

        self.vocab, self.p, self.seed, self.step_no = vocab, p, seed, 0
        self.table = normal(vocab, dim, sigma=0.5)
        self.up = normal(hidden, dim, sigma=1 / math.sqrt(dim))
        self.down = normal(dim, hidden, sigma=1 / math.sqrt(hidden))
        self.out = normal(vocab, dim, sigma=1 / math.sqrt(dim))
        self.layers = None

    def parameters(self):
        return [self.table, self.up, self.down, self.out]

    def refresh(self) -> None:
        """Quantises the weights: at first, and after every optimizer step."""
        if self.layers is None:
            self.layers = [z.Mx4Linear(w) for w in (self.up, self.down, self.out)]
        else:
            for layer in self.layers:
                layer.refresh()

    def loss(self, tokens: torch.Tensor, targets: torch.Tensor, rank: int = 0) -> torch.Tensor:
        up, down, out = self.layers
        offset = 2 * (1024 * self.step_no + rank)        # two dropout calls a rank and step
        h = z.embed(self.table, tokens, pad=0)
        h = z.dropout(h, self.p, self.seed, offset)
        y = down(F.gelu(up(h)))
        h = z.dropout(y, self.p, self.seed, offset + 1, residual=h)
        return F.cross_entropy(out(h).float(), targets, ignore_index=0)


def batch(model: TokenModel, n: int, generator: torch.Generator):
    tokens = torch.randint(0, model.vocab, (n,), generator=generator, device=model.table.device)
    targets = torch.where(tokens > 0, (tokens * 37 + 11) % (model.vocab - 1) + 1, 0)
    return tokens, targets


def check_products() -> None:
    """Raises if a 4-bit product gave up on the device (and stored nothing)."""
    n = z.zero_mx4_timeouts()
    if n:
        raise RuntimeError("%d waits of the 4-bit products ran out" % n)


def train(steps: int = 200, world: int = 2, n: int = 1024, lr: float = 3e-3, seed: int = 0,
          report=None):
    """The mean loss over the ranks, step by step."""
    model = TokenModel(seed=seed)
    opt = z.ZeroAdam(model.parameters(), world=world, lr=lr)
    model.refresh()
    data = [torch.Generator(device="cuda").manual_seed(seed * 1000 + k) for k in range(world)]
    losses = []
    for step in range(steps):
        model.step_no = step
        total = torch.zeros((), device="cuda")
        for k in range(world):
            for p in model.parameters():
                p.grad = None
            loss = model.loss(*batch(model, n, data[k]), rank=k)
            loss.backward()
            for g, p in zip(opt.rank_grads(k), model.parameters()):
                g.copy_(p.grad)
            total += loss.detach() / world
        opt.step()
        model.refresh()
        losses.append(total)
        if report and step % 20 == 19:
            check_products()
            report("step %4d  loss %.4f" % (step + 1, float(total)))
    check_products()
    return [float(v) for v in losses]


if __name__ == "__main__":
    train(report=print)
