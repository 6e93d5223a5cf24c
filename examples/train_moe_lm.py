"""A small language model with experts, trained by the library's parts together:
expert routing with its balance and z losses (autograd.route), the fused linear
cross-entropy of the LM head (autograd.linear_cross_entropy), and Muon for the
experts' matrices.

    python examples/train_moe_lm.py [--steps 30]

The tokens are synthetic: a fixed random permutation maps each token to the
next, and documents of uneven length end with an ignored target, so the loss
can fall far below log V. Prints the losses and how evenly the experts are used.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_cross_entropy_token_gb300 import Muon  # noqa: E402
from linear_cross_entropy_token_gb300.autograd import linear_cross_entropy, route  # noqa: E402


class Experts(torch.nn.Module):
    """E two-layer MLPs; each token goes through its k chosen ones."""

    def __init__(self, hidden, inner, experts, k, device):
        super().__init__()
        self.k = k
        # logits start small, so that the z loss starts near log(experts)^2
        self.router = torch.nn.Parameter(torch.randn(experts, hidden, device=device) * 0.1 * hidden ** -0.5)
        self.up = torch.nn.ParameterList(
            [torch.randn(inner, hidden, device=device) * hidden ** -0.5 for _ in range(experts)])
        self.down = torch.nn.ParameterList(
            [torch.randn(hidden, inner, device=device) * inner ** -0.5 for _ in range(experts)])

    def forward(self, x, valid, offsets):
        weights, experts, counts, balance, z = route(x.float() @ self.router.T, self.k, valid, offsets)
        y = torch.zeros_like(x)
        for e, (up, down) in enumerate(zip(self.up, self.down)):
            token, slot = (experts == e).nonzero(as_tuple=True)
            h = torch.nn.functional.silu(x[token] @ up.T.to(x.dtype)) @ down.T.to(x.dtype)
            y = y.index_add(0, token, h * weights[token, slot].unsqueeze(1).to(x.dtype))
        return x + y, counts, balance, z


class Model(torch.nn.Module):
    def __init__(self, vocab, hidden, inner, experts, k, device):
        super().__init__()
        self.embedding = torch.nn.Parameter(torch.randn(vocab, hidden, device=device))
        self.experts = Experts(hidden, inner, experts, k, device)
        self.head = torch.nn.Parameter(torch.randn(vocab, hidden, device=device) * hidden ** -0.5)

    def forward(self, tokens, targets, valid, offsets):
        x = self.embedding[tokens].bfloat16()
        x, counts, balance, z = self.experts(x, valid, offsets)
        loss = linear_cross_entropy(x, self.head.bfloat16(), targets)
        return loss, balance, z, counts


def batch(tokens_per_batch, vocab, follows, device, generator):
    """Documents of uneven length: tokens, targets (-100 at a document's end), which tokens count, offsets."""
    cuts = torch.randint(1, tokens_per_batch, (7,), generator=generator)
    offsets = torch.cat([torch.tensor([0, tokens_per_batch]), cuts]).sort().values.unique()
    tokens = torch.randint(0, vocab, (tokens_per_batch,), generator=generator)
    targets = follows[tokens]
    targets[offsets[1:] - 1] = -100
    return tokens.to(device), targets.to(device), (targets != -100).to(device), offsets.to(device)


def train(steps=30, vocab=1000, hidden=256, inner=512, experts=8, k=2, tokens_per_batch=4096, device="cuda",
          log=print):
    torch.manual_seed(0)
    generator = torch.Generator().manual_seed(0)
    follows = torch.randperm(vocab, generator=generator)
    model = Model(vocab, hidden, inner, experts, k, device)
    matrices = list(model.experts.up) + list(model.experts.down)
    muon = Muon(matrices, lr=5e-3)
    adam = torch.optim.AdamW([model.embedding, model.head, model.experts.router], lr=1e-2)
    history = []
    for step in range(steps):
        tokens, targets, valid, offsets = batch(tokens_per_batch, vocab, follows, device, generator)
        loss, balance, z, counts = model(tokens, targets, valid, offsets)
        (loss + 0.01 * balance + 0.001 * z).backward()
        muon.step()
        adam.step()
        muon.zero_grad()
        adam.zero_grad()
        used = counts.sum(0)
        history.append((loss.item(), balance.item(), used.sum().item()))
        if step % 5 == 0 or step == steps - 1:
            log(f"step {step:3d}  loss {loss.item():.4f}  balance {balance.item():.4f}  z {z.item():.3f}  "
                f"slots per expert {used.min().item()} to {used.max().item()}")
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=30)
    train(parser.parse_args().steps)
