"""Inputs and 64-bit references of the head's scoring and distillation tests."""
import math

import torch

BF16 = 2.0 ** -8     # half a step of bf16, relative
FP16 = 2.0 ** -11
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make_head(N, H, V, dtype, seed=0, strength=8.0, scale=1.0):
    """x and W with logits of spread 1.3 scale, each row leaning towards one token."""
    g = torch.Generator().manual_seed(seed)
    std = 1.3 / math.sqrt(H)
    W = (torch.randn(V, H, generator=g) * std).to(DT[dtype])
    likely = torch.randint(0, V, (N,), generator=g)
    lean = torch.rand(N, 1, generator=g) * strength
    x = torch.randn(N, H, generator=g) + lean * W[likely].float() / (std * std * H)
    t = torch.where(torch.rand(N, generator=g) < 0.6, likely, torch.randint(0, V, (N,), generator=g))
    return (x * scale).to(DT[dtype]).cuda(), W.cuda(), t.cuda(), g


class Reference:
    """The operators of `live` rows in 64 bits."""

    def __init__(self, x, W, temperature=1.0):
        self.x, self.W, self.tau = x.double(), W.double(), temperature
        self.raw = self.x @ self.W.T
        self.z = self.raw / temperature
        self.lp = torch.log_softmax(self.z, 1)
        self.p = self.lp.exp()
        self.entropy = -(self.p * self.lp).sum(1)

    def top(self, k):
        order = torch.sort(self.raw, dim=1, descending=True, stable=True).indices[:, :k]
        return order, self.lp.gather(1, order)

    def d_scores(self, t, g, h):
        d = -self.p * (g[:, None] + h[:, None] * (self.lp + self.entropy[:, None]))
        return d.scatter_add(1, t[:, None], g[:, None]) / self.tau

    def sum_error(self):
        """What the product's 32-bit sums may be off by: at most a step of the running sum for every 16 products
        (and a few at the end), which stays within a row's largest logit and the sums' random walk."""
        H = self.x.shape[1]
        walk = 4.0 * self.x.norm(dim=1) * self.W.norm(dim=1).max() / math.sqrt(H)
        return (H / 16 + 8) * 2.0 ** -23 * (self.raw.abs().amax(1) + walk) / self.tau


def check_gradients(dx, dW, d, x, W, kept_y=None, dtype="bf16"):
    """dx = d W and dW = dt x against 64 bits. bf16: every entry of d is rounded once (half a step each), the
    result once more; logits kept as fp16 add half a step of their distance y (log2 units) to the exponent. fp32:
    the sums alone."""
    x, W = x.double(), W.double()
    if dtype == "fp32":
        for got, want in ((dx, d @ W), (dW, d.T @ x)):
            if got is not None:
                assert (got.double() - want).norm() <= 1e-5 * want.norm() + 1e-30
        return
    rel = torch.full_like(d, BF16 * 1.02)
    if kept_y is not None:
        rel += kept_y * FP16 * math.log(2.0) * 1.02
    off = d.abs() * rel
    for got, want, bound in ((dx, d @ W, off @ W.abs()), (dW, d.T @ x, off.T @ x.abs())):
        if got is None:
            continue
        last = BF16 if got.dtype == torch.bfloat16 else 0.0
        tol = bound * (1 + last) + want.abs() * last + 1e-5 * want.abs().max() + 1e-30
        worst = ((got.double() - want).abs() / tol).max().item()
        assert worst <= 1.0, f"{worst} of the bound"
        # roundings are independent: their norm is what one rounding of everything may take, once for d and once here
        limit = (2.0 if kept_y is None else 4.0) * BF16
        assert (got.double() - want).norm() <= limit * want.norm() + 1e-30


def kept_distance(raw, c):
    """How far each logit lies below its 64 columns' largest, in log2 units."""
    N, V = raw.shape
    pad = (-V) % 64
    z = torch.nn.functional.pad(raw, (0, pad), value=-math.inf).view(N, -1, 64)
    return ((z.amax(2, keepdim=True) - z).view(N, -1)[:, :V]) * c
