"""The orthogonalised update of low-rank matrices, also within few rows and
columns: the map raises a small singular direction up to 485 times in five
steps, so no rounding may put noise into one."""
import pytest
import torch

from test_gpu_muon import ORTHO, newton_schulz, rel

pytestmark = pytest.mark.gpu

# O against the exact map where all roundings add up: in each of five steps A, B
# and X are rounded to fp16, by at most half a step 2^-11 of themselves, and a
# later step raises what an earlier one left by at most 2 (the map's slope where
# singular values settle), as long as none of it goes into the small directions
COHERENT = 15 * 2.0 ** -11 * 2

# Up to this short side the products run on both fp16 parts of X, A and B: 22
# bits, five steps of three roundings, and the most that the map can raise them by
PAIR_SIDE = 32
PAIRS = 15 * 2.0 ** -22 * 485


def low_rank(m, n, rank, rows, cols, seed, kind="gaussian"):
    g = torch.Generator().manual_seed(seed)
    u, v = torch.randn(rows, rank, generator=g), torch.randn(rank, cols, generator=g)
    if kind == "signs":
        u, v = u.sign(), v.sign()
    if kind == "near":
        u, v = 1 + 0.3 * u.abs().clamp(max=1), 1 + 0.3 * v.abs().clamp(max=1)
    if kind == "decay":
        u, v = u * 0.6 ** torch.arange(rows).unsqueeze(1), v * 0.6 ** torch.arange(cols)
    G = torch.zeros(m, n)
    G[:rows, :cols] = u @ v
    return G


@pytest.mark.parametrize("kind", ["gaussian", "signs", "near", "decay"])
@pytest.mark.parametrize("rank,rows,cols", [(1, 2, 2), (1, 3, 3), (1, 5, 8), (1, 8, 64), (1, 32, 64), (1, 64, 5), (2, 8, 8),
                                            (4, 16, 16), (1, 64, 64), (2, 6, 64)])
@pytest.mark.parametrize("m,n", [(64, 64), (64, 128), (200, 90), (128, 600), (300, 500), (700, 640), (2000, 1100)])
def test_low_rank_in_few_rows_and_columns(m, n, rank, rows, cols, kind):
    from linear_cross_entropy_token_gb300 import orthogonalize
    for seed in range(3):
        G = low_rank(m, n, rank, rows, cols, seed, kind)
        for g in (G, G.t().contiguous()):
            assert rel(orthogonalize(g.cuda(), dtype=torch.float32), newton_schulz(g)) <= COHERENT


@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
@pytest.mark.parametrize("rank,rows,cols", [(1, 3, 3), (1, 5, 8), (2, 8, 300), (1, 40, 40)])
def test_on_each_tile_shape(cta, rank, rows, cols):
    from linear_cross_entropy_token_gb300 import FLCE, orthogonalize
    h = FLCE("bf16", 0, cta=cta)
    try:
        for m, n in ((64, 700), (700, 340), (300, 300)):
            G = low_rank(m, n, rank, rows, cols, 5)
            assert rel(orthogonalize(G.cuda(), dtype=torch.float32, handle=h), newton_schulz(G)) <= COHERENT
    finally:
        h.close()


@pytest.mark.parametrize("m,n", [(1, 1), (2, 3), (4, 4), (8, 8), (16, 20), (31, 33), (32, 40), (40, 33), (8, 5000)])
def test_small_matrices(m, n):
    from linear_cross_entropy_token_gb300 import orthogonalize
    for seed in range(5):
        for rank in sorted({1, min(2, m, n), min(m, n)}):
            G = low_rank(m, n, rank, m, n, seed)
            limit = PAIRS if min(m, n) <= PAIR_SIDE else COHERENT
            for g in (G, G.t().contiguous()):
                assert rel(orthogonalize(g.cuda(), dtype=torch.float32), newton_schulz(g)) <= limit


@pytest.mark.parametrize("cta", ["auto", "single", "pair", "wide"])
@pytest.mark.parametrize("m,n,count", [(2, 9, 3), (8, 8, 1), (17, 400, 3), (32, 32, 2), (32, 1500, 1), (31, 9000, 2), (12, 4096, 40)])
def test_a_side_up_to_32_is_more_exact(m, n, count, cta):
    """On each kernel, with momentum and fp32 weights, repeated bit for bit."""
    from linear_cross_entropy_token_gb300 import FLCE, muon_update
    h = FLCE("bf16", 0, cta=cta)
    try:
        g = torch.Generator().manual_seed(m + n)
        G = [torch.randn(m, n, generator=g) * torch.exp(torch.randn(m, 1, generator=g)) for _ in range(count)]
        M = [torch.randn(m, n, generator=g) for _ in range(count)]
        for transposed in (False, True):
            flip = (lambda t: t.t().contiguous()) if transposed else (lambda t: t)
            first = None
            for _ in range(3):
                got = muon_update([flip(t).cuda() for t in G], [flip(t).cuda() for t in M], beta=0.9,
                                  update_dtype=torch.float32, handle=h)
                first = first or got
                assert all(torch.equal(a, b) for a, b in zip(got, first))
            for a, gi, mi in zip(first, G, M):
                gi, mi = gi.double(), mi.double()
                want = newton_schulz(0.9 * (0.9 * mi + 0.1 * gi) + 0.1 * gi)
                # (and the momentum's two roundings, raised as any difference is)
                assert rel(flip(a) if transposed else a, want) <= PAIRS + 2 * 2.0 ** -24 * 485
    finally:
        h.close()


@pytest.mark.parametrize("m,n", [(33, 47), (64, 64), (128, 128), (333, 1000), (512, 512), (1024, 700)])
def test_full_rank_gradients(m, n):
    """A few strong directions over a noise floor, rows of different magnitude: the ordinary bound."""
    from linear_cross_entropy_token_gb300 import orthogonalize
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        r = max(1, min(m, n) // 16)
        G = torch.randn(m, n, generator=g) + torch.randn(m, r, generator=g) @ torch.randn(r, n, generator=g) / r ** 0.5
        G = G * torch.exp(0.5 * torch.randn(m, 1, generator=g))
        assert rel(orthogonalize(G.cuda(), dtype=torch.float32), newton_schulz(G)) <= ORTHO
