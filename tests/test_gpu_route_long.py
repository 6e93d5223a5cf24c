"""The routing forward in two launches (more rows than one cluster takes) with
many experts: every number of experts per lane, with and without documents,
masks, ties, strides. A batch of up to 512 rows with more than 128 experts runs
as one cluster, so these have more. Against float64 by test_gpu_route's
definition and tolerances: fewer than its 320 roundings lie between a row and a
sum here too (a lane adds at most 40 rows, a block 8 warps' sums, the closing
launch 20 units a lane and a tree of 5)."""
import math

import pytest
import torch

from test_gpu_route import DT, compare, make, run

pytestmark = pytest.mark.gpu

SIZES = [(520, 129, 5), (700, 200, 12), (1500, 256, 8), (20000, 256, 8), (6000, 255, 1), (600, 257, 7), (2500, 384, 8),
         (900, 512, 12), (700, 513, 4), (5000, 700, 6), (1200, 1024, 32)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,E,k", SIZES)
def test_sizes(N, E, k, dtype):
    z, _ = make(N, E, dtype, N + E)
    for renorm in (True, False):
        r, d, ref = run(z, k, renormalize=renorm)
        compare(r, d, ref, z, dtype, 1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("documents", [1, 2, 7, 300])
@pytest.mark.parametrize("N,E,k", [(1500, 130, 4), (3000, 256, 8), (2000, 400, 5), (1100, 1024, 8), (40, 300, 3)])
def test_documents_and_masks(N, E, k, documents, dtype):
    z, g = make(N, E, dtype, documents + E)
    z[:, -3:] = -math.inf                       # padded experts
    z[5] = -math.inf                            # a token with no expert at all
    z[6, 1:] = -math.inf                        # one expert only: k - 1 empty slots
    valid = torch.rand(N, generator=g) > 0.2
    cuts = torch.randint(0, N + 1, (documents - 1,), generator=g)
    if documents > 4:
        cuts[1] = cuts[0]                       # an empty document
        cuts[2] = 0                             # and one at the start
    offsets = torch.cat([torch.tensor([0, N]), cuts]).sort().values
    if documents > 1:
        valid[offsets[1]:offsets[2]] = False    # a document with no live token
    r, d, ref = run(z, k, valid, offsets)
    compare(r, d, ref, z, dtype, documents)
    assert not d.float().cpu()[~ref["live"]].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [130, 200, 256, 384, 512, 1024])
def test_selection_is_exact(E, dtype):
    """The largest side by side, last bits that differ, ties, signed zeros, -inf among them; one expert to 32."""
    from linear_cross_entropy_token_gb300 import route
    g = torch.Generator().manual_seed(E)
    N = 700
    up = torch.arange(E).float().repeat(N, 1) / 16
    together = torch.randn(N, E, generator=g)
    first = torch.randint(0, E - 9, (N, 1), generator=g) + torch.arange(9)
    together.scatter_add_(1, first, torch.full((N, 9), 8.0))
    close = 1.0 + torch.randint(0, 40, (N, E), generator=g).float() * 2.0 ** -23
    few = torch.randint(0, 3, (N, E), generator=g).float() - 1.0
    zeros = torch.randint(0, 2, (N, E), generator=g).float() * -0.0
    zeros[:, ::2] *= -1.0
    holes = torch.where(torch.rand(N, E, generator=g) < 0.97, torch.full((), -math.inf), together)
    mixed = torch.stack([(up, -up, together, close, few, holes)[i % 6][i] for i in range(N)])   # within one warp's rows
    for rows in (up, -up, together, close, -close, few, zeros, holes, mixed):
        z = rows.to(DT[dtype])
        order = torch.sort(z.double(), dim=1, descending=True, stable=True).indices
        for k in (1, 3, 8, 32):
            want = order[:, :k]
            want = torch.where(z.double().gather(1, want) > -math.inf, want, torch.full_like(want, -1))
            got = route(z.cuda(), k).experts.cpu().long()
            assert torch.equal(got, want), (k, int((got != want).any(1).nonzero()[0]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("E", [203, 300, 600])
def test_strided_and_unaligned_rows(E, dtype):
    N = 800
    z, _ = make(N, E, dtype, E)

    def odd(z):
        big = torch.full((N, E + 13), math.nan, dtype=z.dtype, device="cuda")
        big[:, 5:5 + E] = z.cuda()
        return big[:, 5:5 + E]

    def wide(z):
        big = torch.full((N, 640), math.nan, dtype=z.dtype, device="cuda")
        big[:, :E] = z.cuda()
        return big[:, :E]

    for view in (odd, wide):
        r, d, ref = run(z, 5, view=view)
        compare(r, d, ref, z, dtype, 1)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("E", [200, 400, 1000])
def test_nan_and_infinite_logits_stay_in_their_row(E, value):
    import linear_cross_entropy_token_gb300 as flce
    N = 900
    z, _ = make(N, E, "fp32", 1)
    z[617, E - 2] = value
    keep = torch.arange(N) != 617
    r = flce.route(z.cuda(), 3)
    assert math.isnan(float(r.balance)) and bool(r.weights[617].isnan().all())
    assert int(r.experts.min()) >= -1 and int(r.experts.max()) < E
    assert bool(torch.isfinite(r.weights.cpu()[keep]).all())
    r, d, ref = run(torch.where(keep[:, None], z, torch.zeros(())), 3, valid=keep)
    masked = flce.route(z.cuda(), 3, valid=keep.cuda())
    assert torch.equal(masked.experts, r.experts) and torch.equal(masked.state[:4], r.state[:4])
    compare(r, d, ref, z[keep], "fp32", 1)


@pytest.mark.parametrize("E", [256, 300, 1024])
def test_offsets_out_of_order_stay_in_bounds(E):
    import linear_cross_entropy_token_gb300 as flce
    z, _ = make(1400, E, "bf16", 5)
    for off in ([100, 300], [0, 500, 200, 1400], [-50, 10, 9000], [1700, 1800, 1900]):
        r = flce.route(z.cuda(), 2, offsets=torch.tensor(off, device="cuda"))
        d = flce.route_backward(r, z.cuda(), d_balance=torch.ones((), device="cuda"))
        assert int(r.experts.min()) >= -1 and int(r.experts.max()) < E and d.shape == z.shape


@pytest.mark.parametrize("E", [256, 384, 1024])
def test_repeats_bit_for_bit(E):
    import linear_cross_entropy_token_gb300 as flce
    z, g = make(9000, E, "fp32", 2)
    zc, dw, one = z.cuda(), torch.randn(9000, 8, generator=g).cuda(), torch.ones((), device="cuda")
    seen = None
    for _ in range(4):
        r = flce.route(zc, 8)
        now = (flce.route_backward(r, zc, d_weights=dw, d_balance=one, d_z=one), r.weights, r.experts, r.counts,
               r.state[:4].clone())
        seen = seen or now
        assert all(torch.equal(a, b) for a, b in zip(now, seen))
