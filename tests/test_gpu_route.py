"""Expert routing on the GPU against its definition in float64 (torch on the
host): weights, experts, counts, losses and the logits' gradient, over types,
expert counts, strides, documents and masks."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
U = 2.0 ** -24


def reference(z, k, valid=None, offsets=None, renormalize=True, d_weights=None, d_balance=0.0, d_z=0.0,
              experts=None):
    """The definition, in float64 on the host. `experts` fixes the selection (for differences)."""
    z = z.detach().double().cpu() if experts is None else z
    N, E = z.shape
    live = (z > -math.inf).any(1) | z.isnan().any(1)
    if valid is not None:
        live = live & valid.cpu().bool()
    off = [0, N] if offsets is None else offsets.tolist()
    doc = torch.full((N,), -1, dtype=torch.int64)
    for d, (a, b) in enumerate(zip(off[:-1], off[1:])):
        doc[a:b] = d
    live = live & (doc >= 0)
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    lse = torch.logsumexp(zz, 1)
    p = torch.exp(zz - lse[:, None]) * live[:, None]
    if experts is None:
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
        got = live[:, None] & (z.gather(1, order) > -math.inf)
        experts = torch.where(got, order, torch.full_like(order, -1))
    got = experts >= 0
    at = experts.clamp(min=0)
    w = p.gather(1, at) * got
    share = w.sum(1, keepdim=True)
    weights = w / torch.where(share > 0, share, torch.ones_like(share)) if renormalize else w
    D = len(off) - 1
    counts = torch.zeros(D, E, dtype=torch.int64)
    balance = z.new_zeros(())
    n = int(live.sum())
    slope = torch.zeros(N, E, dtype=torch.float64)
    for d in range(D):
        mine = live & (doc == d)
        nd = int(mine.sum())
        if nd == 0:
            continue
        counts[d] = torch.bincount(experts[mine][got[mine]], minlength=E)
        f = E * counts[d].double() / (k * nd)
        balance = balance + (nd / n) * (f * p[mine].sum(0) / nd).sum()
        slope[mine] = f / n
    zl = (lse[live] ** 2).sum() / max(n, 1)
    out = dict(weights=weights, experts=experts, counts=counts, balance=balance, z=zl, live=live, p=p, lse=lse, n=n)
    # the gradient by the formula, and the size of its terms
    u = d_balance * slope
    dw = torch.zeros(N, k, dtype=torch.float64) if d_weights is None else d_weights.double().cpu() * got
    inner = (dw * weights).sum(1, keepdim=True)
    c = weights * (dw - inner) if renormalize else w * dw
    chosen = torch.zeros(N, E, dtype=torch.float64).scatter_add_(1, at, c * got)
    dot = (p * u).sum(1, keepdim=True) + (0.0 if renormalize else inner)
    zterm = 2.0 * d_z * (lse * live)[:, None] / max(n, 1)
    out["d"] = p * (u - dot + zterm) + chosen
    mag = p * (u.abs() + (p * u.abs()).sum(1, keepdim=True) + (dw * weights).abs().sum(1, keepdim=True) + zterm.abs())
    out["mag"] = mag + torch.zeros(N, E, dtype=torch.float64).scatter_add_(
        1, at, (weights * (dw.abs() + (dw * weights).abs().sum(1, keepdim=True))) * got)
    return out


def rel_bound(z):
    """Relative error of an fp32 softmax entry: the exponent's argument d = z - m carries two roundings of
    |d| log2 e each, ex2 two units, the sum and the divide a few more, numerator and denominator alike."""
    zz = z.detach().double().cpu()
    fin = torch.isfinite(zz)
    top = torch.where(fin, zz, torch.full_like(zz, -math.inf)).amax(1)
    low = torch.where(fin, zz, torch.full_like(zz, math.inf)).amin(1)
    reach = float((top - low).clamp(min=0.0).max()) if zz.numel() else 0.0
    return 2.0 * (2.0 * 1.4427 * reach + 4.0 + 12.0) * U


def make(N, E, dtype, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, E, generator=g) * scale + torch.randn(1, E, generator=g) * 0.5
    return z.to(DT[dtype]), g


def compare(r, d, ref, z, dtype, documents):
    tol = rel_bound(z)
    assert torch.equal(r.experts.cpu().long(), ref["experts"])
    assert torch.equal(r.counts.cpu().view(documents, -1), ref["counts"])
    assert int(r.n_live.cpu()) == ref["n"]
    w = r.weights.cpu().double()
    assert bool(((w - ref["weights"]).abs() <= tol * ref["weights"]).all())
    # the sums over tokens: fp32 over at most ~300 tokens of a lane, then fp64
    for name in ("balance", "z"):
        got, want = float(getattr(r, name).cpu()), float(ref[name])
        assert abs(got - want) <= (2 * tol + 320 * U) * abs(want) + 1e-30, (name, got, want)
    if d is not None:
        err = (d.cpu().double() - ref["d"]).abs()
        lim = (3 * tol + 8 * U) * ref["mag"] + HALF_STEP[dtype] * (1 + 1e-3) * ref["d"].abs()
        lim = lim + {"fp32": 1e-44, "bf16": 1e-40, "fp16": 2.0 ** -25}[dtype]   # half a subnormal step
        assert bool((err <= lim).all()), float((err - lim).max())


def run(z, k, valid=None, offsets=None, renormalize=True, seed=0, view=None):
    import linear_cross_entropy_token_gb300 as flce
    N, E = z.shape
    g = torch.Generator().manual_seed(seed + 99)
    dw = torch.randn(N, k, generator=g)
    db, dz = 0.7, 0.3
    zc = z.cuda() if view is None else view(z)
    v = None if valid is None else valid.cuda()
    o = None if offsets is None else offsets.cuda()
    r = flce.route(zc, k, valid=v, offsets=o, renormalize=renormalize)
    d = flce.route_backward(r, zc, d_weights=dw.cuda(), d_balance=torch.tensor(db).cuda(),
                            d_z=torch.tensor(dz).cuda())
    f = lambda x: float(torch.tensor(x))  # noqa: E731  (the fp32 value the device got)
    ref = reference(z, k, valid, offsets, renormalize, dw, f(db), f(dz))
    return r, d, ref


SIZES = [(1, 1, 1), (1, 64, 4), (3, 2, 2), (5, 8, 3), (16, 64, 4), (33, 9, 9), (100, 17, 5), (257, 67, 6),
         (300, 128, 8), (511, 255, 8), (129, 256, 8), (70, 257, 7), (65, 500, 12), (40, 513, 4), (20, 1024, 32),
         (5000, 40, 6), (20000, 16, 2)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,E,k", SIZES)
def test_sizes(N, E, k, dtype):
    z, _ = make(N, E, dtype, N + E)
    for renorm in (True, False):
        r, d, ref = run(z, k, renormalize=renorm)
        compare(r, d, ref, z, dtype, 1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("documents", [1, 2, 7, 300])
def test_documents_and_masks(documents, dtype):
    N, E, k = 2000, 60, 4
    z, g = make(N, E, dtype, documents)
    z[:, -3:] = -math.inf                       # padded experts
    z[5] = -math.inf                            # a token with no expert at all
    z[6, 1:] = -math.inf                        # one expert only: k - 1 empty slots
    z[7] = torch.finfo(z.dtype).min             # masked by the type's lowest value: still live
    valid = torch.rand(N, generator=g) > 0.2
    cuts = torch.randint(0, N + 1, (documents - 1,), generator=g)
    if documents > 4:
        cuts[1] = cuts[0]                       # an empty document
        cuts[2] = 0                             # and one at the start
    offsets = torch.cat([torch.tensor([0, N]), cuts]).sort().values
    valid[offsets[0]:offsets[1]] = False        # a document with no live token
    z[7] = z[7].clamp(min=-1e4)                 # (squares of the lowest value leave fp32)
    r, d, ref = run(z, k, valid, offsets)
    compare(r, d, ref, z, dtype, documents)
    assert not r.weights[5].any() and bool((r.experts[5] == -1).all())
    assert not d.float().cpu()[~ref["live"]].any()


def test_lowest_value_masks():
    """Experts masked by the lowest finite value get weight 0 like -inf ones, but count as chosen."""
    z, _ = make(64, 12, "fp32", 3)
    z[:, 2:] = torch.finfo(torch.float32).min
    r, d, ref = run(z, 4)
    assert torch.equal(r.experts.cpu().long(), ref["experts"])
    assert torch.equal(r.counts.cpu().view(1, -1), ref["counts"])
    assert bool(torch.isfinite(d).all()) and not r.weights[:, 2:].any()


def test_all_tokens_masked_or_none_at_all():
    import linear_cross_entropy_token_gb300 as flce
    z, _ = make(50, 16, "fp32", 0)
    r, d, ref = run(z, 2, valid=torch.zeros(50, dtype=torch.bool))
    assert float(r.balance) == 0.0 and float(r.z) == 0.0 and not r.counts.any() and not d.any()
    r = flce.route(torch.empty(0, 16, device="cuda"), 2)
    assert float(r.balance) == 0.0 and float(r.z) == 0.0 and not r.counts.any()
    assert flce.route_backward(r, torch.empty(0, 16, device="cuda")).shape == (0, 16)


def test_ties_go_to_the_lowest_expert():
    import linear_cross_entropy_token_gb300 as flce
    for E in (7, 64, 200, 700):
        z = torch.zeros(40, E)
        z[:, E // 2] = 1.0
        z[3] = -0.0
        r = flce.route(z.cuda(), 4)
        want = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(r.experts.cpu().long(), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [5, 8, 16, 27, 64, 128, 200, 256, 384, 512, 1024])
def test_selection_where_the_largest_lie_together(E, dtype):
    """Which experts are chosen is exact, whatever their order: the largest side by side (in few lanes of a
    warp), last bits that differ, ties, signed zeros, -inf among them; one expert to 32."""
    from linear_cross_entropy_token_gb300 import route
    g = torch.Generator().manual_seed(E)
    N = 150
    up = torch.arange(E).float().repeat(N, 1) / 16
    together = torch.randn(N, E, generator=g)
    first = torch.randint(0, max(E - 9, 1), (N, 1), generator=g) + torch.arange(min(E, 9))
    together.scatter_add_(1, first, torch.full((N, first.shape[1]), 8.0))
    close = 1.0 + torch.randint(0, 40, (N, E), generator=g).float() * 2.0 ** -23
    few = torch.randint(0, 3, (N, E), generator=g).float() - 1.0
    zeros = torch.randint(0, 2, (N, E), generator=g).float() * -0.0
    zeros[:, ::2] *= -1.0
    holes = torch.where(torch.rand(N, E, generator=g) < 0.9, torch.full((), -math.inf), together)
    for rows in (up, -up, together, close, -close, few, zeros, holes, torch.zeros(N, E)):
        z = rows.to(DT[dtype])
        order = torch.sort(z.double(), dim=1, descending=True, stable=True).indices
        for k in sorted({1, min(E, 3), min(E, 8), min(E, 32)}):
            want = order[:, :k]
            want = torch.where(z.double().gather(1, want) > -math.inf, want, torch.full_like(want, -1))
            got = route(z.cuda(), k).experts.cpu().long()
            assert torch.equal(got, want), (k, int((got != want).any(1).nonzero()[0]))


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nan_and_infinite_logits_show(value):
    import linear_cross_entropy_token_gb300 as flce
    z, _ = make(100, 24, "fp32", 1)
    z[17, 5] = value
    r = flce.route(z.cuda(), 3)
    assert math.isnan(float(r.balance)) and bool(r.weights[17].isnan().all())
    assert int(r.experts.min()) >= -1 and int(r.experts.max()) < 24
    # the masked places of other tokens stay what they are
    keep = torch.arange(100) != 17
    assert bool(torch.isfinite(r.weights.cpu()[keep]).all())
    d = flce.route_backward(r, z.cuda(), d_balance=torch.ones((), device="cuda"))
    assert d.shape == (100, 24)
    # masked out, it does not count
    valid = keep.cuda()
    r = flce.route(z.cuda(), 3, valid=valid)
    d = flce.route_backward(r, z.cuda(), d_balance=torch.ones((), device="cuda"), d_z=torch.ones((), device="cuda"))
    assert math.isfinite(float(r.balance)) and bool(torch.isfinite(d).all()) and not d[17].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_and_unaligned_rows(dtype):
    z, _ = make(130, 37, dtype, 8)

    def odd(z):
        big = torch.full((130, 50), math.nan, dtype=z.dtype, device="cuda")
        big[:, 5:42] = z.cuda()
        return big[:, 5:42]

    def wide(z):
        big = torch.full((130, 64), math.nan, dtype=z.dtype, device="cuda")
        big[:, :37] = z.cuda()
        return big[:, :37]

    for view in (odd, wide):
        r, d, ref = run(z, 5, view=view)
        compare(r, d, ref, z, dtype, 1)


def test_offsets_out_of_order_stay_in_bounds():
    """Offsets that break their contract give unspecified numbers, no fault: tokens outside every
    document route nowhere."""
    import linear_cross_entropy_token_gb300 as flce
    z, _ = make(600, 32, "fp32", 5)
    for off in ([100, 300], [0, 500, 200, 600], [-50, 10, 9000], [700, 800, 900]):
        r = flce.route(z.cuda(), 2, offsets=torch.tensor(off, device="cuda"))
        d = flce.route_backward(r, z.cuda(), d_balance=torch.ones((), device="cuda"))
        assert int(r.experts.min()) >= -1 and int(r.experts.max()) < 32 and d.shape == z.shape
    r = flce.route(z.cuda(), 2, offsets=torch.tensor([100, 300], device="cuda"))
    assert bool((r.experts[:100] == -1).all()) and bool((r.experts[300:] == -1).all())
    assert int(r.n_live) == 200 and int(r.counts.sum()) == 400


def test_repeats_bit_for_bit_and_captures():
    import linear_cross_entropy_token_gb300 as flce
    z, g = make(3000, 96, "bf16", 2)
    zc = z.cuda()
    dw = torch.randn(3000, 6, generator=g).cuda()
    one = torch.ones((), device="cuda")

    def both():
        r = flce.route(zc, 6)
        return r, flce.route_backward(r, zc, d_weights=dw, d_balance=one, d_z=one)

    s = torch.cuda.Stream()                     # and on a stream of its own
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r1, d1 = both()
    torch.cuda.current_stream().wait_stream(s)
    r2, d2 = both()
    assert torch.equal(d1, d2) and torch.equal(r1.weights, r2.weights) and torch.equal(r1.state[:4], r2.state[:4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3, d3 = both()
    z2, _ = make(3000, 96, "bf16", 12)
    zc.copy_(z2)
    graph.replay()
    r4, d4 = both()
    assert torch.equal(d3, d4) and torch.equal(r3.counts, r4.counts) and torch.equal(r3.state[:4], r4.state[:4])


def test_autograd_against_formula_and_differences():
    from linear_cross_entropy_token_gb300.autograd import route
    N, E, k = 24, 10, 3
    z, g = make(N, E, "fp32", 4)
    valid = torch.ones(N, dtype=torch.bool)
    valid[4] = False
    offsets = torch.tensor([0, 9, 24])
    m = torch.randn(N, k, generator=g)
    for renorm in (True, False):
        zc = z.cuda().requires_grad_()
        w, e, c, bal, zl = route(zc, k, valid.cuda(), offsets.cuda(), renorm)
        ((w * m.cuda()).sum() + 0.7 * bal + 0.3 * zl).backward()
        ref = reference(z, k, valid, offsets, renorm, m, float(torch.tensor(0.7)), float(torch.tensor(0.3)))
        tol = rel_bound(z)
        lim = (3 * tol + 8 * U) * ref["mag"] + U * ref["d"].abs()
        assert bool(((zc.grad.cpu().double() - ref["d"]).abs() <= lim + 1e-44).all())
        # central differences of the definition with the selection held

        def total(x):
            o = reference(x, k, valid, offsets, renorm, experts=ref["experts"])
            return (o["weights"] * m.double()).sum() + 0.7 * o["balance"] + 0.3 * o["z"]

        h = 1e-5
        z64 = z.double()
        for i, j in ((0, 0), (3, 7), (4, 2), (11, int(ref["experts"][11, 0])), (23, int(ref["experts"][23, 2]))):
            up, dn = z64.clone(), z64.clone()
            up[i, j] += h
            dn[i, j] -= h
            diff = float((total(up) - total(dn)) / (2 * h))
            # h^2 times a third derivative of order 10, and what fp64 cancels
            assert abs(float(zc.grad[i, j]) - diff) <= 1e-8 + float(lim[i, j])
    # one loss alone, and weights alone
    zc = z.cuda().requires_grad_()
    route(zc, k)[3].backward()
    ref = reference(z, k, d_balance=1.0)
    assert bool(((zc.grad.cpu().double() - ref["d"]).abs() <= (3 * tol + 8 * U) * ref["mag"] + 1e-44).all())
    zc = z.cuda().requires_grad_()
    (route(zc, k)[0] * m.cuda()).sum().backward()
    ref = reference(z, k, d_weights=m)
    assert bool(((zc.grad.cpu().double() - ref["d"]).abs() <= (3 * tol + 8 * U) * ref["mag"] + 1e-44).all())


def test_a_given_output_counts_as_modified():
    import linear_cross_entropy_token_gb300 as flce
    z = torch.randn(20, 16, device="cuda")
    out = torch.zeros_like(z)
    r = flce.route(z, 2)
    before = out._version
    assert flce.route_backward(r, z, d_z=torch.ones((), device="cuda"), out=out) is out
    assert out._version > before


def test_a_second_derivative_is_refused():
    from linear_cross_entropy_token_gb300.autograd import route
    z = torch.randn(20, 16, device="cuda", requires_grad=True)
    # (the gradient that reaches the weights depends on z as well)
    d, = torch.autograd.grad(route(z, 2)[0].square().sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()
