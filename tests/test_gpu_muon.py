"""The orthogonalised momentum update on the GPU against its definition in
float64: shapes on both sides of the tiles, types, strides, momentum, weights,
spectra and scales."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# O against the exact map, in units of its own norm: per step the roundings of
# A, B and X to fp16 (half a step 2^-11 each) enter relative to the whole X;
# they add as independent errors over the products and as many steps as still
# change X, 3 sqrt(3) 2^-11 = 2.5e-3, with the map's slope (at most 2 where
# the singular values settle) for what earlier steps left: twice that
ORTHO = 5e-3


def newton_schulz(u, steps=5, coef=COEF, eps=1e-7, scale=1.0):
    x = u.double().cuda()
    x = x / (torch.linalg.vector_norm(x) + eps)
    rows = [coef] * steps if not hasattr(coef[0], "__len__") else coef
    for a, b, c in rows:
        a, b, c = (float(torch.tensor(v)) for v in (a, b, c))
        left = x.shape[0] <= x.shape[1]
        g = x @ x.mT if left else x.mT @ x
        q = b * g + c * (g @ g)
        x = a * x + (q @ x if left else x @ q)
    return (x * scale).cpu()


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm()) if float(b.norm()) else float(a.norm())


def gaussian(rows, cols, seed, scale=1e-3):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)) * scale


SHAPES = [(1, 1), (1, 9), (9, 1), (5, 64), (64, 5), (33, 33), (64, 64), (65, 130), (128, 128), (129, 257), (257, 129),
          (128, 256), (100, 257), (512, 128), (128, 1024), (1500, 60), (70, 2100), (4096, 128), (128, 4097),
          (200, 3000), (5000, 300), (40, 4600), (256, 256), (300, 1000), (1000, 300), (512, 513), (700, 640), (1024, 96), (72, 5000), (2000, 1100)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize_shapes(rows, cols):
    from linear_cross_entropy_token_gb300 import orthogonalize
    G = gaussian(rows, cols, rows * 7 + cols)
    want = newton_schulz(G, scale=0.5)
    got = orthogonalize(G.cuda(), scale=0.5, dtype=torch.float32)
    assert rel(got, want) <= ORTHO
    got = orthogonalize(G.cuda(), scale=0.5)
    assert got.dtype == torch.bfloat16 and rel(got, want) <= ORTHO + 2.0 ** -8
    got = orthogonalize(G.bfloat16().cuda(), scale=0.5, dtype=torch.float32)
    assert rel(got, newton_schulz(G.bfloat16(), scale=0.5)) <= ORTHO


@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_tile_shapes(rows, cols, cta):
    """The tiled products on each tile shape, for sizes that the one-launch kernel takes too."""
    from linear_cross_entropy_token_gb300 import FLCE, orthogonalize
    h = FLCE("bf16", 0, cta=cta)
    try:
        G = torch.stack([gaussian(rows, cols, rows * 7 + cols + i) for i in range(2)])
        got = orthogonalize(G.cuda(), dtype=torch.float32, handle=h)
        for i in range(2):
            assert rel(got[i], newton_schulz(G[i])) <= ORTHO
        h.async_status()
    finally:
        h.close()


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols,count", [(96, 200, 3), (200, 96, 2), (131, 77, 1), (260, 516, 2), (48, 40, 70)])
def test_update_with_momentum_and_weights(rows, cols, count, nesterov, grad):
    from linear_cross_entropy_token_gb300 import muon_update
    beta, lr, wd, scale = 0.9, 0.05, 0.1, 3.0
    g = [gaussian(rows, cols, i).to(grad) for i in range(count)]
    m = [gaussian(rows, cols, 100 + i) for i in range(count)]
    kw = dict(beta=beta, nesterov=nesterov, scale=scale)
    want_m, want_o = [], []
    for gi, mi in zip(g, m):
        buf = beta * mi.double() + (1 - beta) * gi.double()
        want_m.append(buf)
        want_o.append(newton_schulz(beta * buf + (1 - beta) * gi.double() if nesterov else buf, scale=scale))
    gc = [t.cuda() for t in g]
    mc = [t.cuda() for t in m]
    up = muon_update(gc, mc, **kw)
    for a, b, o, w in zip(mc, want_m, up, want_o):
        # two products and a sum, each rounded
        assert bool(((a.cpu().double() - b).abs() <= 4 * 2.0 ** -24 * (b.abs() + 1e-3)).all())
        assert rel(o, w) <= ORTHO + 2.0 ** -8
    for dt in (torch.float32, torch.bfloat16):
        w = [(0.02 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(i))).to(dt) for i in range(count)]
        wc = [t.cuda() for t in w]
        mc = [t.cuda() for t in m]
        out = muon_update(gc, mc, wc, lr=lr, weight_decay=wd, **kw)
        assert out[0] is wc[0]
        for wi, got, o in zip(w, wc, want_o):
            want = (1 - lr * wd) * wi.double() - lr * o
            err = (got.cpu().double() - want).norm()
            lim = lr * ORTHO * o.norm() + HALF_STEP[dt] * 2 * want.norm()
            assert float(err) <= float(lim)


def _spectrum(m, n, s):
    g = torch.Generator().manual_seed(m + n)
    u, _ = torch.linalg.qr(torch.randn(m, m, generator=g, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(n, m, generator=g, dtype=torch.float64))
    return (u * s) @ v.mT


@pytest.mark.parametrize("kind", ["rank1", "rank16", "rank16+noise", "1/i", "1/i^2", "one row", "one entry",
                                  "orthogonal", "equal rows"])
@pytest.mark.parametrize("m,n", [(128, 128), (320, 700)])
def test_spectra(kind, m, n):
    """Low rank and fast-decaying spectra: the small singular directions are raised by up to 3.4445^5, and
    rounding noise in them with it, unless X keeps more bits than the products' operands."""
    from linear_cross_entropy_token_gb300 import orthogonalize
    i = torch.arange(1, m + 1, dtype=torch.float64)
    if kind.startswith("rank16"):
        G = (gaussian(m, 16, 1, 1) @ gaussian(16, n, 2, 1)).double()
        if kind.endswith("noise"):
            G = G + gaussian(m, n, 3, 0.05)
    elif kind == "one entry":
        G = torch.zeros(m, n, dtype=torch.float64)
        G[5, 7] = -2.0
    elif kind == "one row":
        G = torch.zeros(m, n, dtype=torch.float64)
        G[3] = gaussian(1, n, 4, 1)[0]
    elif kind == "equal rows":
        G = gaussian(1, n, 5, 1).double().expand(m, n).clone()
    else:
        G = _spectrum(m, n, {"rank1": (i == 1).double(), "1/i": 1 / i, "1/i^2": 1 / i ** 2,
                             "orthogonal": torch.ones_like(i)}[kind])
    G = G.float()
    for g in (G, G.t().contiguous()):
        assert rel(orthogonalize(g.cuda(), dtype=torch.float32), newton_schulz(g)) <= ORTHO


@pytest.mark.parametrize("scale,eps", [(1e30, 1e-7), (3e37, 1e-7), (1e-22, 0.0), (1e-35, 0.0), (1e-3, 1.0)])
def test_magnitudes(scale, eps):
    """Sums of squares that leave fp32 on either side, and an eps that counts."""
    from linear_cross_entropy_token_gb300 import orthogonalize
    G = gaussian(96, 160, 6, 1).clamp(-3, 3) * scale
    assert rel(orthogonalize(G.cuda(), eps=eps, dtype=torch.float32), newton_schulz(G, eps=eps)) <= ORTHO


def test_zero_nan_and_infinite_gradients():
    from linear_cross_entropy_token_gb300 import muon_update, orthogonalize
    assert not orthogonalize(torch.zeros(40, 70, device="cuda")).any()
    for bad in (math.nan, math.inf):
        G = gaussian(40, 70, 1)
        G[3, 4] = bad
        fine = gaussian(40, 70, 2)
        # matrices of one call do not touch each other
        a, b = muon_update([G.cuda(), fine.cuda()], update_dtype=torch.float32)
        assert bool(a.isnan().any()) and rel(b, newton_schulz(fine)) <= ORTHO


@pytest.mark.parametrize("rows,cols", [(60, 100), (100, 60)])
def test_strides_and_offsets(rows, cols):
    from linear_cross_entropy_token_gb300 import muon_update
    beta, lr = 0.8, 0.1
    for pad, off in ((3, 1), (4, 0), (8, 4)):
        def view(t, dtype):
            big = torch.full((rows, cols + pad + off), math.nan, dtype=dtype, device="cuda")
            big[:, off:off + cols] = t.cuda()
            return big, big[:, off:off + cols]
        g, m, w = (gaussian(rows, cols, i) for i in range(3))
        for gt in (torch.float32, torch.bfloat16):
            _, gv = view(g.to(gt), gt)
            mbig, mv = view(m, torch.float32)
            wbig, wv = view(w, torch.float32)
            ubig, uv = view(w, torch.bfloat16)
            muon_update([gv], [mv], updates=[uv], beta=beta)
            buf = beta * m.double() + (1 - beta) * g.to(gt).double()
            o = newton_schulz(beta * buf + (1 - beta) * g.to(gt).double())
            assert rel(uv, o) <= ORTHO + 2.0 ** -8
            mv.copy_(m)
            muon_update([gv], [mv], [wv], beta=beta, lr=lr)
            assert float((wv.cpu().double() - (w.double() - lr * o)).norm()) <= lr * ORTHO * float(o.norm()) + 1e-6
            for big in (mbig, wbig, ubig):      # nothing is written beside the matrix
                assert bool(big[:, :off].isnan().all()) and bool(big[:, off + cols:].isnan().all())


def test_steps_and_coefficients():
    from linear_cross_entropy_token_gb300 import orthogonalize
    G = gaussian(150, 210, 3)
    for steps, coef in ((1, COEF), (2, COEF), (8, COEF), (3, (1.5, -0.5, 0.0)), (3, (1.875, -1.25, 0.375)),
                        (2, [COEF, (1.5, -0.5, 0.0)])):
        got = orthogonalize(G.cuda(), steps=steps, coefficients=coef, dtype=torch.float32)
        assert rel(got, newton_schulz(G, steps, coef)) <= ORTHO, (steps, coef)


def test_batches_repeats_and_streams():
    from linear_cross_entropy_token_gb300 import FLCE, orthogonalize
    G = torch.stack([gaussian(90, 300, i) for i in range(40)]).view(5, 8, 90, 300).cuda()
    a = orthogonalize(G, dtype=torch.float32)
    for i in range(0, 40, 13):
        one = orthogonalize(G.view(40, 90, 300)[i], dtype=torch.float32)
        # (the number of matrices sets the CTAs per matrix, and with them the order of sums)
        for got in (one, a.view(40, 90, 300)[i]):
            assert rel(got, newton_schulz(G.view(40, 90, 300)[i].cpu())) <= ORTHO
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = orthogonalize(G, dtype=torch.float32)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)
    assert orthogonalize(torch.empty(0, 5, 6, device="cuda")).shape == (0, 5, 6)
    h = FLCE("fp32", 0)
    try:
        n = h.launch_count()
        assert torch.equal(orthogonalize(G, dtype=torch.float32, handle=h), a)
        assert h.launch_count() > n
        h.async_status()
    finally:
        h.close()


def test_captured_update_replays_on_new_gradients():
    from linear_cross_entropy_token_gb300 import muon_update
    g = gaussian(128, 256, 1).cuda()
    m = torch.zeros(128, 256, device="cuda")
    w = gaussian(128, 256, 2, 0.02).cuda()
    muon_update([g.clone()], [m.clone()], [w.clone()], lr=0.1)
    m0, w0 = m.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        muon_update([g], [m], [w], lr=0.1)
    m.copy_(m0), w.copy_(w0)
    for k in range(3):
        g.copy_(gaussian(128, 256, 10 + k))
        muon_update([g], [m0], [w0], lr=0.1)
        graph.replay()
        assert torch.equal(m, m0) and torch.equal(w, w0)


def test_optimizer_steps_parameters_of_several_shapes():
    from linear_cross_entropy_token_gb300 import Muon
    shapes = [(64, 96), (64, 96), (96, 64), (128, 32)]
    ps = [torch.nn.Parameter(gaussian(r, c, i, 0.02).cuda()) for i, (r, c) in enumerate(shapes)]
    ps.append(torch.nn.Parameter(gaussian(8, 8, 9).cuda()))      # has no gradient: untouched
    kept = ps[-1].detach().clone()
    opt = Muon(ps, lr=0.02, weight_decay=0.1, beta=0.9)
    w = [p.detach().cpu().double() for p in ps]
    m = [torch.zeros_like(x) for x in w]
    for it in range(3):
        for i, (r, c) in enumerate(shapes):
            ps[i].grad = gaussian(r, c, 50 * it + i).cuda()
        opt.step()
        for i, (r, c) in enumerate(shapes):
            gi = ps[i].grad.cpu().double()
            m[i] = 0.9 * m[i] + 0.1 * gi
            o = newton_schulz(0.9 * m[i] + 0.1 * gi, scale=0.2 * math.sqrt(max(r, c)))
            w[i] = (1 - 0.02 * 0.1) * w[i] - 0.02 * o
            assert float((ps[i].detach().cpu().double() - w[i]).norm()) <= (it + 1) * 0.02 * ORTHO * float(o.norm()) + 1e-5
    assert torch.equal(ps[-1].detach(), kept)


def test_a_backward_over_updated_weights_fails():
    """Weights and momenta change in place: autograd must not use the new values for an old forward."""
    from linear_cross_entropy_token_gb300 import muon_update
    w = torch.nn.Parameter(torch.randn(32, 48, device="cuda"))
    m = torch.zeros(32, 48, device="cuda")
    x = torch.randn(8, 48, device="cuda", requires_grad=True)
    before = w._version, m._version
    loss = (x @ w.T).square().sum()
    muon_update([torch.randn(32, 48, device="cuda")], [m], [w.detach()], lr=0.1)
    assert w._version > before[0] and m._version > before[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    u = torch.empty(32, 48, device="cuda", dtype=torch.bfloat16)
    muon_update([torch.randn(32, 48, device="cuda")], updates=[u])
    assert u._version == 1
