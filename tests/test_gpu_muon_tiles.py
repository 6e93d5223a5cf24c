"""The tiled products of the orthogonalised update where their order counts: more
tiles than fit at once, tiles whose epilogue refills its buffers, many matrices
in one launch and in several groups, split sums. Against float64, and repeated
bit for bit: a wait or a barrier that is missing shows as a difference."""
import pytest
import torch

from test_gpu_muon import HALF_STEP, ORTHO, gaussian, newton_schulz

pytestmark = pytest.mark.gpu


def check_updates(rows, cols, count, weight_dtype, cta="auto", repeats=3, seed=0):
    """Momentum, orthogonalisation and weight update of `count` different matrices, three times from one start."""
    from linear_cross_entropy_token_gb300 import FLCE, muon_update
    beta, lr, wd, scale = 0.9, 0.05, 0.1, 2.0
    g = [gaussian(rows, cols, seed + i) for i in range(count)]
    m = [gaussian(rows, cols, seed + 1000 + i) for i in range(count)]
    w = [gaussian(rows, cols, seed + 2000 + i, 0.02).to(weight_dtype) for i in range(count)]
    gc = [t.cuda() for t in g]
    h = FLCE("bf16", 0, cta=cta)
    try:
        first = None
        for _ in range(repeats):
            mc, wc = [t.cuda() for t in m], [t.cuda() for t in w]
            muon_update(gc, mc, wc, beta=beta, scale=scale, lr=lr, weight_decay=wd, handle=h)
            if first is None:
                first = mc, wc
            assert all(torch.equal(a, b) for a, b in zip(mc + wc, first[0] + first[1]))
        h.async_status()
    finally:
        h.close()
    mc, wc = first
    for i in range(count):
        buf = beta * m[i].double() + (1 - beta) * g[i].double()
        assert bool(((mc[i].cpu().double() - buf).abs() <= 4 * 2.0 ** -24 * (buf.abs() + 1e-3)).all())
        o = newton_schulz(beta * buf + (1 - beta) * g[i].double(), scale=scale)
        want = (1 - lr * wd) * w[i].double() - lr * o
        err = float((wc[i].cpu().double() - want).norm())
        # the map's error, and the result's rounding with the two of the fp32 update before it
        assert err <= lr * ORTHO * float(o.norm()) + 2 * HALF_STEP[weight_dtype] * float(want.norm())


@pytest.mark.parametrize("weight_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
@pytest.mark.parametrize("rows,cols", [(9000, 1100), (1100, 9000)])
def test_more_tiles_than_fit_at_once(rows, cols, cta, weight_dtype):
    """X has more tiles than the GPU holds at once (90 of 256 x 512 on 76 pairs); the last step of a tall matrix writes its columns, and on the
    widest tiles loads the next group into the buffer that it has just read."""
    check_updates(rows, cols, 1, weight_dtype, cta)


@pytest.mark.parametrize("rows,cols,count", [(300, 1000, 8), (150, 200, 35), (256, 4096, 3), (5000, 300, 3), (129, 130, 33)])
def test_many_matrices_and_groups(rows, cols, count):
    """Different matrices side by side in one launch, their sums split, and more of them than one group holds
    (32), so that the second group takes over the first one's workspace."""
    check_updates(rows, cols, count, torch.float32)


@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
def test_groups_on_each_tile_shape(cta):
    check_updates(300, 500, 34, torch.bfloat16, cta)
