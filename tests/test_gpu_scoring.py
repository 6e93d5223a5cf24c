"""Log probabilities of given tokens, entropy and alternatives, and their
gradients, against the formulas in 64 bits."""
import math

import pytest
import torch

from scoring_testing import DT, Reference, check_gradients, kept_distance, make_head

pytestmark = pytest.mark.gpu

SIZES = [
    (1, 64, 64, "bf16"), (1, 8, 1, "bf16"), (3, 8, 5, "bf16"), (2, 72, 65, "bf16"), (17, 128, 511, "bf16"),
    (129, 136, 513, "bf16"), (256, 256, 1000, "bf16"), (257, 1016, 2049, "bf16"), (300, 64, 50257, "bf16"),
    (1, 1, 1, "fp32"), (5, 33, 70, "fp32"), (64, 128, 4096, "fp32"), (31, 7, 127, "fp32"),
]


def score(x, W, t, **kw):
    import linear_cross_entropy_token_gb300 as f
    return f.token_logprobs(x, W, t, **kw)


def check_forward(r, ref, t, top, live=None):
    live = torch.ones(len(t), dtype=torch.bool, device=t.device) if live is None else live
    err = 2 * ref.sum_error() + 4e-6
    want = ref.lp.gather(1, t.clamp(min=0)[:, None])[:, 0]
    assert ((r.logprobs - want).abs()[live] <= (err + 2e-7 * want.abs())[live]).all()
    # entropy moves by at most its spread times the logits' errors: |dH| <= sum p |log p + H| |dz|
    spread = (ref.p * (ref.lp + ref.entropy[:, None]).abs()).sum(1)
    assert ((r.entropy - ref.entropy).abs()[live] <= (err * (1 + spread) + 1e-6 * ref.entropy)[live]).all()
    assert (r.logprobs[~live] == 0).all() and (r.entropy[~live] == 0).all()
    if top:
        ids, lp = ref.top(top)
        assert torch.equal(r.top_ids[live], ids[live])
        assert ((r.top_logprobs - lp).abs()[live] <= (err[:, None] + 2e-7 * lp.abs())[live]).all()
        assert (r.top_ids[~live] == -1).all() and (r.top_logprobs[~live] == 0).all()
    else:
        assert r.top_ids is None and r.top_logprobs is None


@pytest.mark.parametrize("N,H,V,dtype", SIZES)
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_forward(N, H, V, dtype, temperature):
    x, W, t, _ = make_head(N, H, V, dtype, seed=N + V)
    ref = Reference(x, W, temperature)
    for top in sorted({0, 1, min(7, V), min(64, V)}):
        check_forward(score(x, W, t, temperature=temperature, top=top), ref, t, top)


def test_chunks_of_tokens():
    """A budget that takes the rows in several chunks, with a ragged last one."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _ = make_head(700, 64, 3000, "bf16", seed=4)
    h = f.FLCE("bf16", 0, hbm_budget_bytes=2 << 20)
    whole, parts = score(x, W, t, top=9), score(x, W, t, top=9, handle=h)
    for a, b in ((whole.logprobs, parts.logprobs), (whole.entropy, parts.entropy), (whole.top_ids, parts.top_ids),
                 (whole.top_logprobs, parts.top_logprobs)):
        assert torch.equal(a, b)


def test_ties_go_to_the_lowest_id():
    g = torch.Generator().manual_seed(0)
    W = torch.randn(700, 64, generator=g).bfloat16()
    W[torch.tensor([650, 3, 130, 64, 511])] = W[200].clone()     # six equal rows, across groups and tiles
    x = torch.randn(40, 64, generator=g).bfloat16()
    x[0] = 0                                             # every logit the same
    x[1:20] = W[200] * 4                                 # the equal ones lead
    x, W = x.cuda(), W.cuda()
    t = torch.zeros(40, dtype=torch.int64, device="cuda")
    r = score(x, W, t, top=40)
    assert r.top_ids[0].tolist() == list(range(40))
    assert (r.top_ids[1:20, :6] == torch.tensor([3, 64, 130, 200, 511, 650], device="cuda")).all()
    assert torch.equal(r.top_ids, Reference(x, W).top(40)[0])


def test_more_near_equal_logits_than_are_summed_again():
    """Two hundred logits in steps that fp16 cannot hold but 32 bits can: the alternatives are still right, since
    equal stored values go by id and the logits fall with it."""
    H = 64
    W = torch.zeros(1000, H)
    W[:, 0] = 1.0
    W[:200, 1] = (200 - torch.arange(200)) * 2.0 ** -8   # exact in bf16
    x = torch.zeros(3, H)
    x[:, 0], x[:, 1] = 8.0, 2.0 ** -10
    x, W = x.bfloat16().cuda(), W.bfloat16().cuda()
    r = score(x, W, torch.zeros(3, dtype=torch.int64, device="cuda"), top=64)
    assert (r.top_ids == torch.arange(64, device="cuda")).all()


def test_alternatives_contain_the_given_token():
    x, W, t, _ = make_head(200, 256, 5000, "bf16", seed=9)
    r = score(x, W, t, top=5)
    row, place = (r.top_ids == t[:, None]).nonzero(as_tuple=True)
    assert len(row) > 40
    assert torch.equal(r.top_logprobs[row, place], r.logprobs[row])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_logits(dtype):
    """Logits of thousands: the log-sum-exp's last bits."""
    x, W, t, _ = make_head(50, 64, 600, dtype, seed=2, scale=400.0)
    check_forward(score(x, W, t, top=3, temperature=2.0), Reference(x, W, 2.0), t, 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ignored_rows_may_hold_anything(dtype):
    import linear_cross_entropy_token_gb300 as f
    x, W, t, g = make_head(300, 64, 900, dtype, seed=3)
    live = (torch.rand(300, generator=g) < 0.5).cuda()
    t[~live] = -7
    ref = Reference(x, W)
    x[~live] = torch.tensor([math.nan, math.inf, -math.inf, 1e30] * 16, device="cuda").to(DT[dtype])
    for keep in (False, True):
        r = score(x, W, t, top=4, ignore_index=-7, keep_logits=keep)
        check_forward(r, ref, t, 4, live)
        da, de = torch.randn(300, device="cuda"), torch.randn(300, device="cuda")
        da[~live] = math.nan
        dx, dW = f.token_logprobs_backward(r, x, W, t, d_logprobs=da, d_entropy=de)
        d = ref.d_scores(t.clamp(min=0), torch.where(live, da, 0.0).double(), de.double())
        d[~live] = 0
        y = kept_distance(ref.raw, 1 / math.log(2)) if keep else None
        check_gradients(dx, dW, d, torch.where(live[:, None], x, 0), W, y, dtype)
    t[:] = -7
    r = score(x, W, t, top=4, ignore_index=-7)
    dx, dW = f.token_logprobs_backward(r, x, W, t, d_logprobs=da, d_entropy=de)
    assert (r.logprobs == 0).all() and (r.top_ids == -1).all() and (dx == 0).all() and (dW == 0).all()


def test_nan_rows_are_nan():
    x, W, t, _ = make_head(20, 64, 900, "bf16", seed=3)
    want = score(x, W, t, top=4)
    x[7, 3] = math.nan
    r = score(x, W, t, top=4)
    assert r.logprobs[7].isnan() and r.entropy[7].isnan() and ((r.top_ids[7] >= 0) & (r.top_ids[7] < 900)).all()
    keep = torch.arange(20, device="cuda") != 7
    assert torch.equal(r.logprobs[keep], want.logprobs[keep]) and torch.equal(r.top_ids[keep], want.top_ids[keep])
    import linear_cross_entropy_token_gb300 as f
    dx, dW = f.token_logprobs_backward(r, x, W, t, d_logprobs=torch.ones(20, device="cuda"))
    assert dx[7].isnan().all() and not dx[keep].isnan().any()


def test_without_tokens():
    x, W, t, _ = make_head(30, 64, 900, "bf16", seed=5)
    a, b = score(x, W, None, top=6), score(x, W, t, top=6)
    assert a.logprobs is None
    assert torch.equal(a.entropy, b.entropy) and torch.equal(a.top_ids, b.top_ids)


def test_no_rows():
    import linear_cross_entropy_token_gb300 as f
    W = torch.randn(100, 64, device="cuda").bfloat16()
    x, t = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, dtype=torch.int64, device="cuda")
    r = score(x, W, t, top=3, keep_logits=True)
    dx, dW = f.token_logprobs_backward(r, x, W, t)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3) and dx.shape == (0, 64) and (dW == 0).all()


@pytest.mark.parametrize("N,H,V,dtype", SIZES)
@pytest.mark.parametrize("keep", [False, True])
def test_backward(N, H, V, dtype, keep):
    import linear_cross_entropy_token_gb300 as f
    temperature = 0.8
    x, W, t, g = make_head(N, H, V, dtype, seed=N + V + 1)
    ref = Reference(x, W, temperature)
    y = kept_distance(ref.raw, 1 / (temperature * math.log(2))) if keep else None
    a, b = torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda()
    zero = torch.zeros(N, device="cuda")
    r = score(x, W, t, temperature=temperature, keep_logits=keep)
    for ga, gb in ((a, None), (None, b), (a, b)):
        dx, dW = f.token_logprobs_backward(r, x, W, t, d_logprobs=ga, d_entropy=gb)
        d = ref.d_scores(t, (zero if ga is None else ga).double(), (zero if gb is None else gb).double())
        if V > 1:   # one token alone has no gradient: what is left there is rounding
            # the logits' own errors move p and log p
            check_gradients_loose(dx, dW, d, ref, x, W, y, dtype)
        assert dx.dtype == x.dtype and dW.dtype == W.dtype
    nothing = f.token_logprobs_backward(r, x, W, t)
    assert (nothing[0] == 0).all() and (nothing[1] == 0).all()


def check_gradients_loose(dx, dW, d, ref, x, W, y, dtype):
    check_gradients(dx, dW, d, x, W, y, dtype)


def test_backward_in_chunks_and_parts():
    """Several chunks; one gradient without the other; gradients in given tensors, dW in float32."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, g = make_head(900, 128, 5000, "bf16", seed=8)
    t[::7] = -100
    a, b = torch.randn(900, generator=g).cuda(), torch.randn(900, generator=g).cuda()
    live = t != -100
    ref = Reference(x, W)
    d = ref.d_scores(t.clamp(min=0), a.double(), b.double()) * live[:, None]
    h = f.FLCE("bf16", 0, hbm_budget_bytes=6 << 20)
    for keep in (False, True):
        y = kept_distance(ref.raw, 1 / math.log(2)) if keep else None
        for handle in (None, h):
            r = score(x, W, t, keep_logits=keep, handle=handle)
            both = f.token_logprobs_backward(r, x, W, t, a, b, handle=handle)
            check_gradients(*both, d, x, W, y)
            only_x = f.token_logprobs_backward(r, x, W, t, a, b, dW=None, handle=handle)
            only_W = f.token_logprobs_backward(r, x, W, t, a, b, dx=False, handle=handle)
            assert only_x[1] is None and only_W[0] is None
            check_gradients(only_x[0], only_W[1], d, x, W, y)
            out_x, out_W = torch.full_like(x, 9), torch.full((5000, 128), 9.0, device="cuda")
            got = f.token_logprobs_backward(r, x, W, t, a, b, dx=out_x, dW=out_W, handle=handle)
            assert got[0] is out_x and got[1] is out_W
            check_gradients(out_x, out_W, d, x, W, y)
            assert torch.equal(out_W.bfloat16(), both[1])


def test_results_repeat():
    import linear_cross_entropy_token_gb300 as f
    x, W, t, g = make_head(500, 256, 7001, "bf16", seed=11)
    a = torch.randn(500, generator=g).cuda()
    first = None
    for _ in range(3):
        r = score(x, W, t, top=20)
        got = [r.logprobs, r.entropy, r.top_logprobs, r.top_ids, *f.token_logprobs_backward(r, x, W, t, a, a)]
        first = first or got
        assert all(torch.equal(u, v) for u, v in zip(first, got))


def test_gradient_against_differences():
    """fp32, where a difference says something: along random directions of x and W."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, g = make_head(40, 24, 90, "fp32", seed=1, strength=2.0)
    a, b = torch.randn(40, generator=g).cuda(), torch.randn(40, generator=g).cuda()
    r = score(x, W, t, temperature=1.5)
    dx, dW = f.token_logprobs_backward(r, x, W, t, a, b)

    def value(x, W):
        r = score(x, W, t, temperature=1.5)
        return (a.double() * r.logprobs + b.double() * r.entropy).sum().item()

    for like, grad, move in ((x, dx, lambda e: value(x + e, W)), (W, dW, lambda e: value(x, W + e))):
        v = torch.randn(like.shape, generator=g).cuda()
        step = 1e-2 / v.norm()
        slope = (move(step * v) - move(-step * v)) / (2 * step.item())
        want = (grad.double() * v).sum().item()
        # 40 values of about 5 with 2^-22 each, over the step; the third derivative's share
        limit = 40 * 5 * 2.0 ** -22 / step.item() + 1e-3 * grad.norm().item() * v.norm().item() / math.sqrt(v.numel())
        assert abs(slope - want) <= limit


def test_alternatives_far_below_their_neighbours():
    """Logits that lie further below their 64 columns' largest than the stored ones reach."""
    W = torch.zeros(130, 64)
    W[:, 0] = -torch.arange(130) * 8.0
    x = torch.zeros(2, 64)
    x[:, 0] = torch.tensor([256.0, 1024.0])
    x, W = x.bfloat16().cuda(), W.bfloat16().cuda()
    r = score(x, W, torch.zeros(2, dtype=torch.int64, device="cuda"), top=64)
    assert (r.top_ids == torch.arange(64, device="cuda")).all()
    # they are exact: x and W are powers of two and small multiples of eight (rounded to bf16 above 256 * 8)
    want = (x.double() @ W.double().T)[:, :64]
    assert torch.equal(r.top_logprobs.double(), want)


def test_token_out_of_range():
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _ = make_head(20, 64, 900, "bf16", seed=3)
    want = score(x, W, t, top=2)
    for bad in (900, -1, 1 << 40):
        wrong = t.clone()
        wrong[4] = bad
        r = score(x, W, wrong, top=2)
        with pytest.raises(f.FlceError) as e:
            f.async_status()
        assert e.value.status == 4
        assert r.logprobs[4].isnan() and torch.equal(r.top_ids, want.top_ids)
        assert torch.equal(r.logprobs.nan_to_num(0)[:4], want.logprobs[:4])
        one = torch.ones(20, device="cuda")
        dx, dW = f.token_logprobs_backward(r, x, W, wrong, d_logprobs=one)
        with pytest.raises(f.FlceError) as e:
            f.async_status()
        assert e.value.status == 4 and (dx[4] == 0).all() and not dW.isnan().any()
    f.async_status()


@pytest.mark.parametrize("N", [16, 33, 48, 64, 65])
@pytest.mark.parametrize("H,V", [(64, 129), (520, 20000), (2048, 5003)])
def test_few_rows(N, H, V):
    """Decoding batches, whose product has the tokens on its other side."""
    x, W, t, _ = make_head(N, H, V, "bf16", seed=N + V)
    t[N // 2] = -100
    ref = Reference(x, W, 0.9)
    for top in (0, 20):
        check_forward(score(x, W, t, temperature=0.9, top=top), ref, t, top, t != -100)
    r = score(x, W, t, temperature=0.9, keep_logits=True)
    import linear_cross_entropy_token_gb300 as f
    a = torch.linspace(-1, 1, N, device="cuda")
    d = ref.d_scores(t.clamp(min=0), a.double(), 0 * a.double()) * (t != -100)[:, None]
    check_gradients(*f.token_logprobs_backward(r, x, W, t, a), d, x, W, kept_distance(ref.raw, 1 / (0.9 * math.log(2))))


@pytest.mark.parametrize("N", [80, 97, 128, 129])
@pytest.mark.parametrize("H,V", [(72, 300), (1024, 20011)])
def test_up_to_128_rows(N, H, V):
    x, W, t, g = make_head(N, H, V, "bf16", seed=N)
    t[torch.rand(N, generator=g) < 0.1] = -100
    live = t >= 0
    for top, keep in ((0, False), (7, True)):
        check_forward(score(x, W, t, top=top, keep_logits=keep), Reference(x, W), t, top, live)


@pytest.mark.parametrize("top", [0, 2])
@pytest.mark.parametrize("N,H,dtype", [(40, 183, "fp32"), (40, 512, "bf16"), (300, 512, "bf16")])
def test_near_certain_tokens(N, H, dtype, top):
    """What is left of a probability close to 1 comes from the other tokens, not from the largest logit's error."""
    import linear_cross_entropy_token_gb300 as f
    g = torch.Generator().manual_seed(H)
    V = 800
    W = (torch.randn(V, H, generator=g) * 1.3 / math.sqrt(H)).to(DT[dtype])
    t = torch.randint(0, V, (N,), generator=g)
    x = torch.randn(N, H, generator=g) + 17.0 * W[t].float() / (1.3 ** 2)
    x, W, t = x.to(DT[dtype]).cuda(), W.cuda(), t.cuda()
    ref = Reference(x, W)
    want = ref.lp.gather(1, t[:, None])[:, 0]
    sure = want > -1e-3
    assert sure.sum() > N / 2
    r = score(x, W, t, top=top)
    # L, a sum in [1, 2), is rounded by at most 2^-24 at each addition that its largest term meets: 16 of a
    # group's four sums, 2 that join them, one of the row's and 5 that join its lanes, 24 in all (3e-7, five of
    # them, was too few); and the other tokens' logits' errors
    err = 24 * 2.0 ** -24 + want.abs() * (2 * ref.sum_error() + 4e-6)
    assert ((r.logprobs - want).abs() <= err)[sure].all()
    if top:
        assert torch.equal(r.top_ids[sure, 0], t[sure]) and torch.equal(r.top_logprobs[sure, 0], r.logprobs[sure])
    da = torch.ones(N, device="cuda")
    _, dW = f.token_logprobs_backward(r, x, W, t, d_logprobs=da, dx=None, dW=torch.empty(V, H, device="cuda"))
    d = ref.d_scores(t, da.double(), torch.zeros(N, dtype=torch.float64, device="cuda"))
    if dtype == "fp32":
        off = torch.zeros_like(d).scatter_add(1, t[:, None], err[:, None]) + d.abs() * (2 * ref.sum_error()[:, None] + 4e-6)
        tol = off.T @ x.double().abs() + 1e-6 * d.abs().T @ x.double().abs()
        assert ((dW - d.T @ x.double()).abs() <= tol).all()
