"""The head's operators as they are used together: in autograd, in captured graphs,
on several streams and handles, beside the fused loss; and what their C entries
refuse."""
import ctypes
import math

import pytest
import torch

from scoring_testing import Reference, check_gradients, make_head

pytestmark = pytest.mark.gpu


def policy_loss(logprobs, entropy, advantage):
    return -(advantage * logprobs).mean() - 0.01 * entropy.mean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("keep", [False, True])
def test_policy_gradient_through_autograd(dtype, keep):
    from linear_cross_entropy_token_gb300.autograd import token_logprobs
    x, W, t, g = make_head(300, 64, 1500, dtype, seed=1)
    t[::4] = -100
    live = (t != -100).cuda()
    advantage = torch.randn(300, generator=g).cuda()
    x.requires_grad_(), W.requires_grad_()
    logprobs, entropy, top, ids = token_logprobs(x, W, t, temperature=0.9, top=3, keep_logits=keep)
    assert not top.requires_grad and not ids.requires_grad
    policy_loss(logprobs, entropy, advantage).backward()
    ref = Reference(x.detach(), W.detach(), 0.9)
    want = ref.lp.gather(1, t.clamp(min=0)[:, None])[:, 0]
    assert ((logprobs - want).abs()[live] <= (2 * ref.sum_error() + 4e-6 + 2e-7 * want.abs())[live]).all()
    d = ref.d_scores(t.clamp(min=0), -advantage.double() / 300, torch.full_like(want, -0.01 / 300)) * live[:, None]
    c = 1 / (0.9 * math.log(2))
    from scoring_testing import kept_distance
    check_gradients(x.grad, W.grad, d, x.detach(), W.detach(), kept_distance(ref.raw, c) if keep else None, dtype)


def test_gradients_that_are_not_asked_for():
    """A frozen head, a frozen trunk, a loss on one of the outputs, and none at all."""
    from linear_cross_entropy_token_gb300.autograd import linear_distillation, token_logprobs
    x, W, t, g = make_head(300, 64, 1500, "bf16", seed=2)
    grads = {}
    for which in ("x", "W", "both"):
        a, b = x.clone().requires_grad_(which != "W"), W.clone().requires_grad_(which != "x")
        logprobs, entropy, _, _ = token_logprobs(a, b, t)
        logprobs.sum().backward()
        ids, z = t[:, None] + torch.zeros(1, 1, dtype=torch.int64, device="cuda"), torch.zeros(300, 1, device="cuda")
        c, e = x.clone().requires_grad_(which != "W"), W.clone().requires_grad_(which != "x")
        (2 * linear_distillation(c, e, ids, z)).backward()
        grads[which] = (a.grad, b.grad, c.grad, e.grad)
    for i, which in enumerate(("x", "W", "x", "W")):
        one, both = grads[which][i], grads["both"][i]
        assert grads["W" if which == "x" else "x"][i] is None
        assert (one.double() - both.double()).norm() <= 2.0 ** -8 * both.double().norm()
    with torch.no_grad():
        assert not token_logprobs(x, W, t)[0].requires_grad
        assert not linear_distillation(x, W, t[:, None], torch.zeros(300, 1, device="cuda")).requires_grad


def test_evaluating_parameters_computes_no_gradients():
    import linear_cross_entropy_token_gb300 as f
    from linear_cross_entropy_token_gb300.autograd import linear_distillation, token_logprobs
    x, W, t, ids, z, _ = inputs(3)
    h = f.FLCE("bf16", 0)

    def launches(call):
        before = h.launch_count()
        call()
        return h.launch_count() - before

    want = launches(lambda: f.distill(x, W, ids, z, backward=False, handle=h))
    a, b = x.clone().requires_grad_(), W.clone().requires_grad_()
    with torch.no_grad():
        assert launches(lambda: linear_distillation(a, b, ids, z, handle=h)) == want
        held = torch.cuda.memory_allocated()
        r = token_logprobs(a, b, t, keep_logits=True, handle=h)
        assert torch.cuda.memory_allocated() - held < x.shape[0] * W.shape[0]
    assert not r[0].requires_grad
    assert launches(lambda: linear_distillation(a, b, ids, z, handle=h)) > want


def test_one_hot_teacher_is_the_cross_entropy():
    """Distillation from one entry a token, the loss it trains beside, and the log probabilities agree."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _ = make_head(500, 128, 3000, "bf16", seed=3)
    t[::7] = -100
    loss, dx, dW = f.forward_backward(x, W, t)
    ids = torch.where(t < 0, -1, t)[:, None].contiguous()
    kl, kdx, kdW = f.distill(x, W, ids, torch.zeros(500, 1, device="cuda"), dW=torch.empty(3000, 128, device="cuda"))
    r = f.token_logprobs(x, W, t)
    n = (t >= 0).sum()
    assert abs(kl.item() - loss) <= 1e-3 * loss       # the loss takes its sums from bf16 logits
    assert abs(kl.item() + (r.logprobs.sum() / n).item()) <= 2e-6 * (1 + loss)
    g = torch.full((500,), -1.0 / n.item(), device="cuda")
    sdx, sdW = f.token_logprobs_backward(r, x, W, t, g, dW=torch.empty(3000, 128, device="cuda"))
    for a, b in ((kdx, dx), (kdW, dW), (sdx, dx), (sdW, dW)):
        # two roundings of the same entries (and those of the loss's bf16 logits)
        assert (a.double() - b.double()).norm() <= 1e-2 * b.double().norm()


def test_what_the_backward_reads_may_not_change():
    from linear_cross_entropy_token_gb300.autograd import token_logprobs
    for which in ("x", "W", "t", "entropy"):
        x, W, t, _ = make_head(300, 64, 900, "bf16", seed=4)
        x.requires_grad_(), W.requires_grad_()
        logprobs, entropy, _, _ = token_logprobs(x, W, t)
        with torch.no_grad():
            {"x": x, "W": W, "t": t, "entropy": entropy.detach()}[which].add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            logprobs.sum().backward()


def run_all(f, x, W, t, ids, z, a, keep):
    r = f.token_logprobs(x, W, t, top=4, keep_logits=keep)
    dx, dW = f.token_logprobs_backward(r, x, W, t, a, a)
    return [r.logprobs, r.entropy, r.top_logprobs, r.top_ids, dx, dW, *f.distill(x, W, ids, z, 1.3)]


def inputs(seed, N=400, V=2500):
    x, W, t, g = make_head(N, 64, V, "bf16", seed=seed)
    t[torch.rand(N, generator=g) < 0.3] = -100
    ids = torch.randint(0, V, (N, 6), generator=g).cuda()
    z = torch.randn(N, 6, generator=g)
    z[torch.rand(N, generator=g) < 0.2] = -math.inf
    return x, W, t, ids, z.cuda(), torch.randn(N, generator=g).cuda()


@pytest.mark.parametrize("keep", [False, True])
def test_captured_and_replayed_on_new_inputs(keep):
    """How many rows count is read on the device, so a captured step follows it."""
    import linear_cross_entropy_token_gb300 as f
    buffers = inputs(0)
    run_all(f, *buffers, keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_all(f, *buffers, keep)
    for seed, share in ((5, None), (6, 0.0), (7, 1.0), (0, None)):
        new = inputs(seed)
        if share is not None:   # all rows count, or none does
            new[2].copy_(torch.full_like(new[2], -100) if share else new[2].clamp(min=0))
            new[4].copy_(torch.full_like(new[4], -math.inf) if share else torch.zeros_like(new[4]))
        for b, n in zip(buffers, new):
            b.copy_(n)
        graph.replay()
        want = run_all(f, *new, keep)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_two_graphs_and_an_eager_call_share_nothing():
    import linear_cross_entropy_token_gb300 as f
    sets = [inputs(s) for s in (1, 2)]
    want = [run_all(f, *s, False) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_all(f, *s, False))
        graphs.append(g)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
        eager = run_all(f, *sets[0], False)
    torch.cuda.synchronize()
    for got, w in zip((*outs, eager), (*want, want[0])):
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_two_streams_of_one_handle():
    import linear_cross_entropy_token_gb300 as f
    sets = [inputs(s, N=700, V=9000) for s in (3, 4)]
    want = [run_all(f, *s, False) for s in sets]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                outs[i].append(run_all(f, *sets[i], False))
    torch.cuda.synchronize()
    for i in (0, 1):
        for got in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
def test_handles_of_every_tile_shape(cta):
    """The head's operators pick their own tiles."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, ids, z, a = inputs(8)
    h = f.FLCE("bf16", 0, cta=cta, dlogits_mode="slabs" if cta == "wide" else "auto")
    want, got = f.token_logprobs(x, W, t), f.token_logprobs(x, W, t, handle=h)
    assert torch.equal(want.logprobs, got.logprobs)
    for u, v in zip(f.distill(x, W, ids, z), f.distill(x, W, ids, z, handle=h)):
        assert torch.equal(u, v)
    with pytest.raises(ValueError):
        f.token_logprobs(x.float(), W.float(), t, handle=h)


def test_tokens_out_of_range_in_a_batch():
    """Beyond 256 rows, where those that do not count are left out: the others' results stand."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, ids, z, a = inputs(9)
    t[5], t[300] = 2500, -3
    r = f.token_logprobs(x, W, t)
    with pytest.raises(f.FlceError):
        f.async_status()
    dx, dW = f.token_logprobs_backward(r, x, W, t, a, a)
    with pytest.raises(f.FlceError):
        f.async_status()
    f.async_status()
    good = t.clone()
    good[5] = good[300] = -100
    rg = f.token_logprobs(x, W, good)
    gx, gW = f.token_logprobs_backward(rg, x, W, good, a, a)
    assert r.logprobs[[5, 300]].isnan().all() and (dx[[5, 300]] == 0).all()
    same = torch.ones(400, dtype=torch.bool, device="cuda")
    same[5] = same[300] = False
    assert torch.equal(r.logprobs[same], rg.logprobs[same]) and torch.equal(dx[same], gx[same])
    # dW sums the same rows, two zero rows among them
    assert (dW.double() - gW.double()).norm() <= 2.0 ** -8 * gW.double().norm()


def test_errors_are_told_once_and_to_their_own():
    """A bad token does not look like an update's wait that ran out."""
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _, _, _ = inputs(10)
    t[0] = 9999999
    f.token_logprobs(x, W, t)
    torch.cuda.synchronize()
    f.muon_update([torch.randn(40, 60, device="cuda")])
    with pytest.raises(f.FlceError) as e:
        f.async_status()
    assert e.value.status == 4
    f.async_status()


@pytest.mark.parametrize("temperature", [1e-4, 1e4])
def test_extreme_temperatures(temperature):
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _ = make_head(40, 64, 3000, "bf16", seed=11)
    ref = Reference(x, W, temperature)
    r = f.token_logprobs(x, W, t, temperature=temperature, top=20)
    ids, lp = ref.top(20)
    assert torch.equal(r.top_ids, ids)
    want = ref.lp.gather(1, t[:, None])[:, 0]
    err = 2 * ref.sum_error() + 4e-6
    assert ((r.logprobs - want).abs() <= err + 4e-7 * want.abs()).all()
    assert ((r.top_logprobs - lp).abs() <= err[:, None] + 4e-7 * lp.abs()).all()


def test_c_entries_refuse():
    import linear_cross_entropy_token_gb300 as f
    from linear_cross_entropy_token_gb300 import flce
    N, H, V = 20, 64, 300
    x, W, t, _ = make_head(N, H, V, "bf16")
    h = f.FLCE("bf16", 0)
    lib = h.lib
    out = torch.empty(8 * N, device="cuda")
    top = torch.empty(2 * N, dtype=torch.int64, device="cuda")
    grads = torch.empty(N * H + V * H + 8, dtype=torch.bfloat16, device="cuda")
    p = out.data_ptr()
    good = dict(x=x.data_ptr(), W=W.data_ptr(), t=t.data_ptr(), N=N, H=H, V=V, ignore_index=-100, temperature=1.0, top=2,
                reserved=0, logprobs=p, entropy=p + 4 * N, stats=p + 8 * N, top_logprobs=p + 16 * N, top_ids=top.data_ptr(),
                kept=None)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def args(**kw):
        return ctypes.byref(flce.LogprobsArgs(**{**good, **kw}))

    def forward(workspace=ws.data_ptr(), size=64 << 20, **kw):
        return lib.flce_logprobs_forward(h.h, args(**kw), workspace, size, None)

    def backward(dx=grads.data_ptr(), dW=grads.data_ptr() + 2 * N * H, code=0, workspace=ws.data_ptr(), size=64 << 20, d=None, **kw):
        return lib.flce_logprobs_backward(h.h, args(**kw), d, None, dx, dW, code, workspace, size, None)

    assert forward() == 0 and backward() == 0 and forward(t=None, logprobs=None) == 0 and backward(dx=None) == 0
    need = lib.flce_logprobs_workspace_bytes(h.h, args(), 0, -1)
    assert forward(size=need) == 0 and forward(size=need - 1) == 3 and forward(workspace=None) == 3
    assert forward(workspace=ws.data_ptr() + 16) == 3
    assert lib.flce_logprobs_forward(h.h, None, ws.data_ptr(), 64 << 20, None) == 1
    for kw in (dict(N=-1), dict(H=0), dict(V=0), dict(H=60), dict(top=-1), dict(top=65), dict(temperature=0.0),
               dict(temperature=math.nan), dict(temperature=math.inf), dict(x=None), dict(W=None), dict(logprobs=None),
               dict(entropy=None), dict(stats=None), dict(top_ids=None), dict(top_logprobs=None), dict(x=x.data_ptr() + 2),
               dict(t=t.data_ptr() + 4), dict(stats=p + 4), dict(entropy=p + 2), dict(kept=ws.data_ptr() + 8),
               dict(N=1 << 31), dict(V=1, top=2)):
        assert forward(**kw) == 1, kw
    for kw in (dict(t=None), dict(dx=grads.data_ptr() + 2), dict(dW=grads.data_ptr() + 4), dict(d=p + 2), dict(stats=None)):
        assert backward(**kw) == 1, kw
    assert backward(code=2) == 2 and backward(code=7) == 2 and backward(size=1 << 10) == 3
    z = torch.zeros(N, 3, device="cuda")
    ids = torch.zeros(N, 3, dtype=torch.int64, device="cuda")
    dgood = dict(x=x.data_ptr(), W=W.data_ptr(), ids=ids.data_ptr(), logits=z.data_ptr(), N=N, H=H, V=V, K=3, ld_ids=3,
                 ld_logits=3, logits_dtype=1, dw_dtype=0, temperature=1.0, loss=p, token_loss=p + 4, dx=grads.data_ptr(),
                 dW=grads.data_ptr() + 2 * N * H)

    def distill(size=64 << 20, **kw):
        return lib.flce_distill(h.h, ctypes.byref(flce.DistillArgs(**{**dgood, **kw})), ws.data_ptr(), size, None)

    assert distill() == 0 and distill(dx=None, dW=None) == 0
    for kw in (dict(K=0), dict(K=257, ld_ids=257, ld_logits=257), dict(ld_ids=2), dict(ld_logits=2), dict(loss=None),
               dict(token_loss=None), dict(ids=None), dict(logits=None), dict(ids=ids.data_ptr() + 4),
               dict(logits=z.data_ptr() + 2), dict(temperature=-1.0), dict(H=12)):
        assert distill(**kw) == 1, kw
    assert distill(logits_dtype=5) == 2 and distill(dw_dtype=2) == 2 and distill(size=256) == 3
    assert lib.flce_distill_workspace_bytes(h.h, None) == 0
    small = f.FLCE("bf16", 0, hbm_budget_bytes=1 << 20)
    big = torch.zeros(200000, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(f.FlceError) as e:
        f.token_logprobs(x.repeat(20, 1), big, t.repeat(20), handle=small)
    assert e.value.status == 3
    torch.cuda.synchronize()


def test_launches_are_counted_and_profiled():
    import linear_cross_entropy_token_gb300 as f
    x, W, t, ids, z, a = inputs(12)
    h = f.FLCE("bf16", 0)
    f.token_logprobs_backward(f.token_logprobs(x, W, t, handle=h), x, W, t, a, handle=h)
    assert h.launch_count() >= 6
    h.set_profiling(True)
    f.token_logprobs_backward(f.token_logprobs(x, W, t, handle=h), x, W, t, a, handle=h)
    f.distill(x, W, ids, z, handle=h)
    p = h.profile()
    assert {"score_stats", "score_rows", "score_gradient", "score_backward", "distill_rows"} <= set(p)
    assert all(v["total_ms"] > 0 for v in p.values())
