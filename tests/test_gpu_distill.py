"""Distillation from a teacher's top logits, against the formulas in 64 bits."""
import math

import pytest
import torch

from scoring_testing import Reference, check_gradients, kept_distance, make_head

pytestmark = pytest.mark.gpu

TEACHER = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp16": torch.float16}


def make_teacher(N, K, V, g, dtype="fp32"):
    ids = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else torch.randint(0, V, (K,), generator=g)
                       for _ in range(N)])
    return ids.cuda(), (torch.randn(N, K, generator=g) * 3).to(TEACHER[dtype]).cuda()


def reference(x, W, ids, logits, tau):
    """loss, d, the rows that count, the 64-bit head."""
    ref = Reference(x, W, tau)
    there = (ids >= 0) & (logits.double() > -math.inf)
    live = there.any(1)
    n = max(int(live.sum()), 1)
    s = torch.where(there, logits.double() / tau, -math.inf)
    q = torch.zeros_like(s)
    q[live] = torch.softmax(s[live], 1)
    at = ids.clamp(min=0)
    terms = torch.where(q > 0, q * (torch.log(q.clamp(min=1e-300)) - ref.lp.gather(1, at)), 0.0)
    target = torch.zeros_like(ref.p).scatter_add(1, at, q)
    d = torch.where(live[:, None], (ref.p - target) * tau / n, 0.0)
    return terms.sum() * tau * tau / n, d, live, ref


def check(x, W, ids, logits, tau=1.0, dtype="bf16", handle=None, xref=None):
    import linear_cross_entropy_token_gb300 as f
    xr = x if xref is None else xref
    want, d, live, ref = reference(xr, W, ids, logits, tau)
    loss, dx, dW = f.distill(x, W, ids, logits, temperature=tau, handle=handle)
    tol = tau * tau * (2 * ref.sum_error().max().item() + 4e-6) + 1e-6 * abs(want.item())
    assert abs(loss.item() - want.item()) <= tol, (loss.item(), want.item(), tol)
    assert abs(f.distill(x, W, ids, logits, temperature=tau, backward=False, handle=handle)[0].item() - loss.item()) <= 1e-6 * (
        1 + abs(loss.item()))
    xz = torch.where(live[:, None], xr, 0)
    check_gradients(dx, dW, d, xz, W, kept_distance(ref.raw, 1 / (tau * math.log(2))) if dtype == "bf16" else None, dtype)
    return loss, dx, dW


@pytest.mark.parametrize("N,H,V,K,dtype,teacher", [
    (1, 64, 64, 1, "bf16", "fp32"), (3, 8, 5, 5, "bf16", "bf16"), (17, 128, 511, 33, "bf16", "fp16"),
    (129, 136, 513, 64, "bf16", "fp32"), (256, 256, 1000, 256, "bf16", "bf16"), (257, 1016, 2049, 7, "bf16", "fp32"),
    (100, 64, 50257, 100, "bf16", "fp16"), (5, 33, 70, 9, "fp32", "fp32"), (64, 128, 4096, 8, "fp32", "bf16"),
    (31, 7, 127, 127, "fp32", "fp16")])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill(N, H, V, K, dtype, teacher, tau):
    x, W, _, g = make_head(N, H, V, dtype, seed=N + K)
    ids, logits = make_teacher(N, K, V, g, teacher)
    check(x, W, ids, logits, tau, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_entries_and_rows_that_do_not_count(dtype):
    x, W, _, g = make_head(200, 64, 700, dtype, seed=2)
    ids, logits = make_teacher(200, 20, 700, g)
    logits[torch.rand(200, 20, generator=g).cuda() < 0.3] = -math.inf
    ids[torch.rand(200, 20, generator=g).cuda() < 0.2] = -1
    ids[logits == -math.inf] = 10 ** 12                   # whatever stands at an entry that does not count
    logits[(ids == -1) & (torch.rand(200, 20, generator=g).cuda() < 0.5)] = math.nan
    ids[::5], logits[::10] = -1, -math.inf
    logits[5::10] = math.inf
    clean_logits = torch.where(ids == -1, -math.inf, logits)
    clean_ids = torch.where(clean_logits == -math.inf, -1, ids)
    full = x.clone()
    dead = (clean_ids == -1).all(1)
    assert 30 < dead.sum() < 100
    x[dead] = math.nan
    import linear_cross_entropy_token_gb300 as f
    got = check(x, W, clean_ids, clean_logits, 1.0, dtype, xref=full)
    raw = f.distill(x, W, ids, logits)
    assert all(torch.equal(a, b) for a, b in zip(got, raw))
    f.async_status()


def test_no_row_counts():
    import linear_cross_entropy_token_gb300 as f
    x, W, _, g = make_head(20, 64, 100, "bf16")
    ids, logits = make_teacher(20, 4, 100, g)
    for i, z in ((torch.full_like(ids, -1), logits), (ids, torch.full_like(logits, -math.inf)), (ids[:0], logits[:0])):
        loss, dx, dW = f.distill(x[:len(i)], W, i, z)
        assert loss.item() == 0 and (dx == 0).all() and (dW == 0).all()


def test_the_lowest_value_of_the_type_counts():
    """A mask of finfo.min is a logit like others: alone it has all of the row's mass."""
    x, W, _, g = make_head(12, 64, 100, "bf16")
    ids, logits = make_teacher(12, 4, 100, g, "bf16")
    low = torch.finfo(torch.bfloat16).min
    logits[:6, 1:] = low
    logits[6:, :] = low
    check(x, W, ids, logits)


def test_entries_that_share_an_id():
    x, W, _, g = make_head(50, 64, 300, "bf16", seed=6)
    ids, logits = make_teacher(50, 12, 300, g)
    ids[:, 5] = ids[:, 0]
    ids[:, 6] = ids[:, 0]
    ids[25:] = ids[25:, :1]
    check(x, W, ids, logits)


def test_strided_rows_chunks_and_parts():
    import linear_cross_entropy_token_gb300 as f
    x, W, _, g = make_head(900, 128, 5000, "bf16", seed=8)
    ids, logits = make_teacher(900, 40, 5000, g, "bf16")
    h = f.FLCE("bf16", 0, hbm_budget_bytes=6 << 20)
    loss, dx, dW = check(x, W, ids[:, 3:17], logits[:, 20:34], 1.5, handle=h)
    args = (x, W, ids[:, 3:17], logits[:, 20:34], 1.5)
    only_x, only_W = f.distill(*args, dW=None, handle=h), f.distill(*args, dx=None, handle=h)
    assert only_x[2] is None and only_W[1] is None and torch.equal(only_x[0], loss)
    out_x, out_W = torch.full_like(x, 9), torch.full((5000, 128), 9.0, device="cuda")
    got = f.distill(*args, dx=out_x, dW=out_W, handle=h)
    assert got[1] is out_x and got[2] is out_W and torch.equal(out_W.bfloat16(), dW) and torch.equal(out_x, dx)
    for a, b in ((only_x[1], dx), (only_W[2], dW)):
        assert (a.double() - b.double()).norm() <= 2.0 ** -8 * b.double().norm()


def test_bad_teachers():
    import linear_cross_entropy_token_gb300 as f
    x, W, _, g = make_head(20, 64, 100, "bf16")
    ids, logits = make_teacher(20, 4, 100, g)
    for bad in (100, -2, 1 << 40):
        wrong = ids.clone()
        wrong[3, 2] = bad
        assert f.distill(x, W, wrong, logits)[0].isnan()
        with pytest.raises(f.FlceError) as e:
            f.async_status()
        assert e.value.status == 4
    f.async_status()
    for value in (math.nan, math.inf):
        wrong = logits.clone()
        wrong[3, 2] = value
        assert f.distill(x, W, ids, wrong)[0].isnan()
    f.async_status()


def test_same_teacher_as_student_is_the_minimum():
    """The student's own top logits: with all of them the divergence and its gradient vanish."""
    import linear_cross_entropy_token_gb300 as f
    x, W, _, _ = make_head(30, 64, 200, "fp32", seed=3)
    z = x.double() @ W.double().T
    ids = torch.arange(200, device="cuda").expand(30, 200).contiguous()
    loss, dx, dW = f.distill(x, W, ids, z.float())
    # log q and log p agree to the steps of numbers of about ten; so does d to those of p, over 30 rows
    assert abs(loss.item()) <= 32 * 2.0 ** -24 * 10
    assert dx.abs().max().item() <= 1e-6 and dW.abs().max().item() <= 1e-6


def test_gradient_against_differences():
    import linear_cross_entropy_token_gb300 as f
    x, W, _, g = make_head(40, 24, 90, "fp32", seed=1, strength=2.0)
    ids, logits = make_teacher(40, 6, 90, g)
    _, dx, dW = f.distill(x, W, ids, logits, 1.5)

    def value(x, W):
        return f.distill(x, W, ids, logits, 1.5, backward=False)[0].double().item()

    for like, grad, move in ((x, dx, lambda e: value(x + e, W)), (W, dW, lambda e: value(x, W + e))):
        v = torch.randn(like.shape, generator=g).cuda()
        step = 3e-2 / v.norm()
        slope = (move(step * v) - move(-step * v)) / (2 * step.item())
        want = (grad.double() * v).sum().item()
        # a loss of about 8 with a few steps of 2^-24, over the step; the third derivative's share
        limit = 8 * 2.0 ** -22 / step.item() + 1e-3 * grad.norm().item() * v.norm().item() / math.sqrt(v.numel())
        assert abs(slope - want) <= limit
