"""Heads that mask tokens: a column of x that is 1 and of W that holds -inf (or the
type's lowest value) gives those tokens probability 0, in whole 64-column groups
too. Against the formulas in 64 bits over the other tokens."""
import math

import pytest
import torch

from scoring_testing import DT, Reference, check_gradients, kept_distance, make_head
from test_gpu_distill import make_teacher, reference

pytestmark = pytest.mark.gpu

V = 1100  # the last group is ragged


def masked_head(N, H, dtype):
    x, W, _, g = make_head(N, H, V, dtype, seed=N)
    x[:, -1] = 1
    W[:, -1] = 0
    hidden = torch.zeros(V, dtype=torch.bool, device="cuda")
    for a, b in ((64, 192), (200, 201), (510, 514), (700, 760), (1088, V)):
        hidden[a:b] = True
    lowest = torch.zeros_like(hidden)
    lowest[260:330] = True
    W[hidden, -1] = -math.inf
    W[lowest, -1] = torch.finfo(DT[dtype]).min
    keep = ~(hidden | lowest)
    which = keep.nonzero()[:, 0]
    t = which[torch.randint(0, len(which), (N,), generator=g).cuda()]
    return x, W, t, g, keep, which, hidden


@pytest.mark.parametrize("N,H,dtype", [(40, 64, "bf16"), (200, 136, "bf16"), (300, 64, "bf16"), (40, 64, "fp32"), (9, 33, "fp32")])
@pytest.mark.parametrize("keep_logits", [False, True])
def test_scoring(N, H, dtype, keep_logits):
    import linear_cross_entropy_token_gb300 as f
    x, W, t, g, keep, which, hidden = masked_head(N, H, dtype)
    ref = Reference(x, W[keep])
    live = (torch.rand(N, generator=g) < 0.7).cuda()
    live[1] = True
    tokens = torch.where(live, t, -100)
    tokens[1] = 70  # masked
    r = f.token_logprobs(x, W, tokens, top=12, keep_logits=keep_logits)
    err = 2 * ref.sum_error() + 4e-6
    want = torch.log_softmax(x.double() @ W.double().T, 1).gather(1, t[:, None])[:, 0]
    known = live.clone()
    known[1] = False
    assert ((r.logprobs - want).abs() <= err + 2e-7 * want.abs())[known].all() and r.logprobs[1].item() == -math.inf
    spread = (ref.p * (ref.lp + ref.entropy[:, None]).abs()).sum(1)
    assert ((r.entropy - ref.entropy).abs() <= err * (1 + spread) + 1e-6 * ref.entropy)[live].all()
    ids, lp = ref.top(12)
    assert torch.equal(r.top_ids[live], which[ids][live])
    assert ((r.top_logprobs - lp).abs() <= err[:, None] + 2e-7 * lp.abs())[live].all()
    da, de = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    dx, dW = f.token_logprobs_backward(r, x, W, tokens, d_logprobs=da, d_entropy=de, dW=torch.empty(V, H, device="cuda"))
    # the masked token's own entry is g, of a column whose other entries are 0
    place = torch.zeros(V, dtype=torch.int64, device="cuda")
    place[which] = torch.arange(len(which), device="cuda")
    d = ref.d_scores(place[t], da.double(), de.double())
    d[1] = ref.d_scores(place[t], torch.zeros(N, device="cuda", dtype=torch.float64), de.double())[1]
    d[1] -= ref.p[1] * da[1].double()
    d[~live] = 0
    full = x.double() @ W.double().T
    y = kept_distance(full, 1 / math.log(2))[:, keep] if keep_logits and dtype == "bf16" else None
    rows = torch.where(live[:, None], x, 0)
    some = known.nonzero()[:, 0]  # the masked token's row of W is -inf times its entry in one column alone
    check_gradients(dx[some, :-1], None, d[some], rows[some, :-1], W[keep][:, :-1], y[some] if y is not None else None, dtype)
    check_gradients(None, dW[keep], d, rows, W[keep], y, dtype)
    rest = ~keep
    rest[70] = False
    assert (dW[rest] == 0).all()
    assert ((dW[70].double() - da[1].double() * x[1].double()).abs() <= 2.0 ** -8 * 1.02 * (da[1] * x[1]).abs().double()).all()


@pytest.mark.parametrize("N,H,dtype", [(40, 64, "bf16"), (300, 136, "bf16"), (40, 64, "fp32")])
def test_distillation(N, H, dtype):
    import linear_cross_entropy_token_gb300 as f
    x, W, _, g, keep, which, hidden = masked_head(N, H, dtype)
    ids, logits = make_teacher(N, 20, len(which), g)
    ids[::7] = -1
    want, d, live, ref = reference(x, W[keep], ids, logits, 1.5)
    given = torch.where(ids >= 0, which[ids.clamp(min=0)], -1)
    loss, dx, dW = f.distill(x, W, given, logits, temperature=1.5)
    tol = 1.5 ** 2 * (2 * ref.sum_error().max().item() + 4e-6) + 1e-6 * abs(want.item())
    assert abs(loss.item() - want.item()) <= tol
    y = kept_distance(x.double() @ W.double().T, 1 / (1.5 * math.log(2)))[:, keep] if dtype == "bf16" else None
    rows = torch.where(live[:, None], x, 0)
    some = live.nonzero()[:, 0]
    check_gradients(dx[some, :-1], None, d[some], rows[some, :-1], W[keep][:, :-1], y[some] if y is not None else None, dtype)
    check_gradients(None, dW[keep], d, rows, W[keep], y, dtype)
    assert (dW[~keep] == 0).all()
    # a teacher's entry that the head masks costs infinitely much
    given[3, 0] = 70
    assert f.distill(x, W, given, logits, temperature=1.5, backward=False)[0].item() == math.inf


@pytest.mark.parametrize("V", [70, 8000, 50000])
@pytest.mark.parametrize("N,dtype", [(3, "bf16"), (70, "bf16"), (3, "fp32")])
def test_fewer_tokens_than_alternatives(V, N, dtype):
    import linear_cross_entropy_token_gb300 as f
    x, W, _, _ = make_head(N, 64, V, dtype)
    x[:, -1] = 1
    W[:, -1] = -math.inf
    left = torch.tensor([2, 3, 40, 65, 69], device="cuda")
    W[left, -1] = 0
    r = f.token_logprobs(x, W, None, top=8)
    ref = Reference(x, W[left])
    ids, lp = ref.top(5)
    assert torch.equal(r.top_ids[:, :5], left[ids])
    assert ((r.top_logprobs[:, :5] - lp).abs() <= 2 * ref.sum_error()[:, None] + 4e-6 + 2e-7 * lp.abs()).all()
    assert (r.top_logprobs[:, 5:] == -math.inf).all()
    assert torch.equal(r.top_ids[:, 5:], torch.tensor([[0, 1, 4]], device="cuda").expand(N, 3))


def test_rows_without_any_token_are_nan():
    import linear_cross_entropy_token_gb300 as f
    x, W, t, _ = make_head(80, 64, 200, "bf16")
    x[:, -1] = 1
    x[5:, -1] = 0.0
    W[:, -1] = 0
    want = f.token_logprobs(x, W, t, top=3)
    W[:, -1] = torch.finfo(torch.bfloat16).min
    r = f.token_logprobs(x, W, t, top=3)
    assert torch.equal(r.logprobs[5:], want.logprobs[5:]) and torch.equal(r.top_ids[5:], want.top_ids[5:])
    x[:5, -1] = 1e30
    r = f.token_logprobs(x, W, t, top=3)
    assert r.logprobs[:5].isnan().all() and ((r.top_ids >= 0) & (r.top_ids < 200)).all()
    assert torch.equal(r.logprobs[5:], want.logprobs[5:])


def test_gradients_may_not_overwrite_what_is_read():
    import linear_cross_entropy_token_gb300 as f
    both = torch.zeros(96, 64, dtype=torch.float32, device="cuda")
    x, W = both[:32], torch.randn(96, 64, device="cuda")
    t = torch.zeros(32, dtype=torch.int64, device="cuda")
    r = f.token_logprobs(x, W, t)
    r.logprobs = both[40:].reshape(-1)[:32]
    with pytest.raises(ValueError, match="share"):
        f.token_logprobs_backward(r, x, W, t, dx=both[30:62], dW=None)
    with pytest.raises(ValueError, match="share"):
        f.token_logprobs_backward(r, x, W, t, dx=both[39:71], dW=None)
    wide = torch.zeros(32, 8, device="cuda")
    with pytest.raises(ValueError, match="share"):
        f.distill(x, W, torch.zeros(32, 2, dtype=torch.int64, device="cuda"), both[64:].reshape(-1)[: 32 * 64].view(32, 64)[:, 4:6],
                  dx=both[64:96])
    f.distill(x, W, torch.zeros(32, 2, dtype=torch.int64, device="cuda"), wide[:, 4:6], dx=both[64:96])
