"""The Muon optimizer on the GPU: a step that is refused changes nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _parameters():
    g = torch.Generator().manual_seed(0)
    ps = [torch.nn.Parameter(torch.randn(r, c, generator=g).cuda()) for r, c in ((40, 60), (200, 300), (60, 40))]
    for p in ps:
        p.grad = torch.randn(*p.shape, generator=g).cuda()
    return ps


def _untouched(ps, before, opt):
    for p, kept in zip(ps, before):
        assert torch.equal(p.detach(), kept) and not opt.state.get(p, {}).get("momentum", torch.zeros(1)).any()


@pytest.mark.parametrize("case", ["strides", "broadcast gradient", "coefficients", "lr"])
def test_a_refused_step_changes_nothing(case):
    """Whatever the last group's parameters or options hold, no group before it has been updated."""
    from linear_cross_entropy_token_gb300 import FlceError, Muon
    ps = _parameters()
    if case == "strides":
        ps[2] = torch.nn.Parameter(torch.randn(40, 60, device="cuda").t())
        ps[2].grad = torch.randn(40, 60, device="cuda").t()
    if case == "broadcast gradient":
        ps[2].grad = torch.randn(1, 40, device="cuda").expand(60, 40)
    opt = Muon([{"params": ps[:2]}, {"params": ps[2:]}], lr=0.1)
    if case == "coefficients":
        opt.param_groups[1]["coefficients"] = (10.0, 0.0, 0.0)
    if case == "lr":
        opt.param_groups[1]["lr"] = float("nan")
    before = [p.detach().clone() for p in ps]
    with pytest.raises((ValueError, FlceError)):
        opt.step()
    torch.cuda.synchronize()
    _untouched(ps, before, opt)


def test_tensors_that_only_the_call_holds():
    """An iterator's temporaries live until the launch: their memory, which would hold the workspace, is not
    taken for it (80 matrices go through it in three groups, so later ones would be overwritten)."""
    from linear_cross_entropy_token_gb300 import muon_update
    from linear_cross_entropy_token_gb300.muon import workspace_bytes
    rows, cols, count = 160, 256, 80
    g = torch.randn(count, rows, cols, device="cuda")
    assert workspace_bytes(rows, cols, count) + 1024 < g.numel() * 4
    want = muon_update(list((g * 3).unbind(0)))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = muon_update(t for t in (g * 3).unbind(0))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_step_after_a_refused_one():
    from linear_cross_entropy_token_gb300 import Muon
    ps, qs = _parameters(), _parameters()
    opt, other = Muon(ps, lr=0.1), Muon(qs, lr=0.1)
    kept = ps[1].grad
    ps[1].grad = torch.randn(1, 300, device="cuda").expand(200, 300)
    with pytest.raises(ValueError):
        opt.step()
    ps[1].grad = kept
    opt.step()
    other.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, qs))
