"""What a caller may change between the routing's forward and its backward, and
what autograd must notice."""
import pytest
import torch

from test_gpu_route import make

pytestmark = pytest.mark.gpu


def _routed(N=400, E=24, k=3):
    from linear_cross_entropy_token_gb300.autograd import route
    z, g = make(N, E, "fp32", 7)
    zc = z.cuda().requires_grad_()
    valid = (torch.rand(N, generator=g) > 0.2).cuda()
    offsets = torch.tensor([0, 100, 250, N], device="cuda")
    out = route(zc, k, valid, offsets)
    mix = torch.randn(N, k, generator=g).cuda()
    return zc, valid, offsets, out, lambda: ((out[0] * mix).sum() + 0.7 * out[3] + 0.3 * out[4]).backward()


def test_counts_and_valid_may_change_before_the_backward():
    """Neither is read by the backward: counts are summed over ranks and steps in place, a mask is a buffer
    that the next batch fills."""
    zc, _, _, _, backward = _routed()
    backward()
    want = zc.grad
    zc, valid, _, out, backward = _routed()
    out[2].mul_(8)
    valid.zero_()
    backward()
    assert torch.equal(zc.grad, want)


@pytest.mark.parametrize("which", ["weights", "experts", "offsets"])
def test_what_the_backward_reads_may_not(which):
    zc, _, offsets, out, backward = _routed()
    with torch.no_grad():
        {"weights": out[0].detach(), "experts": out[1], "offsets": offsets}[which].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        backward()
