"""A device-side wait of the update that runs out: the kernel ends by itself, the
host is told, and the next update is right. Made by asking for one finished tile
more than there are, each wait limited to 20 ms; no GPU fault is involved."""
import ctypes

import pytest
import torch

from test_gpu_muon import ORTHO, gaussian, newton_schulz, rel

pytestmark = pytest.mark.gpu

TIMEOUT = 5


def _run_out(h, rows, cols, count=1, timeout_us=20000):
    """The check's call on matrices of its own; returns its status."""
    from linear_cross_entropy_token_gb300 import flce
    g = [torch.randn(rows, cols, device="cuda") for _ in range(count)]
    u = [torch.empty(rows, cols, device="cuda") for _ in range(count)]
    a = flce.MuonArgs(rows, cols, 1, 1, 1, 1, 5, 0, None, 0.95, 1e-7, 1.0, 0.0, 0.0)
    m = (flce.MuonMatrix * count)()
    for i in range(count):
        m[i].grad, m[i].update, m[i].ld_grad, m[i].ld_update = g[i].data_ptr(), u[i].data_ptr(), cols, cols
    need = h.lib.flce_muon_workspace_bytes(rows, cols, count)
    ws = torch.empty(need + 1024, dtype=torch.uint8, device="cuda")
    st = h.lib.flce_check_muon_timeout(h.h, ctypes.byref(a), m, count, (ws.data_ptr() + 1023) // 1024 * 1024, need,
                                       timeout_us, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("rows,cols,count", [(200, 300, 1), (1500, 700, 2), (256, 6000, 1)])
@pytest.mark.parametrize("cta", ["single", "pair", "wide"])
def test_a_wait_that_runs_out_is_told(cta, rows, cols, count):
    from linear_cross_entropy_token_gb300 import FLCE, FlceError, muon_update, orthogonalize
    h = FLCE("bf16", 0, cta=cta)
    try:
        # by the handle's status, once
        assert _run_out(h, rows, cols, count) == 0
        with pytest.raises(FlceError) as e:
            h.async_status()
        assert e.value.status == TIMEOUT
        h.async_status()
        # or by the next update, which does nothing itself
        assert _run_out(h, rows, cols, count) == 0
        g = gaussian(rows, cols, 1)
        w = torch.full((rows, cols), 3.0, device="cuda")
        with pytest.raises(FlceError) as e:
            muon_update([g.cuda()], None, [w], lr=0.1, handle=h)
        assert e.value.status == TIMEOUT and "earlier update" in str(e.value)
        torch.cuda.synchronize()
        assert bool((w == 3.0).all())
        # and then all is well
        assert rel(orthogonalize(g.cuda(), dtype=torch.float32, handle=h), newton_schulz(g)) <= ORTHO
        h.async_status()
        assert _run_out(h, rows, cols, count, timeout_us=999) == 1
        h.async_status()
    finally:
        h.close()


def test_updates_without_a_handle():
    """Muon.step and muon_update tell by async_status of the package, and by the next step."""
    from linear_cross_entropy_token_gb300 import FlceError, Muon, async_status, flce
    p = torch.nn.Parameter(torch.randn(200, 300, device="cuda"))
    p.grad = torch.randn(200, 300, device="cuda")
    opt = Muon([p])
    opt.step()
    async_status()
    async_status("cuda:0")
    h = flce.cached_handle(0)
    _run_out(h, 200, 300)
    with pytest.raises(FlceError) as e:
        async_status()
    assert e.value.status == TIMEOUT
    _run_out(h, 200, 300)
    before = p.detach().clone()
    with pytest.raises(FlceError):
        opt.step()
    torch.cuda.synchronize()
    assert torch.equal(p.detach(), before)
    opt.step()
    async_status()
    assert not torch.equal(p.detach(), before)
