"""The training-step operators together, as examples/train_moe_lm.py runs them,
and what their entry points refuse on a device."""
import ctypes
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_learns():
    import train_moe_lm
    history = train_moe_lm.train(steps=25, log=lambda *_: None)
    first, last = history[0], history[-1]
    assert abs(first[0] - math.log(1000)) < 1.5          # an untrained head
    assert last[0] < first[0] - 1.0
    # every live token fills its two slots; the balance loss is 1 for an even load, 8 for one expert
    assert all(2 * (4096 - 8) <= slots <= 2 * (4096 - 1) for _, _, slots in history)
    assert all(0.9 <= balance <= 2.0 for _, balance, _ in history)


def test_refusals_of_muon_update():
    from linear_cross_entropy_token_gb300 import FlceError, flce, muon_update
    g = [torch.randn(200, 300, device="cuda")]
    for kw in (dict(coefficients=(10.0, 0.0, 0.0)), dict(coefficients=(3.4445, -4.7750, math.nan)), dict(beta=1.5),
               dict(beta=-0.1), dict(eps=-1.0), dict(scale=math.inf), dict(lr=math.nan)):
        with pytest.raises(FlceError) as e:
            muon_update(g, **kw)
        assert e.value.status == 1, kw
    # a first step that keeps X in range may have any coefficients that do
    muon_update(g, steps=1, coefficients=(3.0, 0.0, 0.0))
    h = flce.cached_handle(0)
    a = flce.MuonArgs(200, 300, 1, 1, 1, 1, 5, 0, None, 0.95, 1e-7, 1.0, 0.0, 0.0)
    u = torch.empty(200, 300, device="cuda")
    m = (flce.MuonMatrix * 1)()
    m[0].grad, m[0].update, m[0].ld_grad, m[0].ld_update = g[0].data_ptr(), u.data_ptr(), 300, 300
    need = h.lib.flce_muon_workspace_bytes(200, 300, 1)
    ws = torch.empty(need + 1024, dtype=torch.uint8, device="cuda")
    base = (ws.data_ptr() + 1023) // 1024 * 1024

    def call(count=1, workspace=base, size=need):
        return h.lib.flce_muon_update(h.h, ctypes.byref(a), m, count, workspace, size, None)

    assert call() == 0 and call(count=0) == 0
    assert call(size=need - 1) == 3 and call(workspace=None) == 3 and call(workspace=base + 16) == 3
    assert call(count=-1) == 1
    for field, bad, status in (("rows", 0, 1), ("cols", 70000, 1), ("steps", 0, 1), ("steps", 33, 1), ("grad_dtype", 2, 2),
                               ("update_dtype", 7, 2)):
        kept = getattr(a, field)
        setattr(a, field, bad)
        assert call() == status, field
        setattr(a, field, kept)
    for field, bad in (("grad", None), ("update", None), ("ld_grad", 299), ("ld_update", 299), ("grad", g[0].data_ptr() + 2)):
        kept = getattr(m[0], field)
        setattr(m[0], field, bad)
        assert call() == 1, field
        setattr(m[0], field, kept)
    assert call() == 0
    torch.cuda.synchronize()


def test_refusals_of_route():
    from linear_cross_entropy_token_gb300 import flce, route, route_backward
    h = flce.cached_handle(0)
    z = torch.randn(50, 16, device="cuda")
    r = route(z, 3)
    need = h.lib.flce_route_workspace_bytes(h.h, 50, 16, 1)
    assert need > 0
    for bad in ((-1, 16, 1), (50, 0, 1), (50, 1025, 1), (50, 16, 0)):
        assert h.lib.flce_route_workspace_bytes(h.h, *bad) == 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = r.bind(z, 50, 16, 16, flce.DTYPE_FP32)
    out = torch.empty_like(z)

    def call(workspace=ws.data_ptr(), size=need):
        return h.lib.flce_route_forward(h.h, ctypes.byref(a), workspace, size, None)

    def back(d=out.data_ptr(), ld=16):
        return h.lib.flce_route_backward(h.h, ctypes.byref(a), None, None, None, d, ld, None)

    assert call() == 0 and back() == 0
    assert call(size=need - 1) == 3 and call(workspace=None) == 3 and call(workspace=ws.data_ptr() + 4) == 3
    assert back(d=None) == 1 and back(ld=15) == 1 and back(d=out.data_ptr() + 1) == 1
    for field, bad, status in (("dtype", 3, 2), ("N", -1, 1), ("E", 0, 1), ("E", 2000, 1), ("k", 0, 1), ("k", 17, 1),
                               ("ld", 15, 1), ("documents", 0, 1), ("documents", 2, 1), ("logits", None, 1),
                               ("weights", None, 1), ("counts", None, 1), ("stats", a.stats + 4, 1),
                               ("logits", z.data_ptr() + 2, 1)):
        kept = getattr(a, field)
        setattr(a, field, bad)
        assert call() == status and back() == status, field
        setattr(a, field, kept)
    assert call() == 0
    with pytest.raises(ValueError):
        route_backward(r, z[:, :8].contiguous())
    with pytest.raises(ValueError):
        route_backward(r, z, d_weights=torch.zeros(50, 2, device="cuda"))
    with pytest.raises(ValueError):
        route_backward(r, z, d_balance=torch.zeros(2, device="cuda"))
    torch.cuda.synchronize()
