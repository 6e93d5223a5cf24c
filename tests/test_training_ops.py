"""Refusals and host-side logic of the training-step operators (no GPU)."""
import ctypes

import pytest
import torch

from linear_cross_entropy_token_gb300 import Muon, flce, muon_update, orthogonalize, route
from linear_cross_entropy_token_gb300.muon import _coefficients, check_muon_tensors, workspace_bytes
from linear_cross_entropy_token_gb300.routing import check_route_tensors


def test_route_accepts():
    z = torch.zeros(6, 8)
    check_route_tensors(z, 2, None, None)
    check_route_tensors(z.half(), 8, torch.ones(6, dtype=torch.bool), torch.tensor([0, 2, 6]))
    check_route_tensors(torch.zeros(6, 20)[:, 3:11], 2, None, None)
    check_route_tensors(torch.zeros(0, 8), 1, None, None)
    check_route_tensors(torch.zeros(1, 8).expand(1, 8), 1, None, None)


@pytest.mark.parametrize("case", ["1d", "dtype", "no_experts", "too_many", "transposed", "expanded", "k0", "k_over_e",
                                  "k_over_max", "valid_shape", "valid_dtype", "valid_strided", "valid_device",
                                  "offsets_2d", "offsets_short", "offsets_dtype", "offsets_device"])
def test_route_refuses(case):
    z, k, valid, off = torch.zeros(6, 8), 2, None, None
    if case == "1d":
        z = torch.zeros(8)
    elif case == "dtype":
        z = z.double()
    elif case == "no_experts":
        z = torch.zeros(6, 0)
    elif case == "too_many":
        z = torch.zeros(2, 1025)
    elif case == "transposed":
        z = torch.zeros(8, 6).t()
    elif case == "expanded":
        z = torch.zeros(1, 8).expand(6, 8)
    elif case == "k0":
        k = 0
    elif case == "k_over_e":
        k = 9
    elif case == "k_over_max":
        z, k = torch.zeros(6, 64), 33
    elif case == "valid_shape":
        valid = torch.ones(5, dtype=torch.bool)
    elif case == "valid_dtype":
        valid = torch.ones(6)
    elif case == "valid_strided":
        valid = torch.ones(12, dtype=torch.bool)[::2]
    elif case == "valid_device":
        valid = torch.ones(6, dtype=torch.bool, device="meta")
    elif case == "offsets_2d":
        off = torch.zeros(2, 2, dtype=torch.int64)
    elif case == "offsets_short":
        off = torch.zeros(1, dtype=torch.int64)
    elif case == "offsets_dtype":
        off = torch.zeros(3, dtype=torch.int32)
    elif case == "offsets_device":
        off = torch.zeros(3, dtype=torch.int64, device="meta")
    with pytest.raises(ValueError):
        check_route_tensors(z, k, valid, off)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        route(torch.zeros(6, 8), 2)
    with pytest.raises(ValueError):
        orthogonalize(torch.zeros(6, 8))
    with pytest.raises(ValueError):
        muon_update([torch.zeros(6, 8)])


def test_muon_accepts():
    g = [torch.zeros(4, 6), torch.zeros(4, 9)[:, 1:7]]
    check_muon_tensors(g, [torch.zeros(4, 6) for _ in g], [torch.zeros(4, 6).bfloat16() for _ in g], None)
    check_muon_tensors([torch.zeros(4, 6).bfloat16()], None, None, [torch.zeros(4, 6)])
    assert muon_update([]) == []


@pytest.mark.parametrize("case", ["1d", "empty", "shapes", "dtypes", "grad_dtype", "momentum_dtype", "weight_dtype",
                                  "momentum_count", "transposed", "expanded", "device", "twice", "shared"])
def test_muon_refuses(case):
    g, m, w = [torch.zeros(4, 6), torch.zeros(4, 6)], [torch.zeros(4, 6), torch.zeros(4, 6)], None
    if case == "1d":
        g = [torch.zeros(4)]
    elif case == "empty":
        g, m = [torch.zeros(0, 6)], None
    elif case == "shapes":
        g[1] = torch.zeros(6, 4)
    elif case == "dtypes":
        g[1] = g[1].bfloat16()
    elif case == "grad_dtype":
        g = [t.half() for t in g]
    elif case == "momentum_dtype":
        m = [t.bfloat16() for t in m]
    elif case == "weight_dtype":
        w = [torch.zeros(4, 6).half() for _ in g]
    elif case == "momentum_count":
        m = m[:1]
    elif case == "transposed":
        m[1] = torch.zeros(6, 4).t()
    elif case == "expanded":
        g[1] = torch.zeros(1, 6).expand(4, 6)
    elif case == "device":
        m[1] = torch.zeros(4, 6, device="meta")
    elif case == "twice":
        m[1] = m[0]
    elif case == "shared":
        w = [m[0], torch.zeros(4, 6)]
    with pytest.raises(ValueError):
        check_muon_tensors(g, m, w, None)


def test_coefficients_and_options():
    assert _coefficients(None, 5) is None
    assert len(_coefficients((1.5, -0.5, 0.0), 4)) == 12
    for bad, steps in (((1.0, 2.0), 5), ([(1.0, 2.0, 3.0)] * 2, 3), (None, 0), (None, 33)):
        with pytest.raises(ValueError):
            _coefficients(bad, steps)
    p = torch.nn.Parameter(torch.zeros(4, 6))
    for kw in (dict(lr=-1.0), dict(beta=1.5), dict(scale="other"), dict(steps=0)):
        with pytest.raises(ValueError):
            Muon([p], **kw)
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(4))])
    with pytest.raises(ValueError):
        muon_update([torch.zeros(4, 6)], None, [torch.zeros(4, 6)], updates=[torch.zeros(4, 6)])


def test_workspaces_and_null_handles():
    lib = flce.load()
    one = workspace_bytes(1024, 4096)
    # X in three fp16 buffers, A and B: 3 m n + 2 m^2 halves; and the splits of X Xt: up to seven
    # fp32 sums of A, at most 40 MiB
    assert 0 <= one - 2 * (3 * 1024 * 4096 + 2 * 1024 * 1024) - 7 * 4 * 1024 * 1024 <= 16384
    assert workspace_bytes(4096, 1024) == one
    assert workspace_bytes(1024, 4096, 10) > 10 * 2 * (3 * 1024 * 4096 + 2 * 1024 * 1024)
    assert workspace_bytes(1024, 4096, 10000) <= 2 << 30
    assert workspace_bytes(65536, 65536) > 0
    for bad in ((0, 4, 1), (4, 0, 1), (65537, 4, 1), (4, 4, 0), (4, 4, -1)):
        assert workspace_bytes(*bad) == 0
    assert lib.flce_route_workspace_bytes(None, 10, 8, 1) == 0
    a, b = flce.RouteArgs(), flce.MuonArgs()
    assert lib.flce_route_forward(None, ctypes.byref(a), None, 0, None) == 1
    assert lib.flce_route_backward(None, ctypes.byref(a), None, None, None, None, 0, None) == 1
    assert lib.flce_muon_update(None, ctypes.byref(b), None, 0, None, 0, None) == 1
