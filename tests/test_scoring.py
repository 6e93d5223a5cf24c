"""Refusals and host-side checks of the head's scoring and distillation calls (no GPU)."""
import ctypes
import math

import pytest
import torch

from linear_cross_entropy_token_gb300 import build as flce_build
from linear_cross_entropy_token_gb300 import distill, flce, token_logprobs, token_logprobs_backward
from linear_cross_entropy_token_gb300.scoring import (TokenLogprobs, _gradient, _vector, check_distill_tensors,
                                                       check_score_tensors)


def head(N=6, H=16, V=20, dtype=torch.bfloat16):
    return torch.zeros(N, H, dtype=dtype), torch.zeros(V, H, dtype=dtype), torch.zeros(N, dtype=torch.int64)


def test_score_accepts():
    x, W, t = head()
    for args in ((x, W, t, 1.0, 0), (x, W, None, 0.5, 20), (x[:0], W, t[:0], 1, 3), (*head(H=7, dtype=torch.float32), 2.0, 1),
                 (*head(V=100), 1e-3, 64)):
        check_score_tensors(*args)


@pytest.mark.parametrize("case", ["x_1d", "W_1d", "W_cols", "W_dtype", "x_dtype", "t_dtype", "t_shape", "t_2d", "t_device",
                                  "x_strided", "W_strided", "no_vocabulary", "no_columns", "odd_columns", "top_negative",
                                  "top_over_v", "top_over_max", "top_float", "top_bool", "temperature_0", "temperature_negative",
                                  "temperature_nan", "temperature_inf", "no_t_W_cols", "no_t_strided", "no_t_1d"])
def test_score_refuses(case):
    x, W, t = head()
    temperature, top = 1.0, 2
    if case == "x_1d":
        x = x[0]
    elif case == "W_1d":
        W = W[0]
    elif case == "W_cols":
        W = torch.zeros(20, 24, dtype=torch.bfloat16)
    elif case == "W_dtype":
        W = W.float()
    elif case == "x_dtype":
        x, W = x.half(), W.half()
    elif case == "t_dtype":
        t = t.int()
    elif case == "t_shape":
        t = t[:5]
    elif case == "t_2d":
        t = t[:, None]
    elif case == "t_device":
        t = t.to("meta")
    elif case == "x_strided":
        x = torch.zeros(6, 32, dtype=torch.bfloat16)[:, ::2]
    elif case == "W_strided":
        W = torch.zeros(20, 32, dtype=torch.bfloat16)[:, :16]
    elif case == "no_vocabulary":
        W, top = W[:0], 0
    elif case == "no_columns":
        x, W = x[:, :0], W[:, :0]
    elif case == "odd_columns":
        x, W, t = head(H=12)
    elif case == "top_negative":
        top = -1
    elif case == "top_over_v":
        top = 21
    elif case == "top_over_max":
        x, W, t = head(V=100)
        top = 65
    elif case == "top_float":
        top = 2.0
    elif case == "top_bool":
        top = True
    elif case.startswith("temperature"):
        temperature = {"0": 0.0, "negative": -1.0, "nan": math.nan, "inf": math.inf}[case.split("_")[1]]
    elif case == "no_t_W_cols":
        W, t = torch.zeros(20, 24, dtype=torch.bfloat16), None
    elif case == "no_t_strided":
        x, t = torch.zeros(6, 32, dtype=torch.bfloat16)[:, ::2], None
    elif case == "no_t_1d":
        x, t = x[0], None
    with pytest.raises(ValueError):
        check_score_tensors(x, W, t, temperature, top)


def test_distill_accepts():
    x, W, _ = head()
    ids, z = torch.zeros(6, 5, dtype=torch.int64), torch.zeros(6, 9)
    assert check_distill_tensors(x, W, ids, z[:, 2:7], 1.0) == [5, 9]
    assert check_distill_tensors(x, W, ids[:, :1], z[:, ::9], 1.0) == [5, 9]
    assert check_distill_tensors(x[:1], W, ids[:1], z[:1, :5].half(), 3.0) == [5, 5]
    assert check_distill_tensors(x[:0], W, ids[:0], z[:0, :5].bfloat16(), 1.0) == [5, 5]


@pytest.mark.parametrize("case", ["1d", "rows", "shapes", "k0", "k_over_max", "ids_dtype", "logits_dtype", "ids_strided",
                                  "logits_expanded", "ids_device", "logits_device", "temperature"])
def test_distill_refuses(case):
    x, W, _ = head()
    ids, z, temperature = torch.zeros(6, 5, dtype=torch.int64), torch.zeros(6, 5), 1.0
    if case == "1d":
        ids, z = ids[:, 0], z[:, 0]
    elif case == "rows":
        ids, z = ids[:5], z[:5]
    elif case == "shapes":
        z = z[:, :4]
    elif case == "k0":
        ids, z = ids[:, :0], z[:, :0]
    elif case == "k_over_max":
        ids, z = torch.zeros(6, 257, dtype=torch.int64), torch.zeros(6, 257)
    elif case == "ids_dtype":
        ids = ids.int()
    elif case == "logits_dtype":
        z = z.double()
    elif case == "ids_strided":
        ids = torch.zeros(6, 10, dtype=torch.int64)[:, ::2]
    elif case == "logits_expanded":
        z = z[:1].expand(6, 5)
    elif case == "ids_device":
        ids = ids.to("meta")
    elif case == "logits_device":
        z = z.to("meta")
    elif case == "temperature":
        temperature = 0.0
    with pytest.raises(ValueError):
        check_distill_tensors(x, W, ids, z, temperature)


def test_host_tensors_are_refused():
    x, W, t = head()
    with pytest.raises(ValueError):
        token_logprobs(x, W, t)
    r = TokenLogprobs()
    r.temperature = 1.0
    with pytest.raises(ValueError):
        token_logprobs_backward(r, x, W, t)
    with pytest.raises(ValueError):
        token_logprobs_backward(r, x, W, None)
    with pytest.raises(ValueError):
        distill(x, W, torch.zeros(6, 5, dtype=torch.int64), torch.zeros(6, 5))


def test_gradient_tensors():
    W = head()[1]
    both = (torch.bfloat16, torch.float32)
    assert _gradient("dW", None, W, both) is None and _gradient("dW", False, W, both) is None
    new = _gradient("dW", True, W, both)
    assert new.shape == W.shape and new.dtype == W.dtype
    given = torch.zeros(20, 16)
    assert _gradient("dW", given, W, both) is given
    for bad in (torch.zeros(20, 15), torch.zeros(20, 16).double(), torch.zeros(16, 20).t(), torch.zeros(20, 16, device="meta"), 1):
        with pytest.raises(ValueError):
            _gradient("dW", bad, W, both)
    with pytest.raises(ValueError):
        _gradient("dx", torch.zeros(20, 16), W, (torch.bfloat16,))
    flat = torch.zeros(40, 16, dtype=torch.bfloat16)
    assert _gradient("dW", flat[20:], flat[:20], both, (flat[:20], None)).data_ptr() == flat[20:].data_ptr()
    for shared in (flat[:20], flat[19:39]):
        with pytest.raises(ValueError):
            _gradient("dW", flat[:20], W, both, (W, shared))
    for bad in (torch.zeros(5), torch.zeros(6).half(), torch.zeros(12)[::2], torch.zeros(6, device="meta"), torch.zeros(6, 1)):
        with pytest.raises(ValueError):
            _vector("d_logprobs", bad, 6, torch.device("cpu"))


def test_null_handles():
    flce_build.build()
    lib = flce.load()
    a, d = flce.LogprobsArgs(), flce.DistillArgs()
    assert lib.flce_logprobs_forward(None, ctypes.byref(a), None, 0, None) == 1
    assert lib.flce_logprobs_backward(None, ctypes.byref(a), None, None, None, None, 1, None, 0, None) == 1
    assert lib.flce_distill(None, ctypes.byref(d), None, 0, None) == 1
    assert lib.flce_logprobs_kept_bytes(None, 1, 1) == 0
    assert lib.flce_logprobs_workspace_bytes(None, ctypes.byref(a), 0, 0) == 0
    assert lib.flce_distill_workspace_bytes(None, ctypes.byref(d)) == 0
