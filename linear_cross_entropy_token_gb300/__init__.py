"""Fused linear cross-entropy (FLCE) on one GB300 (sm_103a).

The computation lives in libflce.so (C ABI: include/flce.h); this package is
its binding. ``FLCE`` wraps a handle; ``forward_backward`` returns the mean
cross-entropy of x·Wᵀ over non-ignored tokens with dx and dW, without ever
holding the N x V logits. Next to it stand two more parts of a training step:
expert routing with its balance loss (``route``, ``route_backward``) and the
orthogonalised momentum update of weight matrices (``muon_update``,
``orthogonalize``, the optimizer ``Muon``). Two more operators of the head start
from x and W: log probabilities of given tokens with entropy and alternatives
(``token_logprobs``, ``token_logprobs_backward``), and distillation from a
teacher's top logits (``distill``).
"""
from .flce import (FLCE, FlceError, KERNEL_KINDS, async_status, forward_backward, header_functions, load,
                   loss_static, plan)

__all__ = ["FLCE", "FlceError", "KERNEL_KINDS", "Muon", "Routing", "TokenLogprobs", "async_status", "distill",
           "forward_backward", "header_functions", "load", "loss_static", "muon_update", "orthogonalize", "plan",
           "route", "route_backward", "token_logprobs", "token_logprobs_backward"]

# these need torch at import, which the rest of the package does not
_LAZY = {"Muon": "muon", "muon_update": "muon", "orthogonalize": "muon", "Routing": "routing",
         "route": "routing", "route_backward": "routing", "TokenLogprobs": "scoring", "distill": "scoring",
         "token_logprobs": "scoring", "token_logprobs_backward": "scoring"}


def __getattr__(name):
    if name in _LAZY:
        import importlib
        value = getattr(importlib.import_module("." + _LAZY[name], __name__), name)
        globals()[name] = value
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
