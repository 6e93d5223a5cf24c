"""Autograd wrapper: the fused call as a differentiable loss.

The LM head is the last layer, so its gradients can be produced during the
forward pass. The FLCE page ("Fused Linear Cross-Entropy: LLM 학습 logits
메모리 병목 없애기", section "FLCE의 핵심 아이디어") quotes Liger's source
comment to that effect. The forward here runs the whole fused forward +
backward in the library and keeps dx and dW. The backward only scales them by
the incoming gradient of the (scalar) loss, which is 1 in the usual
`loss.backward()`, and then no arithmetic runs at all. The pattern is the
hand-written forward/backward pair the Unsloth page shows for its fused
kernels ("Unsloth 심층 아키텍처 …", section "소스코드 레벨 아키텍처 구현 패턴").
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import routing, scoring
from .flce import FLCE, _caches

_handles = {}
_caches.append(_handles)


def _handle(device: torch.device, dtype: torch.dtype, dlogits_mode: str = "auto",
            hbm_budget_bytes: int = 0) -> FLCE:
    key = (device.index or 0, dtype, dlogits_mode, hbm_budget_bytes)
    if key not in _handles:
        _handles[key] = FLCE("bf16" if dtype == torch.bfloat16 else "fp32", key[0],
                             hbm_budget_bytes=hbm_budget_bytes, dlogits_mode=dlogits_mode)
    return _handles[key]


class LinearCrossEntropyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, t, ignore_index: int, chunk: int, reduction: str, handle,
                sync_free: bool = False, dlogits_mode: str = "auto", hbm_budget_bytes: int = 0):
        h = handle if handle is not None else _handle(x.device, x.dtype, dlogits_mode, hbm_budget_bytes)
        if reduction not in ("mean", "sum"):
            raise ValueError("reduction must be 'mean' or 'sum'")
        ctx.sync_free = sync_free
        if sync_free:
            # no host synchronisation anywhere: the loss stays on the device
            # (NaN after a device-side error) and the gradients are always
            # scaled by the incoming gradient on the device
            loss, n_valid, dx, dW = h.forward_backward_async(
                x.contiguous(), W.contiguous(), t.contiguous(), ignore_index=ignore_index,
                chunk=chunk)
            scale = n_valid.float() if reduction == "sum" else torch.ones((), device=x.device)
            ctx.save_for_backward(dx, dW, scale)
            return loss * scale
        loss, dx, dW = h.forward_backward(x.contiguous(), W.contiguous(), t.contiguous(),
                                          ignore_index=ignore_index, chunk=chunk)
        scale = 1.0
        if reduction == "sum":
            # the library returns the mean over the n_valid counted tokens
            scale = float((t != ignore_index).sum().item())
        ctx.scale = scale
        ctx.save_for_backward(dx, dW)
        return torch.tensor(loss * scale, dtype=torch.float32, device=x.device)

    @staticmethod
    def backward(ctx, grad_out):
        if ctx.sync_free:
            dx, dW, scale = ctx.saved_tensors
            g = grad_out * scale
            gx = dx * g.to(dx.dtype) if ctx.needs_input_grad[0] else None
            gW = dW * g if ctx.needs_input_grad[1] else None
            return gx, gW, None, None, None, None, None, None, None, None
        dx, dW = ctx.saved_tensors
        g = grad_out * ctx.scale
        if ctx.needs_input_grad[0]:
            gx = dx if (ctx.scale == 1.0 and bool(grad_out == 1)) else dx * g.to(dx.dtype)
        else:
            gx = None
        if ctx.needs_input_grad[1]:
            gW = dW if (ctx.scale == 1.0 and bool(grad_out == 1)) else dW * g
        else:
            gW = None
        return gx, gW, None, None, None, None, None, None, None, None


def linear_cross_entropy(x: torch.Tensor, W: torch.Tensor, t: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean", chunk: int = 0,
                         handle: FLCE = None, sync_free: bool = False, dlogits_mode: str = "auto",
                         hbm_budget_bytes: int = 0) -> torch.Tensor:
    """Cross-entropy of x·Wᵀ against t, fused: the N x V logits never exist.

    x: (N, H) bf16 or fp32 on a GB300; W: (V, H) same dtype; t: (N,) int64.
    Returns a 0-dim fp32 tensor. `loss.backward()` gives x.grad and W.grad;
    W.grad is computed in fp32 and cast by autograd to W's dtype.

    sync_free=True never blocks the host (a step can then be captured in a
    CUDA graph): the loss is NaN after a device-side error, which
    FLCE.async_status() and async_status() report, and the backward always
    scales dx and dW by the incoming gradient (one extra pass over dW). The
    default synchronises once per call, raises on errors at once, and skips
    that pass when the incoming gradient is 1.

    Without a `handle`, one is kept per (device, dtype, dlogits_mode,
    hbm_budget_bytes): dlogits_mode "slabs" with a small budget gives the
    vocabulary-slab backward, whose workspace does not grow with V.
    """
    return LinearCrossEntropyFunction.apply(x, W, t, ignore_index, chunk, reduction, handle,
                                            sync_free, dlogits_mode, hbm_budget_bytes)


class RouteFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, valid, offsets, renormalize, handle):
        r = routing.route(logits, k, valid=valid, offsets=offsets, renormalize=renormalize, handle=handle)
        # the outputs are separate tensors: the losses of r are views of one
        balance, z = r.balance.clone(), r.z.clone()
        ctx.handle, ctx.k, ctx.renormalize = handle, k, renormalize
        # counts and valid are not read by the backward, so callers may change
        # them (counts summed over ranks, a mask's buffer filled again)
        ctx.counts = r.counts
        ctx.save_for_backward(logits, offsets, r.weights, r.experts, r.state)
        ctx.mark_non_differentiable(r.experts, r.counts)
        ctx.set_materialize_grads(False)
        return r.weights, r.experts, r.counts, balance, z

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _d_experts, _d_counts, d_balance, d_z):
        r = routing.Routing()
        logits, r.offsets, r.weights, r.experts, r.state = ctx.saved_tensors
        r.valid, r.counts, r.k, r.renormalize = None, ctx.counts, ctx.k, ctx.renormalize
        d = None
        if ctx.needs_input_grad[0]:
            if d_weights is not None:
                d_weights = d_weights.contiguous()
            d = routing.route_backward(r, logits, d_weights=d_weights, d_balance=d_balance, d_z=d_z,
                                       handle=ctx.handle)
        return d, None, None, None, None, None


def route(logits: torch.Tensor, k: int, valid=None, offsets=None, renormalize: bool = True,
          handle: FLCE = None):
    """Expert routing as a differentiable call: (weights, experts, counts,
    balance, z) of routing.route. Gradients reach logits from the weights and
    the two losses; the experts and their counts carry none. Neither direction
    synchronises the host."""
    return RouteFunction.apply(logits, k, valid, offsets, renormalize, handle)


def _without_graph(*tensors):
    """The tensors, of which none asks for a gradient where none is recorded: needs_input_grad
    does not see no_grad."""
    return tensors if torch.is_grad_enabled() else tuple(t.detach() for t in tensors)


class TokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, t, temperature, top, ignore_index, keep_logits, handle):
        x, W, t = x.contiguous(), W.contiguous(), t.contiguous()
        keep = keep_logits and (ctx.needs_input_grad[0] or ctx.needs_input_grad[1])
        r = scoring.token_logprobs(x, W, t, temperature=temperature, top=top, ignore_index=ignore_index,
                                   keep_logits=keep, handle=handle)
        ctx.handle, ctx.temperature, ctx.ignore_index = handle, r.temperature, ignore_index
        ctx.save_for_backward(x, W, t, r.logprobs, r.entropy, r.stats, r.kept)
        ctx.set_materialize_grads(False)
        if top:
            ctx.mark_non_differentiable(r.top_logprobs, r.top_ids)
        return r.logprobs, r.entropy, r.top_logprobs, r.top_ids

    @staticmethod
    @once_differentiable
    def backward(ctx, d_logprobs, d_entropy, _d_top_logprobs, _d_top_ids):
        none = (None,) * 6
        if d_logprobs is None and d_entropy is None:
            return (None, None) + none
        r = scoring.TokenLogprobs()
        x, W, t, r.logprobs, r.entropy, r.stats, r.kept = ctx.saved_tensors
        r.top_logprobs = r.top_ids = None
        r.temperature, r.ignore_index = ctx.temperature, ctx.ignore_index
        need_x, need_W = ctx.needs_input_grad[:2]
        if d_logprobs is not None:
            d_logprobs = d_logprobs.contiguous()
        if d_entropy is not None:
            d_entropy = d_entropy.contiguous()
        dx, dW = scoring.token_logprobs_backward(r, x, W, t, d_logprobs=d_logprobs, d_entropy=d_entropy,
                                                 dx=need_x, dW=need_W, handle=ctx.handle)
        return (dx, dW) + none


def token_logprobs(x: torch.Tensor, W: torch.Tensor, t: torch.Tensor, temperature: float = 1.0, top: int = 0,
                   ignore_index: int = -100, keep_logits: bool = False, handle: FLCE = None):
    """Scoring as a differentiable call: (logprobs, entropy, top_logprobs,
    top_ids) of scoring.token_logprobs (the latter two None with top 0).
    Gradients reach x and W from logprobs and entropy; the alternatives carry
    none. Neither direction synchronises the host; an input that needs no
    gradient costs no product. keep_logits holds the logits until the backward,
    which else computes them again. A backward pass that is captured into a CUDA
    graph needs leaves that no graph of autograd from outside the capture still
    holds; scoring.token_logprobs_backward asks for nothing of the kind."""
    x, W = _without_graph(x, W)
    return TokenLogprobsFunction.apply(x, W, t, temperature, top, ignore_index, keep_logits, handle)


class LinearDistillationFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, ids, logits, temperature, handle):
        need_x, need_W = ctx.needs_input_grad[:2]
        loss, dx, dW = scoring.distill(x.contiguous(), W.contiguous(), ids, logits, temperature=temperature,
                                       backward=need_x or need_W, dx=need_x, dW=need_W, handle=handle)
        ctx.save_for_backward(dx, dW)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        dx, dW = ctx.saved_tensors
        # the factor meets the gradients in their own type, as in the fused loss
        return (None if dx is None else dx * grad_out.to(dx.dtype), None if dW is None else dW * grad_out.to(dW.dtype),
                None, None, None, None)


def linear_distillation(x: torch.Tensor, W: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor,
                        temperature: float = 1.0, handle: FLCE = None) -> torch.Tensor:
    """Distillation from a teacher's top logits, fused as linear_cross_entropy is:
    the forward computes the gradients too and the backward scales them. Returns
    the loss of scoring.distill, a 0-dim float32 tensor; never synchronises the
    host. The teacher gets no gradient. To capture a step into a CUDA graph, see
    token_logprobs; scoring.distill is the call without autograd."""
    x, W = _without_graph(x, W)
    return LinearDistillationFunction.apply(x, W, ids, logits, temperature, handle)
