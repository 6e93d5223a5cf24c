"""Expert routing with its balance and z losses, forward and backward.

Per token of router logits: softmax, the k largest experts (ties to the lowest
index) and their probabilities as weights. Over the live tokens: how many
slots chose each expert, the balance loss (per document where documents are
given, each weighted by its tokens) and the z loss. include/flce.h has the
formulas (flce_route_forward). These functions only check and marshal; the
computation runs in the library's kernels on torch's current stream, without a
host synchronisation. ``autograd.route`` is the differentiable form.
"""
from __future__ import annotations

import ctypes

import torch

from .flce import (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32, FLCE, RouteArgs, _stream_ptr, cached_handle)

LOGIT_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32, torch.float16: DTYPE_FP16}
MAX_EXPERTS = 1024
MAX_K = 32


class Routing:
    """What one routing call found, as device tensors.

    weights (N, k) float32 and experts (N, k) int32: each token's slots, best
    first; a slot that routes nowhere has expert -1 and weight 0.
    counts int64: slots per expert, (E,), or (documents, E) with offsets.
    balance, z: the losses, 0-dim float32. n_live: 0-dim int32.
    """

    # `state` holds the call's small results and what the backward reads, one
    # allocation: result (4 floats: balance, z, 1 / n, n), slope, stats, and
    # the forward's workspace behind them
    __slots__ = ("weights", "experts", "counts", "state", "valid", "offsets", "k", "renormalize")

    @property
    def balance(self) -> torch.Tensor:
        return self.state[0]

    @property
    def z(self) -> torch.Tensor:
        return self.state[1]

    @property
    def n_live(self) -> torch.Tensor:
        return self.state[3].view(torch.int32)

    def bind(self, logits, N, E, ld, code) -> RouteArgs:
        """The library's argument block for these logits."""
        offsets = self.offsets
        documents = 1 if offsets is None else offsets.numel() - 1
        slope, stats, _ = _state_layout(N, E, documents)
        base = self.state.data_ptr()
        return RouteArgs(logits.data_ptr(), code, self.k, N, E, ld, self.renormalize, 0,
                         None if self.valid is None else self.valid.data_ptr(),
                         None if offsets is None else offsets.data_ptr(), documents, self.weights.data_ptr(),
                         self.experts.data_ptr(), self.counts.data_ptr(), base + 4 * stats, base + 4 * slope,
                         base)


def _state_layout(N: int, E: int, documents: int):
    """Offsets, in floats, of slope, stats and the workspace in Routing.state."""
    stats = (4 + documents * E + 1) // 2 * 2          # pairs of floats, 8-byte aligned
    return 4, stats, (stats + 2 * N + 63) // 64 * 64   # the workspace on 256 bytes


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def check_route_tensors(logits, k, valid, offsets):
    """Shapes, dtypes, devices and layout of one call. Raises ValueError;
    returns (N, E, row stride, dtype code)."""
    shape = logits.shape
    code = LOGIT_DTYPES.get(logits.dtype)
    if len(shape) != 2 or code is None:
        raise ValueError("logits must be 2-D bfloat16, float32 or float16")
    N, E = shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"logits must have 1 to {MAX_EXPERTS} columns")
    if N >= 2 ** 31:
        raise ValueError("too many rows")
    ld, inner = logits.stride()
    if N <= 1:
        ld = E
    if (E > 1 and N > 0 and inner != 1) or ld < E:
        raise ValueError("the rows of logits must be contiguous and not overlap")
    if not 1 <= k <= min(E, MAX_K):
        raise ValueError(f"k must lie in 1 .. min(columns, {MAX_K})")
    if valid is not None and (valid.shape != (N,) or valid.dtype not in (torch.bool, torch.uint8)
                              or valid.device != logits.device or not valid.is_contiguous()):
        raise ValueError(f"valid must be a contiguous bool or uint8 tensor of shape ({N},) on {logits.device}")
    if offsets is not None and (offsets.dim() != 1 or not 2 <= offsets.numel() <= 2 ** 24
                                or offsets.dtype != torch.int64 or offsets.device != logits.device
                                or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be a contiguous 1-D int64 tensor of at least two entries on {logits.device}")
    return N, E, ld, code


def _handle(t: torch.Tensor, handle) -> FLCE:
    if not t.is_cuda:
        raise ValueError("the tensors must be on a CUDA device")
    index = t.device.index
    if handle is None:
        return cached_handle(index)
    if handle.device != index:
        raise ValueError(f"the handle is on device {handle.device}, the tensors on {t.device}")
    return handle


def _scalar(name, t, dev) -> int:
    if t.numel() != 1 or t.dtype != torch.float32 or t.device != dev:
        raise ValueError(f"{name} must be one float32 element on {dev}")
    return t.data_ptr()


def _workspace_bytes(h: FLCE, N: int, E: int, documents: int) -> int:
    return int(h.lib.flce_route_workspace_bytes(h.h, N, E, documents))


def route(logits: torch.Tensor, k: int, valid=None, offsets=None, renormalize: bool = True,
          handle: FLCE = None) -> Routing:
    """Route every row of logits (N, E) to its k largest experts.

    valid: (N,) bool, False for tokens that do not count (as ignored targets do
    not). offsets: (documents + 1,) int64 ascending from 0 to N, to balance
    each document by itself. renormalize: a token's weights sum to one.
    """
    N, E, ld, code = check_route_tensors(logits, k, valid, offsets)
    h = _handle(logits, handle)
    dev = logits.device
    documents = 1 if offsets is None else offsets.numel() - 1
    r = Routing()
    r.k, r.renormalize, r.valid, r.offsets = k, bool(renormalize), valid, offsets
    empty = torch.empty
    r.weights = empty((N, k), dtype=torch.float32, device=dev)
    r.experts = empty((N, k), dtype=torch.int32, device=dev)
    r.counts = empty((E,) if offsets is None else (documents, E), dtype=torch.int64, device=dev)
    nbytes = _workspace_bytes(h, N, E, documents)
    ws = _state_layout(N, E, documents)[2]
    r.state = empty(ws + (nbytes + 3) // 4, dtype=torch.float32, device=dev)
    a = r.bind(logits, N, E, ld, code)
    st = h.lib.flce_route_forward(h.h, ctypes.byref(a), a.result + 4 * ws, nbytes, _stream_ptr(dev))
    if st:
        h._check(st, "flce_route_forward")
    return r


def route_backward(r: Routing, logits: torch.Tensor, d_weights=None, d_balance=None, d_z=None,
                   out=None, handle: FLCE = None) -> torch.Tensor:
    """d logits (in the dtype of logits) from the gradients of r.weights
    (N, k) float32, of r.balance and of r.z (one float32 element on the device
    each); None stands for zero. logits are those that r was made from."""
    k = r.k
    N, E, ld, code = check_route_tensors(logits, k, r.valid, r.offsets)
    h = _handle(logits, handle)
    dev = logits.device
    if r.weights.shape != (N, k) or r.counts.shape[-1] != E or r.weights.device != dev:
        raise ValueError("the routing was not made from these logits")
    p_weights = p_balance = p_z = None
    if d_weights is not None:
        if (d_weights.shape != (N, k) or d_weights.dtype != torch.float32 or d_weights.device != dev
                or not d_weights.is_contiguous()):
            raise ValueError(f"d_weights must be contiguous float32 of shape ({N}, {k}) on {dev}")
        p_weights = d_weights.data_ptr()
    if d_balance is not None:
        p_balance = _scalar("d_balance", d_balance, dev)
    if d_z is not None:
        p_z = _scalar("d_z", d_z, dev)
    given = out is not None
    if not given:
        out = torch.empty((N, E), dtype=logits.dtype, device=dev)
        ld_out = E
    else:
        if (out.shape != (N, E) or out.dtype != logits.dtype or out.device != dev
                or (E > 1 and N > 0 and out.stride(1) != 1) or (N > 1 and out.stride(0) < E)):
            raise ValueError(f"out must be {logits.dtype} of shape ({N}, {E}) with contiguous rows on {dev}")
        ld_out = _row_stride(out)
    a = r.bind(logits, N, E, ld, code)
    st = h.lib.flce_route_backward(h.h, ctypes.byref(a), p_weights, p_balance, p_z, out.data_ptr(), ld_out,
                                   _stream_ptr(dev))
    if st:
        h._check(st, "flce_route_backward")
    if given:
        torch.autograd.graph.increment_version(out)
    return out
