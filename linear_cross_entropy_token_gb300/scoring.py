"""The head's operators beside the mean loss: log probabilities of given tokens
with entropy and top alternatives, and distillation from a teacher's top logits.

Both start from hidden states x (N, H) and the head's weights W (V, H) and hold
no N x V logits, unless a caller asks to keep them for the backward.
include/flce.h has the formulas (flce_logprobs_forward, flce_distill). These
functions only check and marshal; the computation runs in the library's kernels
on torch's current stream, without a host synchronisation: what only the device
can see (a token id out of range) is reported by ``async_status``.
``autograd.token_logprobs`` and ``autograd.linear_distillation`` are the
differentiable forms.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .flce import (DTYPE_BF16, DTYPE_FP16, DTYPE_FP32, FLCE, FlceError, DistillArgs, LogprobsArgs, _stream_ptr,
                   cached_handle, check_call_tensors)

TEACHER_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32, torch.float16: DTYPE_FP16}
HANDLE_DTYPES = {torch.bfloat16: "bf16", torch.float32: "fp32"}
MAX_TOP = 64
MAX_TEACHER = 256


class TokenLogprobs:
    """What one scoring call found, as device tensors.

    logprobs (N,) float32: each given token's log probability (None without t).
    entropy (N,) float32: of each row's distribution, in nats.
    top_logprobs (N, top) float32 and top_ids (N, top) int64: the alternatives,
    best first (None with top 0).
    Rows whose token is ignore_index hold zeros, their ids -1.
    """

    # stats and kept are what the backward reads besides
    __slots__ = ("logprobs", "entropy", "top_logprobs", "top_ids", "stats", "kept", "temperature", "ignore_index")

    def bind(self, x, W, t, top: int) -> LogprobsArgs:
        """The library's argument block for these inputs."""
        ptr = _ptr
        return LogprobsArgs(x.data_ptr(), W.data_ptr(), ptr(t), x.shape[0], x.shape[1], W.shape[0], self.ignore_index,
                            self.temperature, top, 0, ptr(self.logprobs), self.entropy.data_ptr(),
                            self.stats.data_ptr(), ptr(self.top_logprobs), ptr(self.top_ids), ptr(self.kept))


def _ptr(t):
    return None if t is None else t.data_ptr()


def check_score_tensors(x, W, t, temperature, top) -> None:
    """Shapes, dtypes, devices and layout of one scoring call. Raises ValueError."""
    if x.dtype not in HANDLE_DTYPES:
        raise ValueError("x must be bfloat16 or float32")
    if t is None:
        if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1] or W.dtype != x.dtype:
            raise ValueError("x and W must be 2-D, of one dtype and of as many columns")
        for name, ten in (("x", x), ("W", W)):
            if ten.device != x.device or not ten.is_contiguous():
                raise ValueError(f"{name} must be a contiguous tensor on {x.device}")
    else:
        check_call_tensors(x, W, t, None, None, x.dtype, x.device, x.device)
    V, H = W.shape
    if V < 1 or H < 1:
        raise ValueError("W must have at least one row and one column")
    if x.dtype == torch.bfloat16 and H % 8:
        raise ValueError("bfloat16 x and W must have a multiple of 8 columns")
    _check_temperature(temperature)
    if isinstance(top, bool) or not isinstance(top, int) or not 0 <= top <= min(V, MAX_TOP):
        raise ValueError(f"top must be an int in 0 .. min(rows of W, {MAX_TOP})")


def _check_temperature(temperature) -> None:
    if not 1e-30 < temperature < 1e30:   # NaN fails too
        raise ValueError("the temperature must be positive and finite")


def check_distill_tensors(x, W, ids, logits, temperature):
    """Shapes, dtypes, devices and layout of one distillation call. Raises
    ValueError; returns the row strides of ids and logits."""
    check_score_tensors(x, W, None, temperature, 0)
    N = x.shape[0]
    if ids.dim() != 2 or logits.shape != ids.shape or ids.shape[0] != N:
        raise ValueError(f"ids and logits must both be ({N}, K)")
    K = ids.shape[1]
    if not 1 <= K <= MAX_TEACHER:
        raise ValueError(f"K must lie in 1 .. {MAX_TEACHER}")
    if ids.dtype != torch.int64 or logits.dtype not in TEACHER_DTYPES:
        raise ValueError("ids must be int64, logits bfloat16, float32 or float16")
    strides = []
    for name, ten in (("ids", ids), ("logits", logits)):
        if ten.device != x.device:
            raise ValueError(f"{name} must be on {x.device}")
        if (K > 1 and N > 0 and ten.stride(1) != 1) or (N > 1 and ten.stride(0) < K):
            raise ValueError(f"the rows of {name} must be contiguous and not overlap")
        strides.append(ten.stride(0) if N > 1 else K)
    return strides


def _handle(x: torch.Tensor, handle) -> FLCE:
    if not x.is_cuda:
        raise ValueError("the tensors must be on a CUDA device")
    index = x.device.index
    if handle is None:
        return cached_handle(index, HANDLE_DTYPES[x.dtype])
    if handle.device != index:
        raise ValueError(f"the handle is on device {handle.device}, the tensors on {x.device}")
    if handle.dtype != HANDLE_DTYPES[x.dtype]:
        raise ValueError(f"the handle is for {handle.dtype}, the tensors are {x.dtype}")
    return handle


def _vector(name, t, n, dev):
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != torch.float32 or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 of shape ({n},) on {dev}")
    return t.data_ptr()


def _span(a):
    """First and last byte of a tensor's memory, from its strides."""
    if a.numel() == 0:
        return a.data_ptr(), a.data_ptr()
    last = sum((n - 1) * s for n, s in zip(a.shape, a.stride()))
    return a.data_ptr(), a.data_ptr() + (last + 1) * a.element_size()


def _overlap(a, b) -> bool:
    """Whether the memory of one tensor reaches into that of the other."""
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _gradient(name, want, like, dtypes, read=()):
    """The tensor of a gradient: None for no gradient, a new one for True, or the
    caller's, which may share no memory with what the call reads."""
    if want is None or want is False:
        return None
    if want is True:
        return torch.empty_like(like)
    if (not isinstance(want, torch.Tensor) or want.shape != like.shape or want.dtype not in dtypes
            or want.device != like.device or not want.is_contiguous()):
        raise ValueError(f"{name} must be True, None or a contiguous tensor of shape {tuple(like.shape)}, "
                         f"{' or '.join(str(d) for d in dtypes)}, on {like.device}")
    if any(t is not None and t.device == want.device and _overlap(want, t) for t in read):
        raise ValueError(f"{name} must not share memory with the inputs or the other gradient")
    return want


def _written(*pairs) -> None:
    """Tensors of the caller's that a call wrote count as modified for autograd."""
    for given, out in pairs:
        if out is not None and given is out:
            torch.autograd.graph.increment_version(out)


def _dw_code(dW) -> int:
    return -1 if dW is None else TEACHER_DTYPES[dW.dtype]


def _workspace(h: FLCE, nbytes: int, dev, what: str) -> torch.Tensor:
    if nbytes == 0:
        msg = h.lib.flce_last_error(h.h).decode()
        raise FlceError(3, f"{what}: {msg}")
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def token_logprobs(x: torch.Tensor, W: torch.Tensor, t=None, temperature: float = 1.0, top: int = 0,
                   ignore_index: int = -100, keep_logits: bool = False, handle: FLCE = None) -> TokenLogprobs:
    """Score every row of x (N, H) against the head W (V, H).

    t: (N,) int64 tokens to take the log probability of; None for entropy and
    alternatives alone. temperature divides the logits. top: so many
    alternatives a row (at most 64). keep_logits: hold the N x V logits (two
    bytes each; four of float32 inputs) for token_logprobs_backward, which
    then need not compute them again.
    """
    check_score_tensors(x, W, t, temperature, top)
    h = _handle(x, handle)
    N, V, dev = x.shape[0], W.shape[0], x.device
    r = TokenLogprobs()
    r.temperature, r.ignore_index = float(temperature), ignore_index
    empty = torch.empty
    r.logprobs = None if t is None else empty(N, dtype=torch.float32, device=dev)
    r.entropy = empty(N, dtype=torch.float32, device=dev)
    r.stats = empty((N, 2), dtype=torch.float32, device=dev)
    r.top_logprobs = empty((N, top), dtype=torch.float32, device=dev) if top else None
    r.top_ids = empty((N, top), dtype=torch.int64, device=dev) if top else None
    r.kept = None
    if keep_logits:
        r.kept = empty(int(h.lib.flce_logprobs_kept_bytes(h.h, N, V)), dtype=torch.uint8, device=dev)
    a = r.bind(x, W, t, top)
    ref = ctypes.byref(a)
    nbytes = int(h.lib.flce_logprobs_workspace_bytes(h.h, ref, 0, -1))
    ws = _workspace(h, nbytes, dev, "flce_logprobs_forward")
    st = h.lib.flce_logprobs_forward(h.h, ref, ws.data_ptr(), nbytes, _stream_ptr(dev))
    if st:
        h._check(st, "flce_logprobs_forward")
    return r


def token_logprobs_backward(r: TokenLogprobs, x: torch.Tensor, W: torch.Tensor, t: torch.Tensor, d_logprobs=None,
                            d_entropy=None, dx=True, dW=True, handle: FLCE = None):
    """(dx, dW) from the gradients of r.logprobs and r.entropy, (N,) float32
    each; None stands for zero. x, W and t are those that r was made from, and r's
    tensors are as they were.

    dx, dW: True for a new tensor of the type of x or W, None to leave that
    gradient (and its product) out, or the tensor to write: dW may be float32
    for bfloat16 W. They are overwritten, and may share no memory with the
    inputs.
    """
    if t is None:
        raise ValueError("the backward needs the tokens")
    check_score_tensors(x, W, t, r.temperature, 0)
    h = _handle(x, handle)
    N, V, dev = x.shape[0], W.shape[0], x.device
    if r.logprobs is None or r.entropy.shape != (N,) or r.entropy.device != dev:
        raise ValueError("the result was not made from these tokens")
    if r.kept is not None and r.kept.numel() != int(h.lib.flce_logprobs_kept_bytes(h.h, N, V)):
        raise ValueError("the kept logits are of other sizes")
    p_logprobs = _vector("d_logprobs", d_logprobs, N, dev)
    p_entropy = _vector("d_entropy", d_entropy, N, dev)
    read = (x, W, t, d_logprobs, d_entropy, r.logprobs, r.entropy, r.stats, r.kept)
    out_x = _gradient("dx", dx, x, (x.dtype,), read)
    out_W = _gradient("dW", dW, W, tuple({W.dtype, torch.float32}), (*read, out_x))
    a = r.bind(x, W, t, 0)
    ref = ctypes.byref(a)
    nbytes = int(h.lib.flce_logprobs_workspace_bytes(h.h, ref, 1, _dw_code(out_W)))
    ws = _workspace(h, nbytes, dev, "flce_logprobs_backward")
    st = h.lib.flce_logprobs_backward(h.h, ref, p_logprobs, p_entropy, _ptr(out_x), _ptr(out_W), _dw_code(out_W),
                                      ws.data_ptr(), nbytes, _stream_ptr(dev))
    if st:
        h._check(st, "flce_logprobs_backward")
    _written((dx, out_x), (dW, out_W))
    return out_x, out_W


def distill(x: torch.Tensor, W: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor, temperature: float = 1.0,
            backward: bool = True, dx=True, dW=True, handle: FLCE = None):
    """(loss, dx, dW): the divergence of the head's distribution from a teacher's
    top logits, and its gradients in the same pass.

    ids (N, K) int64 and logits (N, K): each token's entries of the teacher, K
    at most 256. Entries with id -1 or logit -inf do not count, and neither do
    tokens without one that does. The teacher's distribution is the softmax of
    logits / temperature over a token's entries; loss is the mean over tokens,
    times temperature^2, as a 0-dim float32 tensor. Without backward dx and dW
    are None; else as for token_logprobs_backward.
    """
    ld_ids, ld_logits = check_distill_tensors(x, W, ids, logits, temperature)
    h = _handle(x, handle)
    N, V, dev = x.shape[0], W.shape[0], x.device
    out_x = _gradient("dx", dx, x, (x.dtype,), (x, W, ids, logits)) if backward else None
    out_W = _gradient("dW", dW, W, tuple({W.dtype, torch.float32}), (x, W, ids, logits, out_x)) if backward else None
    loss = torch.empty((), dtype=torch.float32, device=dev)
    token_loss = torch.empty(N, dtype=torch.float32, device=dev)
    a = DistillArgs(x.data_ptr(), W.data_ptr(), ids.data_ptr(), logits.data_ptr(), N, x.shape[1], V, ids.shape[1],
                    ld_ids, ld_logits, TEACHER_DTYPES[logits.dtype], _dw_code(out_W), float(temperature),
                    loss.data_ptr(), token_loss.data_ptr(), _ptr(out_x), _ptr(out_W))
    ref = ctypes.byref(a)
    nbytes = int(h.lib.flce_distill_workspace_bytes(h.h, ref))
    ws = _workspace(h, nbytes, dev, "flce_distill")
    st = h.lib.flce_distill(h.h, ref, ws.data_ptr(), nbytes, _stream_ptr(dev))
    if st:
        h._check(st, "flce_distill")
    _written((dx, out_x), (dW, out_W))
    return loss, out_x, out_W
