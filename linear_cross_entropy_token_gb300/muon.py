"""The orthogonalised momentum update of weight matrices (Newton-Schulz).

``muon_update`` takes matrices of one shape through momentum, normalisation,
the Newton-Schulz steps on the short side and the weight update in one group of
launches; ``orthogonalize`` is the map alone; ``Muon`` is a torch optimizer on
top. include/flce.h has the formulas and the precision (flce_muon_update).
These functions only check and marshal; the computation runs in the library's
kernels on torch's current stream, without a host synchronisation.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .flce import DTYPE_BF16, DTYPE_FP32, FLCE, MuonArgs, MuonMatrix, _stream_ptr, load
from .routing import _handle, _row_stride

DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}
MAX_DIM = 65536
MAX_STEPS = 32


def check_muon_tensors(grads, momenta, weights, updates) -> None:
    """Shapes, dtypes, devices and layout of one call's matrices, and that none
    that is written shares memory with another. Raises ValueError."""
    rows, cols = grads[0].shape if grads[0].dim() == 2 else (0, 0)
    if not (1 <= rows <= MAX_DIM and 1 <= cols <= MAX_DIM):
        raise ValueError(f"the matrices must be 2-D with 1 to {MAX_DIM} rows and columns")
    dev = grads[0].device
    spans = []   # first byte, one past the last, row stride and row length in bytes, whether it is written
    for name, group, dtypes in (("grads", grads, DTYPES), ("momenta", momenta, (torch.float32,)),
                                ("weights", weights, DTYPES), ("updates", updates, DTYPES)):
        if group is None:
            continue
        if len(group) != len(grads):
            raise ValueError(f"{name} must have as many matrices as grads")
        dtype = group[0].dtype
        if dtype not in dtypes:
            raise ValueError(f"{name} must be of a supported dtype")
        size = group[0].element_size()
        length, reach, is_written = cols * size, (rows - 1) * size, name != "grads"
        for t in group:
            if tuple(t.shape) != (rows, cols) or t.dtype != dtype:
                raise ValueError(f"{name} must all be of shape ({rows}, {cols}) and of one supported dtype")
            stride, inner = t.stride()
            if t.device != dev or (cols > 1 and inner != 1) or (rows > 1 and stride < cols):
                raise ValueError(f"{name} must have contiguous rows that do not overlap, on {dev}")
            start = t.data_ptr()
            spans.append((start, start + reach * stride + length, stride * size, length, is_written))
    spans.sort()
    if dev.type == "meta" or all(one[1] <= two[0] for one, two in zip(spans, spans[1:])):
        return
    open_spans = []   # that reach past the current one's first byte: slices of one tensor, or gradients
    for span in spans:
        open_spans = [other for other in open_spans if other[1] > span[0]]
        if any((span[4] or other[4]) and _meet(other, span) for other in open_spans):
            raise ValueError("a matrix that is written overlaps another of the call")
        open_spans.append(span)


def _meet(a, b) -> bool:
    """Whether two matrices whose address ranges meet, the second starting no
    earlier than the first, share a byte."""
    (start_a, end_a, stride_a, length_a, _), (start_b, end_b, stride_b, length_b, _) = a, b
    if end_a - start_a == length_a and end_b - start_b == length_b:   # one row each
        return True
    if stride_a == stride_b:   # slices of one tensor: each row of b stands alike to a row of a and the next
        row, into = divmod(start_b - start_a, stride_a)
        return into < length_a or (into + length_b > stride_a and start_a + (row + 1) * stride_a < end_a)
    while start_a < end_a and start_b < end_b:   # row by row
        if start_a + length_a <= start_b:
            start_a += stride_a
        elif start_b + length_b <= start_a:
            start_b += stride_b
        else:
            return True
    return False


def _coefficients(coefficients, steps):
    if not 1 <= steps <= MAX_STEPS:
        raise ValueError(f"steps must lie in 1 .. {MAX_STEPS}")
    if coefficients is None:
        return None
    rows = list(coefficients)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients must be (a, b, c), or one such triple for every step")
    return (ctypes.c_float * (3 * steps))(*(float(v) for r in rows for v in r))


def muon_update(grads, momenta=None, weights=None, *, beta: float = 0.95, nesterov: bool = True,
                steps: int = 5, coefficients=None, eps: float = 1e-7, scale: float = 1.0,
                lr: float = 0.0, weight_decay: float = 0.0, updates=None,
                update_dtype: torch.dtype = torch.bfloat16, handle: FLCE = None):
    """One update of matrices of one shape.

    grads: list of (rows, cols) float32 or bfloat16 tensors. momenta: list of
    float32 tensors, updated in place, or None to orthogonalise the gradients
    themselves. weights: list of float32 or bfloat16 tensors, updated in place
    with lr and weight_decay (returned), or None: the updates scale * O are
    written to `updates`, new tensors of update_dtype by default (returned).
    Gradients may share memory; a matrix that is written may share no element
    with another. No result carries a gradient.

    The products round their operands to fp16: O is 1e-4 to 5e-3 of its own norm
    off the exact result (1.5e-2 at most, include/flce.h), one bfloat16
    rounding's size, and in float32 updates and weights no closer. Matrices with
    at most 32 rows or columns are 1e-6 to 6e-5 off.

    The call returns once its work is enqueued. A device-side wait that ran out
    (a GPU that no longer makes progress) leaves the results unspecified:
    async_status() raises for it, or the next update does.
    """
    return _update(*_marshal(grads, momenta, weights, beta, nesterov, steps, coefficients, eps, scale, lr, weight_decay,
                             updates, update_dtype, handle))


def _marshal(grads, momenta, weights, beta, nesterov, steps, coefficients, eps, scale, lr, weight_decay, updates=None,
             update_dtype=torch.bfloat16, handle=None):
    """The checks of one call, and its library arguments: what _update takes,
    the tensors that must live until it has launched among it."""
    grads = list(grads)
    momenta = None if momenta is None else list(momenta)
    weights = None if weights is None else list(weights)
    if weights is not None and updates is not None:
        raise ValueError("weights are updated in place: no updates are written")
    table = _coefficients(coefficients, steps)
    if not grads:
        return None, None, (), grads, [] if weights is None else weights, ()
    if updates is None and weights is None:
        if update_dtype not in DTYPES:
            raise ValueError("updates must be bfloat16 or float32")
        updates = [torch.empty(g.shape, dtype=update_dtype, device=g.device) for g in grads]
    updates = None if updates is None else list(updates)
    check_muon_tensors(grads, momenta, weights, updates)
    h = _handle(grads[0], handle)
    rows, cols = grads[0].shape
    a = MuonArgs(rows, cols, DTYPES[grads[0].dtype],
                 DTYPE_FP32 if weights is None else DTYPES[weights[0].dtype],
                 DTYPE_FP32 if updates is None else DTYPES[updates[0].dtype], int(nesterov), steps, 0,
                 table, beta, eps, scale, lr, weight_decay)
    mats = (MuonMatrix * len(grads))()
    for i, m in enumerate(mats):
        m.grad, m.ld_grad = grads[i].data_ptr(), _row_stride(grads[i])
        if momenta is not None:
            m.momentum, m.ld_momentum = momenta[i].data_ptr(), _row_stride(momenta[i])
        if weights is not None:
            m.weight, m.ld_weight = weights[i].data_ptr(), _row_stride(weights[i])
        else:
            m.update, m.ld_update = updates[i].data_ptr(), _row_stride(updates[i])
    # written behind autograd's back: a backward that saved one of these must fail
    written = [*(momenta or ()), *(weights or ()), *(updates or ())]
    return h, a, mats, grads, updates if weights is None else weights, written


def _update(h, a, mats, grads, result, written):
    if not mats:
        return result
    dev = grads[0].device
    nbytes = h.lib.flce_muon_workspace_bytes(a.rows, a.cols, len(mats))
    # torch's allocations are 512-byte aligned, the workspace 1024
    ws = torch.empty(nbytes + 1024, dtype=torch.uint8, device=dev)
    base = (ws.data_ptr() + 1023) // 1024 * 1024
    h._check(h.lib.flce_muon_update(h.h, ctypes.byref(a), mats, len(mats), base, nbytes, _stream_ptr(dev)),
             "flce_muon_update")
    torch.autograd.graph.increment_version(written)
    return result


def orthogonalize(G: torch.Tensor, *, steps: int = 5, coefficients=None, eps: float = 1e-7,
                  scale: float = 1.0, dtype: torch.dtype = torch.bfloat16, handle: FLCE = None) -> torch.Tensor:
    """scale * the Newton-Schulz map of G (..., rows, cols), matrix by matrix:
    the singular vectors of G with singular values near one. The result carries
    no gradient; its precision is muon_update's."""
    if G.dim() < 2:
        raise ValueError("G must have at least two dimensions")
    out = torch.empty(G.shape, dtype=dtype, device=G.device)
    if G.numel() == 0:
        return out
    flat = G.reshape(-1, *G.shape[-2:])
    muon_update(list(flat.unbind(0)), steps=steps, coefficients=coefficients, eps=eps, scale=scale,
                updates=list(out.view(-1, *G.shape[-2:]).unbind(0)), handle=handle)
    return out


def workspace_bytes(rows: int, cols: int, count: int = 1) -> int:
    """Device workspace of muon_update for count matrices (host only)."""
    return int(load().flce_muon_workspace_bytes(rows, cols, count))


class Muon(torch.optim.Optimizer):
    """Momentum, orthogonalisation and weight update for 2-D parameters.

    Parameters of one shape and type go through one call. scale: "rms" for
    0.2 sqrt(max(rows, cols)), which gives an update's entries the size of an
    adaptive optimizer's, "spectral" for sqrt(max(1, rows / cols)), or a
    number. Vectors, embeddings and the LM head belong to another optimizer.
    Momenta are float32 whatever the parameters' type, in checkpoints too. The
    orthogonalisation's precision is muon_update's.
    """

    def __init__(self, params, lr: float = 2e-2, beta: float = 0.95, weight_decay: float = 0.0,
                 nesterov: bool = True, steps: int = 5, coefficients=None, eps: float = 1e-7,
                 scale="rms"):
        defaults = dict(lr=lr, beta=beta, weight_decay=weight_decay, nesterov=nesterov, steps=steps,
                        coefficients=coefficients, eps=eps, scale=scale)
        self._check_group({"params": (), **defaults})
        super().__init__(params, defaults)

    def add_param_group(self, param_group) -> None:
        """As torch's (the constructor's groups come here too), refused where
        step could not take the group: the optimizer then stays as it was."""
        super().add_param_group(param_group)
        try:
            self._check_group(self.param_groups[-1])
        except Exception:
            self.param_groups.pop()
            raise

    @staticmethod
    def _check_group(group) -> None:
        if not (group["lr"] >= 0.0 and 0.0 <= group["beta"] <= 1.0 and group["weight_decay"] >= 0.0
                and group["eps"] >= 0.0):
            raise ValueError("need lr, weight_decay, eps >= 0 and 0 <= beta <= 1")
        if group["scale"] not in ("rms", "spectral") and not isinstance(group["scale"], (int, float)):
            raise ValueError("scale must be 'rms', 'spectral' or a number")
        _coefficients(group["coefficients"], group["steps"])
        for p in group["params"]:
            if p.dim() != 2 or p.dtype not in DTYPES:
                raise ValueError("Muon takes 2-D float32 or bfloat16 parameters")

    def load_state_dict(self, state_dict) -> None:
        """As torch's, but the momenta stay float32: torch gives floating-point
        state the parameter's type, which for bfloat16 parameters drops bits
        that no cast back returns. They are taken from the saved tensors."""
        loaded = []

        def note(_, given):   # after every other such hook: what is really loaded
            loaded[:] = [given]

        def restore(_):       # before every other: they see the final state
            given, = loaded
            ids = [i for group in given["param_groups"] for i in group["params"]]
            params = [p for group in self.param_groups for p in group["params"]]
            for i, p in zip(ids, params):
                momentum = given["state"].get(i, {}).get("momentum")
                if momentum is not None:
                    # a copy: momenta are updated in place, the saved ones may be another optimizer's
                    self.state[p]["momentum"] = momentum.to(dtype=torch.float32, device=p.device, copy=True)

        hooks = (self.register_load_state_dict_pre_hook(note),
                 self.register_load_state_dict_post_hook(restore, prepend=True))
        try:
            super().load_state_dict(state_dict)
        finally:
            for hook in hooks:
                hook.remove()

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # every group is checked before the first is launched, so that a step
        # that is refused changes nothing
        calls = []
        for group in self.param_groups:
            alike = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "momentum" not in state:
                    state["momentum"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                alike.setdefault((tuple(p.shape), p.dtype, p.grad.dtype, p.device), []).append(p)
            for (shape, _, _, _), ps in alike.items():
                scale = group["scale"]
                if scale == "rms":
                    scale = 0.2 * math.sqrt(max(shape))
                elif scale == "spectral":
                    scale = math.sqrt(max(1.0, shape[0] / shape[1]))
                call = _marshal([p.grad for p in ps], [self.state[p]["momentum"] for p in ps], ps, group["beta"],
                                group["nesterov"], group["steps"], group["coefficients"], group["eps"], scale,
                                group["lr"], group["weight_decay"])
                # the library's own checks of the options: with no matrices it makes those alone
                h, args = call[:2]
                h._check(h.lib.flce_muon_update(h.h, ctypes.byref(args), None, 0, None, 0, None), "flce_muon_update")
                calls.append(call)
        for call in calls:
            _update(*call)
        return loss
