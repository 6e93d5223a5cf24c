"""Cases of the training-step operators beside the fused loss, for timing and
comparison: the expert router with its balance and z losses (forward, and
forward + backward), and the orthogonalised (Newton-Schulz) momentum update of
weight matrices.

`own` selects what `run` calls: False, the plain form in elementary torch
operations (32-bit arithmetic, 64-bit where long sums need it, one rounding at
the end); True, this framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # the quintic map of one Newton-Schulz step
STEPS = 5
EPS = 1e-7
BETA = 0.95
LR = 0.02
DECAY = 0.1


def listed():
    return [
        # a router at serving time: a handful of tokens, where only latency counts
        {"name": "route_decode", "op": "route", "n": 16, "e": 64, "k": 4, "dtype": "bf16", "documents": 0,
         "masked": 0.0, "padded": 0, "renormalize": True, "backward": False},
        # a few coarse experts in full precision, one small training batch
        {"name": "route_few_experts", "op": "route", "n": 2048, "e": 8, "k": 2, "dtype": "fp32", "documents": 0,
         "masked": 0.1, "padded": 0, "renormalize": False, "backward": True},
        # packed documents of uneven lengths balanced one by one, an odd number of experts of which
        # the last are padding (-inf), a tenth of the tokens ignored
        {"name": "route_documents", "op": "route", "n": 9001, "e": 67, "k": 5, "dtype": "fp16", "documents": 37,
         "masked": 0.1, "padded": 3, "renormalize": True, "backward": True},
        # an ordinary training batch
        {"name": "route_batch", "op": "route", "n": 16384, "e": 128, "k": 8, "dtype": "bf16", "documents": 0,
         "masked": 0.05, "padded": 0, "renormalize": True, "backward": True},
        # scoring a long context without training
        {"name": "route_long_forward", "op": "route", "n": 131072, "e": 64, "k": 6, "dtype": "bf16", "documents": 8,
         "masked": 0.0, "padded": 0, "renormalize": False, "backward": False},
        # a long-context training step, many experts, full-precision logits
        {"name": "route_long", "op": "route", "n": 131072, "e": 256, "k": 8, "dtype": "fp32", "documents": 0,
         "masked": 0.0, "padded": 0, "renormalize": True, "backward": True},
        # one small projection: latency of the whole chain of products
        {"name": "muon_small", "op": "muon", "count": 1, "rows": 128, "cols": 128, "grad": "fp32",
         "momentum": False, "nesterov": False, "weights": "none"},
        # ragged sizes: tiles, vectors and rows all end early
        {"name": "muon_odd", "op": "muon", "count": 3, "rows": 1000, "cols": 333, "grad": "bf16",
         "momentum": True, "nesterov": True, "weights": "none"},
        # the square projections of several layers of a small model, weights updated in place
        {"name": "muon_layers", "op": "muon", "count": 8, "rows": 1024, "cols": 1024, "grad": "fp32",
         "momentum": True, "nesterov": True, "weights": "bf16"},
        # tall matrices (more rows than columns): the products run on the short side
        {"name": "muon_tall", "op": "muon", "count": 2, "rows": 4096, "cols": 1024, "grad": "bf16",
         "momentum": True, "nesterov": False, "weights": "none"},
        # one large square projection
        {"name": "muon_square", "op": "muon", "count": 1, "rows": 4096, "cols": 4096, "grad": "fp32",
         "momentum": True, "nesterov": True, "weights": "none"},
        # the widest matrix of a large layer, with its weights
        {"name": "muon_wide", "op": "muon", "count": 1, "rows": 4096, "cols": 16384, "grad": "bf16",
         "momentum": True, "nesterov": True, "weights": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.5:
        e = _log(rng, 4, 384)
        n = _log(rng, 1, 131072)
        while n * e > 131072 * 256:
            n = _log(rng, 1, 131072)
        return {"op": "route", "n": n, "e": e, "k": rng.randint(1, min(e, 12)),
                "dtype": rng.choice(("fp32", "bf16", "fp16")),
                "documents": rng.choice((0, 1, _log(rng, 2, 200))), "masked": rng.choice((0.0, 0.05, 0.3)),
                "padded": rng.choice((0, 0, e // 8)), "renormalize": rng.random() < 0.5,
                "backward": rng.random() < 0.7}
    largest = _products(4096, 16384)
    while True:
        case = {"op": "muon", "count": rng.choice((1, 1, 2, 3, 5, 8)), "rows": _log(rng, 8, 8192),
                "cols": _log(rng, 8, 8192), "grad": rng.choice(("fp32", "bf16")),
                "momentum": rng.random() < 0.7, "nesterov": rng.random() < 0.5,
                "weights": rng.choice(("none", "none", "bf16"))}
        if case["count"] * _products(case["rows"], case["cols"]) <= largest:
            return case


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "route":
        n, e = case["n"], case["e"]
        # a router's logits: a common preference over the experts, and each token's own
        z = torch.randn(n, e, generator=g, device="cuda") * 1.5
        z += torch.randn(1, e, generator=g, device="cuda") * 0.7
        if case["padded"]:
            z[:, e - case["padded"]:] = -math.inf
        s = {"case": case, "logits": z.to(DTYPES[case["dtype"]]), "valid": None, "offsets": None}
        if case["masked"]:
            s["valid"] = torch.rand(n, generator=g, device="cuda") >= case["masked"]
        if case["documents"]:
            cuts = torch.randint(0, n + 1, (case["documents"] - 1,), generator=g, device="cuda")
            ends = torch.tensor([0, n], device="cuda")
            s["offsets"] = torch.cat([ends, cuts]).sort().values
        if case["backward"]:
            # the gradients that reach the router: of the experts' weights, and the two losses' factors
            s["d_weights"] = torch.randn(n, case["k"], generator=g, device="cuda") * (1.0 / max(n, 1))
            s["d_balance"] = torch.full((), 0.01, device="cuda")
            s["d_z"] = torch.full((), 0.001, device="cuda")
        return s
    count, rows, cols = case["count"], case["rows"], case["cols"]
    rank = max(1, min(rows, cols) // 16)

    def gradient():
        # a few strong directions over a noise floor, rows of different magnitude
        a = torch.randn(count, rows, rank, generator=g, device="cuda")
        b = torch.randn(count, rank, cols, generator=g, device="cuda")
        noise = torch.randn(count, rows, cols, generator=g, device="cuda")
        scale = torch.exp(0.5 * torch.randn(count, rows, 1, generator=g, device="cuda"))
        return 1e-3 * scale * (noise + a @ b / math.sqrt(rank))

    s = {"case": case, "momenta": None, "weights": None}
    s["grads"] = list(gradient().to(DTYPES[case["grad"]]).unbind(0))
    if case["momentum"]:
        s["momenta"] = list(gradient().unbind(0))
    if case["weights"] != "none":
        w = 0.02 * torch.randn(count, rows, cols, generator=g, device="cuda")
        s["weights"] = list(w.to(DTYPES[case["weights"]]).unbind(0))
    return s


def _scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


# ------------------------------------------------------------------ plain forms

def _document_of(offsets, n, device):
    """The document of every token, as an index into the documents."""
    if offsets is None:
        return torch.zeros(n, dtype=torch.int64, device=device), 1
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(n, device=device), right=True), offsets.numel() - 1


def _plain_route(s):
    case = s["case"]
    z = s["logits"].float()
    n, e = z.shape
    k = case["k"]
    document, documents = _document_of(s["offsets"], n, z.device)
    top = z.max(dim=1, keepdim=True).values
    live = (top > -math.inf).squeeze(1)
    if s["valid"] is not None:
        live = live & s["valid"]
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    ex = torch.exp(z - top)
    total = ex.sum(dim=1, keepdim=True)
    p = torch.where(live.unsqueeze(1), ex / total, torch.zeros_like(ex))
    lse = torch.where(live, (top + torch.log(total)).squeeze(1), torch.zeros_like(total).squeeze(1))
    # the k largest logits, ties to the lowest expert
    chosen, experts = (v[:, :k] for v in torch.sort(z, dim=1, descending=True, stable=True))
    taken = live.unsqueeze(1) & (chosen > -math.inf)
    experts = torch.where(taken, experts, torch.full_like(experts, -1))
    weights = torch.where(taken, p.gather(1, experts.clamp(min=0)), torch.zeros_like(chosen))
    share = weights.sum(dim=1, keepdim=True)
    if case["renormalize"]:
        weights = torch.where(share > 0, weights / share, weights)
    hit = torch.zeros(n, e, dtype=torch.float64, device=z.device)
    hit.scatter_add_(1, experts.clamp(min=0).long(), taken.double())
    member = (document.unsqueeze(0) == torch.arange(documents, device=z.device).unsqueeze(1)).double()
    counts = member @ hit
    mass = member @ p.double()
    n_doc = member @ live.double()
    n_live = n_doc.sum()
    # d balance / d p of a token: E counts / (k n_document n_live)
    slope = e * counts / (k * n_doc.clamp(min=1.0) * n_live.clamp(min=1.0)).unsqueeze(1)
    balance = (slope * mass).sum()
    z_loss = lse.double().square().sum() / n_live.clamp(min=1.0)
    out = {"weights": weights, "experts": experts.int(), "counts": counts.long(),
           "balance": balance.float(), "z": z_loss.float()}
    if not case["backward"]:
        return out
    d_p = s["d_balance"] * slope.float()[document]
    d_w = torch.where(taken, s["d_weights"], torch.zeros_like(s["d_weights"]))
    if case["renormalize"]:
        d_w = torch.where(share > 0, (d_w - (d_w * weights).sum(dim=1, keepdim=True)) / share, d_w)
    d_p = d_p.scatter_add(1, experts.clamp(min=0).long(), d_w)
    d_logits = p * (d_p - (d_p * p).sum(dim=1, keepdim=True))
    d_logits = d_logits + p * (2.0 * s["d_z"] * lse / n_live.clamp(min=1.0).float()).unsqueeze(1)
    out["d_logits"] = d_logits.to(s["logits"].dtype)
    return out


def _plain_muon(s):
    case = s["case"]
    rows, cols = case["rows"], case["cols"]
    u = torch.stack(s["grads"]).float()
    out = {}
    if s["momenta"] is not None:
        m = torch.stack(s["momenta"]) * BETA + u * (1.0 - BETA)
        u = m * BETA + u * (1.0 - BETA) if case["nesterov"] else m
        s["momenta"] = list(m.unbind(0))
        out["momenta"] = s["momenta"]
    if rows > cols:
        u = u.transpose(1, 2)
    x = u / (u.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if rows > cols:
        x = x.transpose(1, 2)
    x = x * _scale(rows, cols)
    if s["weights"] is None:
        out["updates"] = list(x.to(torch.bfloat16).unbind(0))
    else:
        w = torch.stack(s["weights"])
        w = (w.float() * (1.0 - LR * DECAY) - LR * x).to(w.dtype)
        s["weights"] = list(w.unbind(0))
        out["weights"] = s["weights"]
    return out


# ---------------------------------------------------------- the framework's calls

def _own_route(s):
    import linear_cross_entropy_token_gb300 as flce
    case = s["case"]
    r = flce.route(s["logits"], case["k"], valid=s["valid"], offsets=s["offsets"],
                   renormalize=case["renormalize"])
    out = {"weights": r.weights, "experts": r.experts, "counts": r.counts, "balance": r.balance, "z": r.z}
    if case["backward"]:
        out["d_logits"] = flce.route_backward(r, s["logits"], d_weights=s["d_weights"],
                                              d_balance=s["d_balance"], d_z=s["d_z"])
    if s["offsets"] is None:
        out["counts"] = out["counts"].view(1, -1)
    return out


def _own_muon(s):
    import linear_cross_entropy_token_gb300 as flce
    case = s["case"]
    out = {}
    updates = flce.muon_update(s["grads"], momenta=s["momenta"], weights=s["weights"], beta=BETA,
                               nesterov=case["nesterov"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                               scale=_scale(case["rows"], case["cols"]), lr=LR, weight_decay=DECAY)
    if s["momenta"] is not None:
        out["momenta"] = s["momenta"]
    if s["weights"] is None:
        out["updates"] = updates
    else:
        out["weights"] = s["weights"]
    return out


def run(state):
    if own:
        return _own_route(state) if state["case"]["op"] == "route" else _own_muon(state)
    return _plain_route(state) if state["case"]["op"] == "route" else _plain_muon(state)


# ------------------------------------------------------------------- work and exact

def _products(rows, cols):
    """Multiply-adds x 2 of the Newton-Schulz products of one matrix on its short side m: X Xt and A A are
    symmetric, so half of each suffices; B X is full."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)


def work(case):
    if case["op"] == "route":
        n, e, k, b = case["n"], case["e"], case["k"], BYTES[case["dtype"]]
        documents = max(1, case["documents"])
        moved = n * e * b + n * k * 8 + documents * e * 8 + (n if case["masked"] else 0) + 8
        flops = n * e * 5
        if case["backward"]:
            moved += n * e * b + n * k * 4
            flops += n * e * 6
        return {"bytes": moved, "flops": flops}
    elements = case["count"] * case["rows"] * case["cols"]
    moved = elements * BYTES[case["grad"]]
    if case["momentum"]:
        moved += elements * 8
    moved += elements * (2 if case["weights"] == "none" else 2 * BYTES[case["weights"]])
    return {"bytes": moved, "flops": case["count"] * _products(case["rows"], case["cols"]) + 8 * elements}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "muon":
        updates, momenta, weights = [], [], []
        for i, grad in enumerate(s["grads"]):
            v = grad.double()
            if case["momentum"]:
                buf = BETA * s["momenta"][i].double() + (1.0 - BETA) * v
                momenta.append(buf)
                v = BETA * buf + (1.0 - BETA) * v if case["nesterov"] else buf
            y = v / (torch.linalg.vector_norm(v) + EPS)
            for _ in range(STEPS):
                # on the side where the Gram matrix is small
                left = case["rows"] <= case["cols"]
                gram = y @ y.mT if left else y.mT @ y
                poly = COEFFICIENTS[1] * gram + COEFFICIENTS[2] * (gram @ gram)
                y = COEFFICIENTS[0] * y + (poly @ y if left else y @ poly)
            y = y * _scale(case["rows"], case["cols"])
            updates.append(y)
            if case["weights"] != "none":
                weights.append((1.0 - LR * DECAY) * s["weights"][i].double() - LR * y)
        out = {"momenta": momenta} if case["momentum"] else {}
        out["updates" if case["weights"] == "none" else "weights"] = updates if case["weights"] == "none" else weights
        return out
    z = s["logits"].double()
    n, e = z.shape
    k = case["k"]
    live = torch.isfinite(z).any(dim=1)
    if s["valid"] is not None:
        live &= s["valid"]
    p = torch.softmax(z, dim=1)
    p[~live] = 0.0
    lse = torch.logsumexp(z, dim=1)
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k]
    picked = torch.isfinite(z.gather(1, order)) & live[:, None]
    inside = p.gather(1, order) * picked
    mass = inside.sum(dim=1, keepdim=True)
    mass[mass == 0] = 1.0
    weights = inside / mass if case["renormalize"] else inside
    bounds = [0, n] if s["offsets"] is None else s["offsets"].tolist()
    n_live = max(int(live.sum()), 1)
    balance = torch.zeros((), dtype=torch.float64, device="cuda")
    slope = torch.zeros_like(z)
    for lo, hi in zip(bounds[:-1], bounds[1:]):
        inside_live = int(live[lo:hi].sum())
        if inside_live == 0:
            continue
        counts = torch.bincount(order[lo:hi][picked[lo:hi]], minlength=e).double()
        f = e / (k * inside_live) * counts
        balance += (inside_live / n_live) * (f * p[lo:hi].sum(dim=0) / inside_live).sum()
        slope[lo:hi] = f / n_live
    out = {"weights": weights, "experts": None, "counts": None, "balance": balance,
           "z": lse[live].square().sum() / n_live}
    if case["backward"]:
        # by the chain rule through each output: the chosen weights, then the two losses
        up = 0.01 * slope
        back = s["d_weights"].double() * picked
        if case["renormalize"]:
            back = (back - (back * weights).sum(dim=1, keepdim=True)) / mass
        up = up.scatter_add(1, order, back)
        lse = torch.where(live, lse, torch.zeros_like(lse))
        out["d_logits"] = p * (up - (up * p).sum(dim=1, keepdim=True) + 0.002 / n_live * lse[:, None])
    return out
