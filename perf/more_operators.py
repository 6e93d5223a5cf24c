"""Cases of the LM-head operators beside the mean loss, for timing and comparison: log probabilities of
given tokens with entropy and top alternatives (forward, and forward + backward), and distillation from
a teacher's top logits with its gradients. Both start from hidden states x (N, H) and the head's weights
W (V, H).

`own` selects what `run` calls: False, the plain form in elementary torch operations (32-bit arithmetic,
64-bit where the order of near-equal alternatives needs it, one rounding at the end); True, this
framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
IGNORE = -100


def listed():
    return [
        # serving, one token at a time: the head's weights are all there is to read
        {"name": "score_one_token", "op": "score", "n": 1, "h": 4096, "v": 128256, "dtype": "bf16",
         "temperature": 1.0, "top": 20, "ignored": 0.0, "backward": False, "keep": False},
        # serving, a decoding batch with alternatives
        {"name": "score_decode", "op": "score", "n": 48, "h": 4096, "v": 151936, "dtype": "bf16",
         "temperature": 0.7, "top": 5, "ignored": 0.0, "backward": False, "keep": False},
        # scoring padded prompts of odd sizes: rows, columns and tiles all end early
        {"name": "score_odd", "op": "score", "n": 1003, "h": 1016, "v": 50257, "dtype": "bf16",
         "temperature": 1.3, "top": 33, "ignored": 0.3, "backward": False, "keep": False},
        # scoring a long context
        {"name": "score_long", "op": "score", "n": 16384, "h": 4096, "v": 128256, "dtype": "bf16",
         "temperature": 1.0, "top": 1, "ignored": 0.05, "backward": False, "keep": False},
        # a policy-gradient step of a tiny full-precision model: latency of the whole chain
        {"name": "policy_tiny", "op": "score", "n": 256, "h": 128, "v": 4096, "dtype": "fp32",
         "temperature": 1.0, "top": 0, "ignored": 0.25, "backward": True, "keep": False},
        # the same of a small model, its logits kept from the forward to the backward
        {"name": "policy_small", "op": "score", "n": 2048, "h": 1024, "v": 32000, "dtype": "bf16",
         "temperature": 1.0, "top": 0, "ignored": 0.1, "backward": True, "keep": True},
        # a long rollout of a large model, without the memory to keep N x V logits
        {"name": "policy_long", "op": "score", "n": 16384, "h": 4096, "v": 128256, "dtype": "bf16",
         "temperature": 1.0, "top": 0, "ignored": 0.5, "backward": True, "keep": False},
        # distilling a tiny full-precision student
        {"name": "distill_tiny", "op": "distill", "n": 256, "h": 128, "v": 4096, "dtype": "fp32", "k": 8,
         "teacher": "fp32", "temperature": 1.0, "padded": 0.0, "empty": 0.1, "backward": True},
        # ragged sizes, entries cut off at a probability (padding) and rows without any
        {"name": "distill_odd", "op": "distill", "n": 777, "h": 1000, "v": 50257, "dtype": "bf16", "k": 33,
         "teacher": "fp16", "temperature": 2.0, "padded": 0.3, "empty": 0.2, "backward": True},
        # evaluating a student: the loss alone
        {"name": "distill_evaluate", "op": "distill", "n": 4096, "h": 4096, "v": 32768, "dtype": "bf16", "k": 100,
         "teacher": "bf16", "temperature": 1.0, "padded": 0.0, "empty": 0.0, "backward": False},
        # an ordinary step of a small student
        {"name": "distill_small", "op": "distill", "n": 2048, "h": 1024, "v": 32000, "dtype": "bf16", "k": 64,
         "teacher": "fp32", "temperature": 1.5, "padded": 0.0, "empty": 0.05, "backward": True},
        # a long context of a large student
        {"name": "distill_long", "op": "distill", "n": 16384, "h": 4096, "v": 128256, "dtype": "bf16", "k": 64,
         "teacher": "bf16", "temperature": 1.0, "padded": 0.0, "empty": 0.05, "backward": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    largest = max(work(c)["flops"] for c in listed())
    while True:
        case = {"op": "score" if rng.random() < 0.55 else "distill", "n": _log(rng, 1, 16384),
                "dtype": "fp32" if rng.random() < 0.2 else "bf16",
                "temperature": rng.choice((1.0, 1.0, 0.7, 1.3, 2.0)), "backward": rng.random() < 0.6}
        if case["dtype"] == "fp32":
            # full precision is for small models
            case["n"] = min(case["n"], 1 + case["n"] % 512)
            case["h"], case["v"] = _log(rng, 33, 256), _log(rng, 500, 6000)
        else:
            case["h"], case["v"] = 8 * _log(rng, 8, 1024), _log(rng, 600, 160000)
        if case["op"] == "score":
            case["top"] = rng.choice((0, 1, _log(rng, 2, 64)))
            case["ignored"] = rng.choice((0.0, 0.1, 0.5))
            case["keep"] = case["backward"] and rng.random() < 0.4
        else:
            case["k"] = _log(rng, 1, 256)
            case["teacher"] = rng.choice(("fp32", "bf16", "fp16"))
            case["padded"], case["empty"] = rng.choice((0.0, 0.3)), rng.choice((0.0, 0.1))
        if work(case)["flops"] <= largest:
            return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, h, v = case["n"], case["h"], case["v"]
    dtype = DTYPES[case["dtype"]]
    std = 1.3 / math.sqrt(h)              # logits of a token with no preference: 1.3 around zero
    W = torch.empty(v, h, dtype=dtype, device="cuda")
    for i in range(0, v, 32768):
        rows = min(32768, v - i)
        W[i:i + rows] = (torch.randn(rows, h, generator=g, device="cuda") * std).to(dtype)
    # each token prefers one next token, by nothing up to a near certainty; frequent ids are more frequent
    u = torch.rand(n, generator=g, device="cuda")
    likely = ((v ** u - 1.0) * (v / max(v - 1, 1))).long().clamp(0, v - 1)
    strength = torch.rand(n, 1, generator=g, device="cuda") * 14.0
    x = torch.randn(n, h, generator=g, device="cuda") + strength * W[likely].float() / (std * std * h)
    s = {"case": case, "x": x.to(dtype), "W": W}
    if case["op"] == "score":
        other = torch.randint(0, v, (n,), generator=g, device="cuda")
        t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.7, likely, other)
        # the first token counts in every batch
        gone = torch.rand(n, generator=g, device="cuda") < case["ignored"]
        gone[0] = False
        t[gone] = IGNORE
        s["t"] = t
        if case["backward"]:
            # an advantage per token, and the entropy bonus' factor
            s["d_logprobs"] = torch.randn(n, generator=g, device="cuda") / n
            s["d_entropy"] = torch.full((n,), -0.01 / n, device="cuda")
        return s
    k = min(case["k"], v)
    # the teacher's ids are distinct: the likely one, then gaps that never go round the vocabulary
    gaps = torch.randint(1, max(v // k, 1) + 1, (n, k), generator=g, device="cuda")
    gaps[:, 0] = likely
    s["ids"] = gaps.cumsum(1) % v
    falls = -torch.log1p(-torch.rand(n, k, generator=g, device="cuda")) * 0.4
    falls[:, 0] = -8.0 * torch.rand(n, generator=g, device="cuda") - 6.0
    logits = (-falls.cumsum(1)).to(DTYPES[case["teacher"]])
    if case["padded"]:
        # entries below a probability are cut off: the tail of the row
        left = (k * (1.0 - 2.0 * case["padded"] * torch.rand(n, 1, generator=g, device="cuda"))).ceil()
        cut = torch.arange(k, device="cuda") >= left.clamp(min=1)
        s["ids"][cut] = -1
        logits[cut] = -math.inf
    if case["empty"]:
        gone = torch.rand(n, generator=g, device="cuda") < case["empty"]
        gone[0] = False
        s["ids"][gone] = -1
        logits[gone] = -math.inf
    s["teacher"] = logits
    return s


# ------------------------------------------------------------------ plain forms

def _chunks(n, v):
    rows = max(1, min(n, (1 << 29) // v))
    return [(i, min(n, i + rows)) for i in range(0, n, rows)]


def _plain_alternatives(x, W, z, top, v):
    """Ids and logits of the `top` largest, ties to the lowest id. Logits that 32-bit sums cannot tell apart are
    summed in 64 bits: candidates a little beyond the border, by id, then stably by value."""
    near = z.topk(min(top + 8, v), dim=1).indices.sort(dim=1).values
    values = torch.empty(near.shape, dtype=torch.float64, device=z.device)
    rows = max(1, (1 << 27) // (near.shape[1] * x.shape[1]))
    for i in range(0, x.shape[0], rows):
        picked = W[near[i:i + rows]].double()
        values[i:i + rows] = (picked * x[i:i + rows, None, :].double()).sum(dim=2)
    values, order = torch.sort(values, dim=1, descending=True, stable=True)
    return near.gather(1, order)[:, :top], values[:, :top]


def _plain_score(s):
    case = s["case"]
    n, v, top, scale = case["n"], case["v"], min(case["top"], case["v"]), 1.0 / case["temperature"]
    x, W, t = s["x"], s["W"], s["t"]
    xf, Wf = x.float(), W.float()
    live = t != IGNORE
    out = {"logprobs": torch.zeros(n, device="cuda"), "entropy": torch.zeros(n, device="cuda")}
    if top:
        out["top_logprobs"] = torch.zeros(n, top, device="cuda")
        out["top_ids"] = torch.full((n, top), -1, dtype=torch.int64, device="cuda")
    if case["backward"]:
        dx = torch.empty(n, case["h"], device="cuda")
        dW = torch.zeros(v, case["h"], device="cuda")
    for i, j in _chunks(n, v):
        z = xf[i:j] @ Wf.T
        on = live[i:j]
        largest = z.max(dim=1, keepdim=True).values
        c = (z - largest) * scale
        total = torch.exp(c).sum(dim=1, keepdim=True)
        log_p = c - torch.log(total)
        p = torch.exp(log_p)
        target = t[i:j].clamp(min=0).unsqueeze(1)
        entropy = -(p * log_p).sum(dim=1)
        out["logprobs"][i:j] = torch.where(on, log_p.gather(1, target).squeeze(1), 0.0)
        out["entropy"][i:j] = torch.where(on, entropy, 0.0)
        if top:
            ids, values = _plain_alternatives(x[i:j], W, z, top, v)
            values = (values - largest.double()) * scale - torch.log(total).double()
            out["top_logprobs"][i:j] = torch.where(on[:, None], values.float(), 0.0)
            out["top_ids"][i:j] = torch.where(on[:, None], ids, -1)
        if case["backward"]:
            g = torch.where(on, s["d_logprobs"][i:j], 0.0)[:, None]
            e = torch.where(on, s["d_entropy"][i:j], 0.0)[:, None]
            d = p * (g + e * (log_p + entropy[:, None]))
            d = d.neg_().scatter_add_(1, target, g) * scale
            dx[i:j] = d @ Wf
            dW += d.T @ xf[i:j]
    if case["backward"]:
        out["dx"], out["dW"] = dx.to(x.dtype), dW.to(W.dtype)
    return out


def _plain_distill(s):
    case = s["case"]
    n, v, scale = case["n"], case["v"], 1.0 / case["temperature"]
    xf, Wf, ids = s["x"].float(), s["W"].float(), s["ids"]
    logits = s["teacher"].float() * scale
    there = (ids >= 0) & (logits > -math.inf)
    logits = torch.where(there, logits, -math.inf)
    on = there.any(dim=1, keepdim=True)
    count = on.sum().float().clamp(min=1.0)
    largest = torch.where(on, logits.max(dim=1, keepdim=True).values, 0.0)
    q = torch.exp(logits - largest)
    log_q = logits - largest - torch.log(torch.where(on, q.sum(dim=1, keepdim=True), 1.0))
    q = torch.exp(log_q)
    ids = ids.clamp(min=0)
    losses = torch.zeros(n, dtype=torch.float64, device="cuda")
    if case["backward"]:
        dx = torch.empty(n, case["h"], device="cuda")
        dW = torch.zeros(v, case["h"], device="cuda")
    for i, j in _chunks(n, v):
        z = xf[i:j] @ Wf.T
        c = (z - z.max(dim=1, keepdim=True).values) * scale
        log_p = c - torch.log(torch.exp(c).sum(dim=1, keepdim=True))
        terms = q[i:j] * (log_q[i:j] - log_p.gather(1, ids[i:j]))
        losses[i:j] = torch.where(there[i:j], terms, 0.0).sum(dim=1)
        if case["backward"]:
            d = torch.where(on[i:j], torch.exp(log_p), 0.0)
            d = d.scatter_add_(1, ids[i:j], -q[i:j]) * (case["temperature"] / count)
            dx[i:j] = d @ Wf
            dW += d.T @ xf[i:j]
    out = {"loss": (losses.sum() * case["temperature"] ** 2 / count).float()}
    if case["backward"]:
        out["dx"], out["dW"] = dx.to(s["x"].dtype), dW.to(s["W"].dtype)
    return out


# ---------------------------------------------------------- the framework's calls

def _own_score(s):
    import linear_cross_entropy_token_gb300 as flce
    case = s["case"]
    r = flce.token_logprobs(s["x"], s["W"], s["t"], temperature=case["temperature"],
                            top=min(case["top"], case["v"]), ignore_index=IGNORE, keep_logits=case["keep"])
    out = {"logprobs": r.logprobs, "entropy": r.entropy}
    if case["top"]:
        out["top_logprobs"], out["top_ids"] = r.top_logprobs, r.top_ids
    if case["backward"]:
        out["dx"], out["dW"] = flce.token_logprobs_backward(r, s["x"], s["W"], s["t"], d_logprobs=s["d_logprobs"],
                                                            d_entropy=s["d_entropy"])
    return out


def _own_distill(s):
    import linear_cross_entropy_token_gb300 as flce
    case = s["case"]
    loss, dx, dW = flce.distill(s["x"], s["W"], s["ids"], s["teacher"], temperature=case["temperature"],
                                backward=case["backward"])
    return {"loss": loss, "dx": dx, "dW": dW} if case["backward"] else {"loss": loss}


def run(state):
    if state["case"]["op"] == "score":
        return _own_score(state) if own else _plain_score(state)
    return _own_distill(state) if own else _plain_distill(state)


# ------------------------------------------------------------------- work and exact

def work(case):
    n, h, v, b = case["n"], case["h"], case["v"], BYTES[case["dtype"]]
    moved = (n + v) * h * b
    flops = 2 * n * h * v + 4 * n * v
    if case["op"] == "score":
        moved += n * (8 + 8 + 12 * case["top"]) + (8 * n if case["backward"] else 0)
    else:
        moved += n * case["k"] * (8 + BYTES[case["teacher"]]) + 4
    if case["backward"]:
        moved += (n + v) * h * b
        flops += 4 * n * h * v + 4 * n * v
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    # 64-bit products run at about a trillion operations a second
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    n, v, tau = case["n"], case["v"], case["temperature"]
    x, W = s["x"].double(), s["W"].double()
    step = max(1, (1 << 28) // v)
    dx, dW = torch.zeros_like(x), torch.zeros_like(W)
    out = {}
    if case["op"] == "score":
        live = (s["t"] != IGNORE).nonzero().squeeze(1)
        top = min(case["top"], v)
        out["logprobs"] = torch.zeros(n, dtype=torch.float64, device="cuda")
        out["entropy"] = torch.zeros(n, dtype=torch.float64, device="cuda")
        if top:
            out["top_logprobs"] = torch.zeros(n, top, dtype=torch.float64, device="cuda")
            out["top_ids"] = torch.full((n, top), -1, dtype=torch.int64, device="cuda")
        for rows in live.split(step):
            lp = torch.log_softmax((x[rows] @ W.T) / tau, dim=1)
            t = s["t"][rows, None]
            out["logprobs"][rows] = lp.gather(1, t).squeeze(1)
            p = lp.exp()
            entropy = -(p * lp).sum(1, keepdim=True)
            out["entropy"][rows] = entropy.squeeze(1)
            if top:
                best = torch.sort(lp, dim=1, descending=True, stable=True)
                out["top_logprobs"][rows], out["top_ids"][rows] = best.values[:, :top], best.indices[:, :top]
            if case["backward"]:
                a, b = s["d_logprobs"].double()[rows, None], s["d_entropy"].double()[rows, None]
                d = -a * p - b * p * (lp + entropy)
                d.scatter_add_(1, t, a)
                d /= tau
                dx[rows] = d @ W
                dW += d.mT @ x[rows]
    else:
        teacher = s["teacher"].double() / tau
        teacher[s["ids"] < 0] = -math.inf
        live = torch.isfinite(teacher).any(dim=1).nonzero().squeeze(1)
        count = max(live.numel(), 1)
        loss = torch.zeros((), dtype=torch.float64, device="cuda")
        for rows in live.split(step):
            lp = torch.log_softmax((x[rows] @ W.T) / tau, dim=1)
            q = torch.softmax(teacher[rows], dim=1)
            target = torch.zeros_like(lp)
            target.scatter_add_(1, s["ids"][rows].clamp(min=0), q)
            log_q = torch.where(q > 0, q.log(), torch.zeros_like(q))
            loss += ((q * log_q).sum() - (target * lp).sum()) * tau * tau / count
            if case["backward"]:
                d = (lp.exp() - target) * (tau / count)
                dx[rows] = d @ W
                dW += d.mT @ x[rows]
        out["loss"] = loss
    if case["backward"]:
        out["dx"], out["dW"] = dx, dW
    return out
