"""Cases, plain forms and 64-bit references of the expert-routing and gradient
operators: `route`, `route_bwd`, `grad_norm` and `grad_clip`.

Each operator has a plain form in elementary torch operations (`own` false)
and the calls of this package (`own` true) on the same inputs.  The formulas:

  route      p = softmax(l) or sigmoid(l) per token; the selection score is
             s = p + bias.  With groups, a group's score is the sum of its
             best `group_top` selection scores; the best `topk_groups` groups
             stay open.  The topk largest s of the open experts are taken in
             descending order, ties to the lower expert (and the lower group).
             An expert with a logit of -inf is closed.  gate = scale * p, with
             renorm scale * p / (sum of the chosen p).  counts[e] = number of
             (token, slot) pairs routed to e.
  route_bwd  the gradient of the gates with respect to the logits, the choice
             of experts held fixed.
  grad_norm  sqrt(sum of x^2) of every tensor and of all of them together.
  grad_clip  grad_norm, then x * min(1, max_norm / (norm + 1e-6)).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ESIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases
def _route(name, op, T, E, k, score, dtype, *, bias=False, groups=(1, 1, 1), renorm=True, scale=1.0, pad=0,
           closed=0):
    return {"name": name, "op": op, "tokens": T, "experts": E, "topk": k, "score": score, "dtype": dtype,
            "bias": bias, "n_groups": groups[0], "topk_groups": groups[1], "group_top": groups[2],
            "renorm": renorm, "scale": scale, "pad": pad, "closed": closed}


def listed():
    return [
        # one token of one sequence: the launch and the chain of k choices are all there is
        _route("route_one_token", "route", 1, 256, 8, "sigmoid", "fp32", bias=True, groups=(8, 4, 2), scale=2.5),
        # one decoding step of a batch of sequences, on the 128 experts top-8 of the framework's layer
        _route("route_batch", "route", 96, 128, 8, "softmax", "bf16"),
        # the framework's own expert layer: 2048 tokens, 128 experts, top-8
        _route("route_layer", "route", 2048, 128, 8, "softmax", "bf16"),
        # a long prompt (or a training step's micro-batch) with the bias-balanced, group-limited router
        _route("route_prompt", "route", 32768, 256, 8, "sigmoid", "fp32", bias=True, groups=(8, 4, 2), scale=2.5),
        # ragged: 60 experts, an odd number of tokens, rows inside a wider projection, three experts switched off
        _route("route_ragged", "route", 40009, 60, 4, "softmax", "fp16", renorm=False, pad=5, closed=3),
        # gradients of the same routers: the layer's, the long micro-batch's, the ragged one's
        _route("route_bwd_layer", "route_bwd", 2048, 128, 8, "softmax", "bf16"),
        _route("route_bwd_long", "route_bwd", 32768, 256, 8, "sigmoid", "fp32", bias=True, groups=(8, 4, 2),
               scale=2.5),
        _route("route_bwd_ragged", "route_bwd", 40009, 60, 4, "softmax", "fp16", renorm=False, pad=5, closed=3),
        # the router's own gradient and a few vectors: latency
        {"name": "grad_norm_router", "op": "grad_norm", "set": "router", "hidden": 4096, "experts": 128, "inter": 1536},
        # every weight gradient of the framework's expert layer (8 ranks x gate, up, down, and the router)
        {"name": "grad_norm_layer", "op": "grad_norm", "set": "layer", "hidden": 4096, "experts": 128, "inter": 1536},
        # many small tensors of odd sizes and mixed types: norms, biases, adapters
        {"name": "grad_clip_many", "op": "grad_clip", "set": "many", "tensors": 230, "longest": 30000,
         "max_norm": 1.0},
        # the weight gradients of a layer of 32 experts
        {"name": "grad_clip_layer", "op": "grad_clip", "set": "layer", "hidden": 4096, "experts": 32, "inter": 1536,
         "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "route_bwd", "grad_norm", "grad_clip"])
    if op in ("route", "route_bwd"):
        E = _log_int(rng, 8, 512)
        if rng.random() < 0.5:
            E = max(8, E // 8 * 8)
        T = _log_int(rng, 1, min(65536, (32768 * 256) // E))
        k = min(E, _log_int(rng, 1, 16))
        groups = (1, 1, 1)
        opts = [g for g in (2, 3, 4, 5, 6, 8, 16) if E % g == 0 and E // g >= 2]
        if opts and rng.random() < 0.5:
            g = rng.choice(opts)
            need = -(-k // (E // g))
            groups = (g, rng.randint(need, g), rng.choice([1, 2]))
        c = _route("", op, T, E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "fp16", "fp32"]),
                   bias=rng.random() < 0.5, groups=groups, renorm=rng.random() < 0.6,
                   scale=rng.choice([1.0, 1.0, 2.5, 0.5]), pad=rng.choice([0, 0, 0, 3, 8]),
                   closed=rng.choice([0, 0, 0, 1, 2]) if E > k + 8 and groups[0] == 1 else 0)
    else:
        kind = rng.choice(["many", "layer", "router"])
        c = {"op": op, "set": kind}
        if kind == "many":
            c.update(tensors=_log_int(rng, 1, 400), longest=_log_int(rng, 1, 200000))
        elif kind == "layer":
            c.update(hidden=256 * rng.randint(1, 16), experts=8 * rng.randint(1, 4), inter=128 * rng.randint(1, 12))
        else:
            c.update(hidden=_log_int(rng, 33, 8192), experts=_log_int(rng, 8, 256), inter=_log_int(rng, 8, 4096))
        if op == "grad_clip":
            c["max_norm"] = rng.choice([0.1, 1.0, 1.0, 1e6])
    c.pop("name", None)
    return c


def _grad_shapes(case):
    """(elements, dtype name) of every tensor of a gradient set."""
    if case["set"] == "router":
        return [(case["hidden"] * case["experts"], "fp32"), (case["experts"], "fp32"), (case["hidden"], "fp32"),
                (case["hidden"], "bf16"), (case["inter"], "bf16")]
    if case["set"] == "layer":
        per = case["experts"] // 8 * case["hidden"] * case["inter"]
        return [(per, "bf16")] * 24 + [(case["hidden"] * case["experts"], "fp32")]
    names = ["bf16", "fp32", "bf16", "fp16"]
    # sizes between 1 and `longest`, spread over their logarithm by a fixed low-discrepancy sequence
    return [(max(1, int(case["longest"] ** ((i * 0.6180339887498949 + 0.5) % 1.0))), names[i % 4])
            for i in range(case["tensors"])]


def work(case):
    if case["op"] in ("route", "route_bwd"):
        T, E, k, es = case["tokens"], case["experts"], case["topk"], ESIZE[case["dtype"]]
        if case["op"] == "route":
            return {"bytes": T * E * es + T * k * 8 + E * 4 + (E * 4 if case["bias"] else 0), "flops": 4 * T * E}
        read = T * k * 12  # idx, gate, dgate
        if case["score"] == "softmax" and not case["renorm"]:
            read += T * E * es          # every logit of a row takes part
        elif case["score"] == "sigmoid":
            read += T * k * es          # the chosen logits
        return {"bytes": read + T * E * es, "flops": 6 * T * k + (4 * T * E if read > T * k * 12 + T * k * es else 0)}
    n = sum(c for c, _ in _grad_shapes(case))
    b = sum(c * ESIZE[d] for c, d in _grad_shapes(case))
    return {"bytes": b + 4, "flops": 2 * n} if case["op"] == "grad_norm" else {"bytes": 2 * b + 4, "flops": 3 * n}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)


def _route_inputs(case, seed):
    g = _gen(seed)
    T, E, k = case["tokens"], case["experts"], case["topk"]
    dt = DTYPES[case["dtype"]]
    # token-dependent logits on top of each expert's own popularity
    wide = torch.randn(T, E + case["pad"], generator=g, device="cuda")
    wide[:, :E] = wide[:, :E] * 1.3 + 0.5 * torch.randn(E, generator=g, device="cuda")
    if case["closed"]:
        wide[:, torch.randperm(E, generator=g, device="cuda")[:case["closed"]]] = -math.inf
    wide = wide.to(dt)
    st = {"logits": wide[:, :E]}
    # the balance bias is a sum of steps of 0.001
    st["bias"] = (torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * 0.001) if case["bias"] else None
    if case["op"] == "route_bwd":
        st["topk_idx"], st["topk_gate"], _ = _plain_route(case, st["logits"], st["bias"])
        st["dgate"] = torch.randn(T, k, generator=g, device="cuda") * 0.01
    return st


def _buckets(case):
    """One flat buffer per type and the gradients as consecutive views of it
    (a small odd-sized gradient then starts at any element), or for the layer
    a tensor of its own per gradient."""
    shapes = _grad_shapes(case)
    if case["set"] != "many":
        xs = [torch.empty(n, dtype=DTYPES[d], device="cuda") for n, d in shapes]
        return xs, xs
    flat = {d: torch.empty(sum(n for n, t in shapes if t == d), dtype=DTYPES[d], device="cuda")
            for d in sorted({t for _, t in shapes})}
    at = dict.fromkeys(flat, 0)
    views = []
    for n, d in shapes:
        views.append(flat[d][at[d]:at[d] + n])
        at[d] += n
    return list(flat.values()), views


def _grad_inputs(case, seed):
    g = _gen(seed)
    flat, views = _buckets(case)
    for i, x in enumerate(views):
        x.normal_(0.0, 10.0 ** (-4 + i % 3), generator=g)
        if i % 11 == 7:
            x.zero_()  # an expert or a vector that no token reached
    return {"grads": views, "buckets": flat}


def prepare(case, seed):
    st = {"case": case}
    if case["op"] in ("route", "route_bwd"):
        st.update(_route_inputs(case, seed))
    else:
        st.update(_grad_inputs(case, seed))
    if own:
        import comm_persistent_gemm_gb300 as K
        st["K"] = K
        if case["op"] in ("route", "route_bwd"):
            T, E, k = case["tokens"], case["experts"], case["topk"]
            st["router"] = K.router(topk=k, score=K.SCORE_SIGMOID if case["score"] == "sigmoid" else K.SCORE_SOFTMAX,
                                    n_groups=case["n_groups"], topk_groups=case["topk_groups"],
                                    group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
            if case["op"] == "route":
                st["topk_idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
                st["topk_gate"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
                st["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
                st["ws"] = K.route_workspace(E)
            else:
                st["dlogits"] = torch.empty(T, E, dtype=DTYPES[case["dtype"]], device="cuda")
        else:
            st["out_buckets"], outs = _buckets(case) if case["op"] == "grad_clip" else (None, None)
            st["set"] = K.GradSet(st["grads"], outs)
            st["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
            st["tensor_norms"] = torch.empty(len(st["grads"]), dtype=torch.float32, device="cuda")
            st["ws"] = K.grad_workspace(st["set"])
    return st


# ------------------------------------------------------------- the plain forms
def _plain_scores(case, logits, dt):
    x = logits.to(dt)
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _take_first(s):
    """The largest value of each row and its lowest index."""
    m = s.amax(1, keepdim=True)
    col = torch.arange(s.shape[1], device=s.device)
    return torch.where(s == m, col, s.shape[1]).amin(1)


def _plain_route(case, logits, bias):
    T, E, k = case["tokens"], case["experts"], case["topk"]
    G, GK = case["n_groups"], case["topk_groups"]
    # scores next to one another decide the choice: 64 bits
    s = _plain_scores(case, logits, torch.float64)
    if bias is not None:
        s = s + bias.double()
    s = torch.where(torch.isneginf(logits), -math.inf, s)
    if G > 1:
        gs = s.reshape(T * G, E // G).clone()
        score = torch.zeros(T * G, dtype=torch.float64, device=s.device)
        for i in range(case["group_top"]):
            j = _take_first(gs)[:, None]
            v = gs.gather(1, j)[:, 0]
            score = score + (v if i == 0 else torch.where(torch.isneginf(v), 0.0, v))
            gs.scatter_(1, j, -math.inf)
        score = score.reshape(T, G)
        keep = torch.zeros(T, G, dtype=torch.bool, device=s.device)
        for _ in range(GK):
            j = _take_first(torch.where(keep, -math.inf, score))[:, None]
            keep.scatter_(1, j, True)
        s = torch.where(keep.repeat_interleave(E // G, 1), s, -math.inf)
    idx = torch.empty(T, k, dtype=torch.int64, device=s.device)
    for i in range(k):
        idx[:, i] = _take_first(s)
        s.scatter_(1, idx[:, i:i + 1], -math.inf)
    p = _plain_scores(case, logits, torch.float32).gather(1, idx)
    gate = p / p.sum(1, keepdim=True) if case["renorm"] else p
    counts = (idx.reshape(-1, 1) == torch.arange(E, device=s.device)).sum(0) if T * k * E <= 1 << 22 else \
        torch.zeros(E, dtype=torch.int64, device=s.device).index_add_(0, idx.reshape(-1), torch.ones_like(idx.reshape(-1)))
    return idx.int(), gate * case["scale"], counts.int()


def _plain_route_bwd(case, st):
    logits, idx, dg = st["logits"], st["topk_idx"].long(), st["dgate"]
    p = _plain_scores(case, logits, torch.float32)
    pk = p.gather(1, idx)
    if case["renorm"]:
        S = pk.sum(1, keepdim=True)
        dpk = case["scale"] * (dg - (dg * pk).sum(1, keepdim=True) / S) / S
    else:
        dpk = case["scale"] * dg
    if case["score"] == "sigmoid":
        x = logits.gather(1, idx).float()
        dl = torch.zeros_like(p).scatter_(1, idx, dpk * pk / (1.0 + torch.exp(x)))
    elif case["renorm"]:
        dl = torch.zeros_like(p).scatter_(1, idx, dpk * pk)  # the sum of dp * p is zero
    else:
        dl = p * (torch.zeros_like(p).scatter_(1, idx, dpk) - (dpk * pk).sum(1, keepdim=True))
    return dl.to(logits.dtype)


def _plain_squares(grads):
    """Sum of squares of every tensor: long sums, 64 bits."""
    return torch.stack([x.float().square().sum(dtype=torch.float64) for x in grads])


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        K = state["K"]
        if op == "route":
            K.route(state["logits"], state["router"], state["topk_idx"], state["topk_gate"], bias=state["bias"],
                    expert_counts=state["counts"], ws=state["ws"])
            return {"idx": state["topk_idx"], "gate": state["topk_gate"], "counts": state["counts"]}
        if op == "route_bwd":
            K.route_bwd(state["logits"], state["router"], state["topk_idx"], state["topk_gate"], state["dgate"],
                        state["dlogits"])
            return {"dlogits": state["dlogits"]}
        if op == "grad_norm":
            K.grad_norm(state["set"], state["norm"], state["ws"], tensor_norms=state["tensor_norms"])
            return {"norm": state["norm"], "tensor_norms": state["tensor_norms"]}
        K.grad_clip(state["set"], case["max_norm"], state["norm"], state["ws"])
        return {"norm": state["norm"], "grads": state["out_buckets"]}
    if op == "route":
        idx, gate, counts = _plain_route(case, state["logits"], state["bias"])
        return {"idx": idx, "gate": gate, "counts": counts}
    if op == "route_bwd":
        return {"dlogits": _plain_route_bwd(case, state)}
    sq = _plain_squares(state["grads"])
    norm = torch.sqrt(sq.sum())
    if op == "grad_norm":
        return {"norm": norm.float().reshape(1), "tensor_norms": torch.sqrt(sq).float()}
    coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1), "grads": [(x.float() * coef).to(x.dtype) for x in state["buckets"]]}


# -------------------------------------------------- the definitions in 64 bits
def _exact_choice(case, l, bias):
    """Chosen experts per token by stable descending sorts."""
    T, E = l.shape
    k, G, GK = case["topk"], case["n_groups"], case["topk_groups"]
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    if bias is not None:
        s = s + bias.double()
    s = s.masked_fill(torch.isneginf(l), -math.inf)
    if G > 1:
        best = torch.sort(s.view(T, G, E // G), dim=2, descending=True, stable=True).values[:, :, :case["group_top"]]
        score = best[:, :, 0].clone()
        for i in range(1, best.shape[2]):
            score += torch.nan_to_num(best[:, :, i], neginf=0.0)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(G, device=l.device).expand(T, G))
        closed = (rank >= GK)[:, :, None].expand(T, G, E // G).reshape(T, E)
        s = s.masked_fill(closed, -math.inf)
    return torch.sort(s, dim=1, descending=True, stable=True).indices[:, :k]


def exact(case, seed):
    if case["op"] in ("route", "route_bwd"):
        st = _route_inputs(case, seed)
        l = st["logits"].double()
        k = case["topk"]
        chosen = _exact_choice(case, l, st["bias"]) if case["op"] == "route" else st["topk_idx"].long()
        l = l.clone().requires_grad_(True)
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        gate = p.gather(1, chosen)
        if case["renorm"]:
            gate = gate / gate.sum(1, keepdim=True)
        gate = gate * case["scale"]
        if case["op"] == "route_bwd":
            (dl,) = torch.autograd.grad(gate, l, st["dgate"].double())
            return {"dlogits": dl}
        return {"idx": chosen.int(), "gate": gate.detach(),
                "counts": torch.bincount(chosen.reshape(-1), minlength=case["experts"]).int()}
    st = _grad_inputs(case, seed)
    each = []
    for x in st["grads"]:
        parts = [part.double() for part in x.split(1 << 26)]
        each.append(math.fsum(float(torch.dot(d, d)) for d in parts))
    norm = math.sqrt(math.fsum(each))
    n = torch.tensor([norm], dtype=torch.float64, device="cuda")
    if case["op"] == "grad_norm":
        return {"norm": n, "tensor_norms": torch.tensor(each, dtype=torch.float64, device="cuda").sqrt()}
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norm": n, "grads": [x.double() * coef for x in st["buckets"]]}
