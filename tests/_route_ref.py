"""The routing and clipping operators restated in 64 bits (torch double on the
CPU), one definition per function, for the tests."""
import math

import torch


def log_softmax(x):
    """Relative to the row's largest value, so that huge equal values keep
    their share; a row of -inf alone stays -inf."""
    m = x.amax(1, keepdim=True)
    m = torch.where(torch.isneginf(m), 0.0, m)
    y = x - m
    return y - torch.where(torch.isneginf(y).all(1, keepdim=True), 0.0, torch.logsumexp(y, 1, keepdim=True))


def log_p(x, score):
    """log of the scores; -inf logits give -inf."""
    x = x.double()
    if score == "sigmoid":
        return -torch.nn.functional.softplus(-x, threshold=40)  # log(1 + e^y) = y to 64 bits beyond 40
    return log_softmax(x)


def route_ref(logits, *, topk, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=True,
              scale=1.0):
    """(idx, gate, open, counts) of rows without NaN or +inf."""
    T, E = logits.shape
    x = logits.double()
    closed = torch.isneginf(x)
    s = torch.exp(log_p(torch.where(closed, -math.inf, x), score))
    s = torch.where(closed, 0.0, s)  # a softmax row of -inf alone has no scores
    if bias is not None:
        s = s + bias.double()
        closed = closed | torch.isneginf(s) | torch.isnan(s)
    # without a bias the order of the scores is the order of the logits
    key = torch.where(closed, -math.inf, x if bias is None else s)
    if topk_groups < n_groups:
        gk = key if group_top == 1 else torch.where(closed, -math.inf, s)
        best = torch.sort(gk.view(T, n_groups, -1), dim=2, descending=True).values
        gscore = best[:, :, 0].clone()
        if group_top == 2:
            gscore += torch.where(torch.isneginf(best[:, :, 1]), 0.0, best[:, :, 1])
        order = torch.sort(gscore, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros(T, n_groups, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // n_groups, 1), key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    is_open = ~torch.isneginf(key.gather(1, idx))
    gate = gates_ref(logits, idx, is_open, score=score, renorm=renorm, scale=scale)
    return idx, gate, is_open, torch.bincount(idx.reshape(-1), minlength=E)


def gates_ref(logits, idx, is_open, *, score, renorm, scale):
    lp = log_p(logits, score).gather(1, idx)
    lp = torch.where(is_open, lp, -math.inf)
    if renorm:
        lp = log_softmax(lp)
    return torch.where(is_open, scale * torch.exp(lp), 0.0)


def route_bwd_ref(logits, idx, is_open, dgate, *, score, renorm, scale):
    """Gradient of gates_ref by automatic differentiation, and per element
    the magnitude that rounding errors are relative to."""
    x = logits.double().clone()
    closed = torch.isneginf(x)
    x[closed] = 0.0
    x.requires_grad_(True)
    xs = torch.where(closed, -math.inf, x)
    p = torch.sigmoid(xs) if score == "sigmoid" else torch.softmax(xs, 1)
    if score == "softmax" and renorm:
        # the row's sum cancels: gates are the softmax of the chosen logits
        xk = torch.where(is_open, xs.gather(1, idx), -math.inf)
        pk = torch.exp(xk - xk.detach().amax(1, keepdim=True))
    else:
        pk = p.gather(1, idx)
    pk = torch.where(is_open, pk, 0.0)
    S = pk.sum(1, keepdim=True)
    g = scale * (pk / S if renorm else pk)
    g = torch.where(is_open, g, 0.0)
    dg = torch.where(is_open, dgate.double(), 0.0)
    (dl,) = torch.autograd.grad((g * dg).sum(), x)
    dl = torch.nan_to_num(dl, nan=0.0)
    g, p = g.detach(), p.detach()
    A = (g * dg.abs()).sum(1, keepdim=True)
    mag = torch.zeros_like(dl).scatter_(1, idx, g * (dg.abs() + (A / scale if renorm else 0.0)))
    if score == "softmax" and not renorm:
        mag = mag + torch.nan_to_num(p, nan=0.0) * A
    return dl, mag
