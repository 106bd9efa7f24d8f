"""GPU parity of the routing operators against their definition in 64 bits.

Indices and counts are whole numbers and must be equal.  Tolerances, in units
of u = 2^-24 (half a step of fp32):
  gates   : exponential, sums of up to E/32 + 5 terms per lane and tree level,
            division, scale and product: (32 + E/32) u, and the rounding of the
            exponent's argument, whose size is at most the row's range R: 2 R u.
  dlogits : the same error on each factor of g (|dg| + D) (mag), twice (the gates are
            the forward's own), plus one rounding to the logits' type
            (eps / 2 of the value; fp16 below 2^-14: half of 2^-24)."""
import math

import pytest
import torch

from _helpers import kosmos
from _route_ref import gates_ref, route_bwd_ref, route_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kosmos()


def make_router(K, c):
    return K.router(topk=c["topk"], score=K.SCORE_SIGMOID if c["score"] == "sigmoid" else K.SCORE_SOFTMAX,
                    n_groups=c.get("n_groups", 1), topk_groups=c.get("topk_groups", 1),
                    group_top=c.get("group_top", 1), renorm=c.get("renorm", True), scale=c.get("scale", 1.0))


def run_route(K, logits, c, bias=None, counts=True, ws=None):
    T, E = logits.shape
    idx = torch.full((T, c["topk"]), -7, dtype=torch.int32, device="cuda")
    gate = torch.full((T, c["topk"]), math.nan, device="cuda")
    cnt = torch.full((E,), -7, dtype=torch.int32, device="cuda") if counts else None
    if counts and ws is None:
        ws = K.route_workspace(E)
    K.route(logits, make_router(K, c), idx, gate, bias=bias, expert_counts=cnt, ws=ws)
    return idx, gate, cnt


def ref_args(c):
    return {k: v for k, v in c.items() if k in ("topk", "score", "n_groups", "topk_groups", "group_top", "renorm",
                                                "scale")}


def row_range(x):
    f = x[torch.isfinite(x)]
    return float(f.max() - f.min()) if f.numel() else 0.0


def check_route(K, logits, c, bias=None):
    """Runs and compares; returns what the backward test needs."""
    T, E = logits.shape
    idx, gate, cnt = run_route(K, logits, c, bias)
    x = logits.detach().float().cpu()
    ri, rg, ro, rc = route_ref(x, bias=bias.cpu() if bias is not None else None, **ref_args(c))
    gi = idx.cpu().long()
    assert torch.equal(gi, ri), f"rows {torch.where((gi != ri).any(1))[0][:8].tolist()}"
    assert torch.equal(cnt.cpu().long(), rc)
    tol = (32 + E / 32 + 2 * min(row_range(x), 104.0)) * U
    err = (gate.cpu().double() - rg).abs()
    lim = tol * rg + c.get("scale", 1.0) * 2.0 ** -126
    assert bool((err <= lim).all()), float((err - lim).max())
    return gi, gate, ro


CASES = [
    # T, E, topk, score, dtype, extra
    (1, 1, 1, "softmax", "fp32", {}),
    (1, 2, 2, "sigmoid", "bf16", {"renorm": False}),
    (1, 256, 8, "sigmoid", "fp32", {"bias": 1, "n_groups": 8, "topk_groups": 4, "group_top": 2, "scale": 2.5}),
    (3, 7, 3, "softmax", "fp16", {"pad": 1}),
    (33, 8, 2, "softmax", "bf16", {}),
    (65, 60, 4, "softmax", "fp16", {"renorm": False, "pad": 5}),
    (129, 64, 6, "softmax", "bf16", {"bias": 1}),
    (200, 65, 16, "sigmoid", "bf16", {"bias": 1, "pad": 7}),
    (513, 96, 5, "sigmoid", "fp16", {"n_groups": 32, "topk_groups": 3, "group_top": 1, "renorm": False}),
    (500, 128, 8, "softmax", "bf16", {"scale": 0.5}),
    (700, 160, 6, "softmax", "fp32", {"n_groups": 8, "topk_groups": 3, "group_top": 1, "bias": 1, "scale": 16.0}),
    (300, 160, 6, "softmax", "bf16", {"n_groups": 8, "topk_groups": 3, "group_top": 2, "renorm": False}),
    (1000, 255, 7, "sigmoid", "fp32", {"n_groups": 5, "topk_groups": 2, "group_top": 2, "bias": 1}),
    (2048, 256, 8, "sigmoid", "bf16", {"n_groups": 8, "topk_groups": 4, "group_top": 2, "bias": 1}),
    (5000, 256, 8, "sigmoid", "fp16", {"n_groups": 16, "topk_groups": 5, "group_top": 2}),
    (777, 384, 16, "softmax", "fp32", {}),
    (321, 512, 10, "softmax", "bf16", {"renorm": False, "bias": 1}),
    (257, 1000, 9, "sigmoid", "fp32", {"n_groups": 10, "topk_groups": 10, "bias": 1, "pad": 24}),
    (99, 1024, 16, "softmax", "fp16", {"n_groups": 32, "topk_groups": 8, "group_top": 2, "bias": 1}),
    (40, 1024, 1, "sigmoid", "bf16", {"pad": 8, "renorm": False}),
]


def case_inputs(i):
    T, E, k, score, dtype, extra = CASES[i]
    g = torch.Generator().manual_seed(100 + i)
    extra = dict(extra)
    pad, has_bias = extra.pop("pad", 0), extra.pop("bias", 0)
    wide = (torch.randn(T, E + pad, generator=g) * 1.5).to(DT[dtype]).cuda()
    bias = (torch.randint(-60, 61, (E,), generator=g).float() * 0.001).cuda() if has_bias else None
    return wide[:, :E], {"topk": k, "score": score, **extra}, bias, g


@pytest.mark.parametrize("i", range(len(CASES)))
def test_route_and_gradient(K, i):
    logits, c, bias, g = case_inputs(i)
    T, E = logits.shape
    gi, gate, is_open = check_route(K, logits, c, bias)
    dgate = torch.randn(T, c["topk"], generator=g)
    pad = CASES[i][5].get("pad", 0)
    out = torch.full((T, E + pad), 7.0, dtype=logits.dtype, device="cuda")
    K.route_bwd(logits, make_router(K, c), gi.int().cuda(), gate, dgate.cuda(), out[:, :E])
    assert bool((out[:, E:] == 7.0).all())  # nothing beyond the rows
    args = {"score": c["score"], "renorm": c.get("renorm", True), "scale": c.get("scale", 1.0)}
    x = logits.float().cpu()
    dl, mag = route_bwd_ref(x, gi, is_open, dgate, **args)
    tol = 2 * (32 + E / 32 + 2 * row_range(x)) * U
    lim = tol * mag + torch.finfo(logits.dtype).eps / 2 * dl.abs() * (1 + 2 ** -6) + \
        (2.0 ** -25 if logits.dtype == torch.float16 else 1e-38)
    err = (out[:, :E].cpu().double() - dl).abs()
    assert bool((err <= lim).all()), float((err - lim).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(K, score, renorm):
    """fp32 gradients against central differences of the 64-bit gates.  The
    differences' own error: h^2 times a third derivative of order 1, and
    2^-52 / h: both under 1e-9 for h = 1e-5."""
    T, E, k, h = 5, 12, 4, 1e-5
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, E, generator=g)
    dgate = torch.randn(T, k, generator=g)
    c = {"topk": k, "score": score, "renorm": renorm, "scale": 1.5}
    gi, gate, is_open = check_route(K, x.cuda(), c)
    out = torch.empty(T, E, device="cuda")
    K.route_bwd(x.cuda(), make_router(K, c), gi.int().cuda(), gate, dgate.cuda(), out)
    num = torch.zeros(T, E, dtype=torch.float64)
    for e in range(E):
        d = torch.zeros(T, E, dtype=torch.float64)
        d[:, e] = h
        f = [(gates_ref(x.double() + s * d, gi, is_open, score=score, renorm=renorm, scale=1.5) *
              dgate.double()).sum(1) for s in (1, -1)]
        num[:, e] = (f[0] - f[1]) / (2 * h)
    _, mag = route_bwd_ref(x, gi, is_open, dgate, score=score, renorm=renorm, scale=1.5)
    err = (out.cpu().double() - num).abs()
    assert bool((err <= 2 * (33 + 2 * row_range(x)) * U * mag + U * num.abs() + 2e-9).all()), float(err.max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["plain", "bias", "groups", "groups_bias"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_masks(K, score, kind, dtype):
    """Equal logits, signed zeros, -inf and lowest-value masks, rows with fewer
    open experts than topk, rows with none, saturated scores."""
    E, k = 48, 6
    g = torch.Generator().manual_seed(11)
    low = torch.finfo(DT[dtype]).min
    rows = [torch.zeros(E), torch.full((E,), low), torch.full((E,), -math.inf)]
    z = torch.zeros(E); z[::2] = -0.0; rows.append(z)
    r = torch.randint(-1, 2, (E,), generator=g).float(); rows.append(r)           # many ties
    m = torch.randn(E, generator=g); m[torch.randperm(E, generator=g)[:E - 3]] = -math.inf; rows.append(m)  # 3 open
    m = torch.randn(E, generator=g); m[:40] = low; rows.append(m)
    m = torch.full((E,), -math.inf); m[17] = -3.0; rows.append(m)
    m = torch.full((E,), low); m[5] = -math.inf; rows.append(m)
    rows.append(torch.randn(E, generator=g) * 12)                                  # wide
    rows.append(torch.arange(E).float() / 8 - 20)                                  # small sigmoids
    m = torch.randn(E, generator=g); m[8:32] = -math.inf; rows.append(m)          # whole groups closed
    x = torch.stack(rows).to(DT[dtype])
    c = {"topk": k, "score": score}
    if kind in ("groups", "groups_bias"):
        c.update(n_groups=6, topk_groups=2, group_top=2 if kind == "groups_bias" else 1)
    bias = None
    if kind in ("bias", "groups_bias"):
        bias = torch.randint(-3, 4, (E,), generator=g).float() * 0.125
        bias[7] = -math.inf
        bias = bias.cuda()
    for renorm in (True, False):
        c["renorm"] = renorm
        gi, gate, is_open = check_route(K, x.cuda(), c, bias)
        dgate = torch.randn(len(rows), k, generator=g)
        out = torch.empty(len(rows), E, dtype=DT[dtype], device="cuda")
        K.route_bwd(x.cuda(), make_router(K, c), gi.int().cuda(), gate, dgate.cuda(), out)
        xf = x.float()
        f = xf.clone(); f[f <= low] = 0
        assert bool(torch.isfinite(out).all())
        for t in range(len(rows)):
            if not bool(is_open[t].any()):
                assert bool((out[t] == 0).all())  # no gate, no gradient
        # closed picks take no gradient
        picked = out.cpu().float().gather(1, gi)
        if not (score == "softmax" and not renorm):
            assert bool((picked[~is_open] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_next_to_one_another(K, score):
    """Every selection score of a row within a few fp32 steps of the others:
    the order is that of the 64-bit scores."""
    T, E = 64, 80
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, E, generator=g)
    # per row: bias is one vector, so make the logits fit it instead
    bias = (torch.rand(E, generator=g) * 0.4).float()
    s = 0.75
    want = s - bias.double()
    xs = torch.log(want / (1 - want)) if score == "sigmoid" else torch.log(want)
    x = xs.float().repeat(T, 1)
    x = x + torch.randint(-2, 3, (T, E), generator=g) * x.abs() * 2.0 ** -23  # a few steps apart
    for k, kw in ((8, {}), (16, {"n_groups": 8, "topk_groups": 4, "group_top": 2})):
        check_route(K, x.cuda(), {"topk": k, "score": score, **kw}, bias.cuda())


@pytest.mark.parametrize("bits", [23, 30, 37, 43, 49])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_next_to_one_another(K, score, bits):
    """A few distinct logits and biases that are multiples of 2^-bits: order,
    borders and groups are decided by differences of that size.  The
    multiples add to the scores exactly in 64 bits, so that groups whose sums
    agree are ties there too."""
    T, E = 40, 96
    g = torch.Generator().manual_seed(9)
    x = torch.randint(0, 3, (T, E), generator=g).float() * 0.5
    bias = torch.randint(-20, 21, (E,), generator=g).float() * 2.0 ** -bits
    for k, kw in ((7, {}), (8, {"n_groups": 8, "topk_groups": 3, "group_top": 2}),
                  (12, {"n_groups": 12, "topk_groups": 5, "group_top": 1})):
        check_route(K, x.cuda(), {"topk": k, "score": score, **kw}, bias.cuda())


# T, E, topk, groups: so many tokens that a warp takes two, four, eight rows at once
SHARED = [
    (4001, 256, 8, (8, 4, 2)),
    (7003, 40, 16, (1, 1, 1)),
    (10007, 256, 8, (8, 4, 2)),
    (10007, 128, 6, (16, 3, 1)),
    (10007, 60, 8, (1, 1, 1)),
    (12001, 500, 10, (1, 1, 1)),
    (20011, 60, 4, (1, 1, 1)),
    (20011, 8, 2, (1, 1, 1)),
    (20011, 3, 3, (1, 1, 1)),
    (20011, 1, 1, (1, 1, 1)),
    (40009, 100, 4, (1, 1, 1)),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,pad", [(37, 8, 2, 0), (501, 16, 9, 3), (2003, 31, 16, 0), (160003, 8, 2, 0),
                                       (160003, 57, 6, 1)])
def test_gradient_of_gates_that_are_not_renormalised(K, T, E, k, pad, dtype):
    """Few experts, where many rows share a warp, with masked rows among them."""
    g = torch.Generator().manual_seed(T + E)
    wide = torch.randn(T, E + pad, generator=g)
    wide[::13, : E - 1] = -math.inf
    wide[::29] = -math.inf
    logits = wide.to(DT[dtype]).cuda()[:, :E]
    x = logits.float().cpu()
    c = {"topk": k, "score": "softmax", "renorm": False, "scale": 0.75}
    gi, gate, is_open = check_route(K, logits, c)
    dgate = torch.randn(T, k, generator=g)
    out = torch.full((T, E + pad), 7.0, dtype=logits.dtype, device="cuda")
    K.route_bwd(logits, make_router(K, c), gi.int().cuda(), gate, dgate.cuda(), out[:, :E])
    assert bool((out[:, E:] == 7.0).all())
    dl, mag = route_bwd_ref(x, gi, is_open, dgate, score="softmax", renorm=False, scale=0.75)
    tol = 2 * (32 + E / 32 + 2 * row_range(x)) * U
    lim = tol * mag + torch.finfo(logits.dtype).eps / 2 * dl.abs() * (1 + 2 ** -6) + \
        (2.0 ** -25 if logits.dtype == torch.float16 else 1e-38)
    err = (out[:, :E].cpu().double() - dl).abs()
    assert bool((err <= lim).all()), float((err - lim).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("has_bias", [False, True])
@pytest.mark.parametrize("i", range(len(SHARED)))
def test_rows_that_share_a_warp(K, i, has_bias, score, dtype):
    """Ordinary rows next to masked ones, ties, scores that differ by 2^-30 and
    (compared with the run without them) rows with NaN: each is decided as if
    it were alone.  Groups scored by sums have no rows of ties under a bias:
    whether such sums are equal would depend on their roundings in 64 bits."""
    T, E, k, (n_groups, topk_groups, group_top) = SHARED[i]
    g = torch.Generator().manual_seed(200 + i)
    x = torch.randn(T, E, generator=g)
    t = torch.arange(T)
    if group_top == 1 or not has_bias:
        x[t % 11 == 1] = 0.0
    if n_groups == 1:
        x[t % 11 == 3] = torch.randint(0, 3, (int((t % 11 == 3).sum()), E), generator=g).float() * 0.5
    few = torch.rand(T, E, generator=g) < 0.02
    x[(t % 11 == 5)[:, None] & ~few] = -math.inf                                  # a few open, or none
    x[(t % 11 == 6)[:, None] & few] = -math.inf
    x[t % 997 == 7] = -math.inf
    x = x.to(DT[dtype])
    bias = None
    if has_bias:
        bias = torch.randint(-20, 21, (E,), generator=g).float() * 2.0 ** -30
        if E > 4:
            bias[E // 2] = -math.inf
        bias = bias.cuda()
    c = {"topk": k, "score": score, "n_groups": n_groups, "topk_groups": topk_groups, "group_top": group_top,
         "scale": 1.5}
    check_route(K, x.cuda(), c, bias)
    c["renorm"] = False
    gi, gate, _ = check_route(K, x.cuda(), c, bias)
    bad = (t % 101 == 50) & (t % 11 != 5)
    x[bad, E // 3] = math.nan
    idx, gate_nan, _ = run_route(K, x.cuda(), c, bias)
    keep = ~bad
    assert torch.equal(idx.cpu().long()[keep], gi[keep])
    assert torch.equal(gate_nan.cpu()[keep], gate.cpu()[keep])
    assert bool(torch.isnan(gate_nan.cpu()[bad]).all())


def test_nan_and_infinite_logits(K):
    for score in ("softmax", "sigmoid"):
        for dtype in (torch.float32, torch.bfloat16):
            x = torch.zeros(4, 20)
            x[:, :] = torch.linspace(-1, 1, 20)
            x[0, 3] = math.nan
            x[1, 19] = math.nan
            x[2, 4] = math.inf
            x[3, :] = math.nan
            idx, gate, cnt = run_route(K, x.to(dtype).cuda(), {"topk": 5, "score": score})
            i, gt = idx.cpu(), gate.cpu()
            assert i.min() >= 0 and i.max() < 20 and int(cnt.sum()) == 20
            assert all(len(set(r.tolist())) == 5 for r in i)
            assert bool(torch.isnan(gt[[0, 1, 3]]).all())
            assert 3 not in i[0].tolist() and 19 not in i[1].tolist()
            assert i[3].tolist() == [0, 1, 2, 3, 4]
            if score == "softmax":
                assert bool(torch.isnan(gt[2]).all())
            else:
                assert i[2, 0] == 4 and bool(torch.isfinite(gt[2]).all())


def test_no_tokens_and_counts_between_calls(K):
    E, k = 64, 4
    ws = K.route_workspace(E)
    c = {"topk": k, "score": "softmax"}
    idx, gate, cnt = run_route(K, torch.empty(0, E, device="cuda"), c, ws=ws)
    assert int(cnt.abs().sum()) == 0
    for T in (5, 9000, 17):  # one block, many, one again on the same workspace
        x = torch.randn(T, E, device="cuda")
        idx, gate, cnt = run_route(K, x, c, ws=ws)
        assert torch.equal(cnt.cpu().long(), torch.bincount(idx.cpu().long().reshape(-1), minlength=E))
        i2, g2, _ = run_route(K, x, c, counts=False)
        assert torch.equal(idx, i2) and torch.equal(gate, g2)
    assert int(ws.sum()) == 0
    out = torch.empty(0, E, device="cuda")
    K.route_bwd(out, make_router(K, c), torch.empty(0, k, dtype=torch.int32, device="cuda"),
                torch.empty(0, k, device="cuda"), torch.empty(0, k, device="cuda"), out)


def test_rows_beyond_32_bit_offsets(K):
    T, E, ld = 66000, 40, 65536  # 4.3 G elements between the first and the last row
    wide = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    x = wide[:, :E]
    x.copy_(torch.randn(T, E, device="cuda"))
    c = {"topk": 4, "score": "sigmoid"}
    idx, gate, _ = run_route(K, x, c)
    i2, g2, _ = run_route(K, x.contiguous(), c)
    assert torch.equal(idx, i2) and torch.equal(gate, g2)
    dg = torch.randn(T, 4, device="cuda")
    small = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    K.route_bwd(x.contiguous(), make_router(K, c), idx, gate, dg, small)
    K.route_bwd(x, make_router(K, c), idx, gate, dg, x)  # the gradient over the logits themselves
    assert torch.equal(x, small)


def test_indices_outside_the_experts_contribute_nothing(K):
    E = 24
    x = torch.randn(2, E, device="cuda")
    idx = torch.tensor([[0, -1], [E, 5]], dtype=torch.int32, device="cuda")
    gate = torch.full((2, 2), 0.5, device="cuda")
    out = torch.full((2, E), 9.0, device="cuda")
    K.route_bwd(x, make_router(K, {"topk": 2, "score": "sigmoid", "renorm": False}), idx, gate, torch.ones(2, 2, device="cuda"), out)
    o = out.cpu()
    assert set(torch.nonzero(o[0]).flatten().tolist()) == {0} and set(torch.nonzero(o[1]).flatten().tolist()) == {5}


def test_side_stream_and_graph(K):
    T, E, k = 600, 128, 8
    c = {"topk": k, "score": "sigmoid", "scale": 2.0}
    r = make_router(K, c)
    bias = torch.linspace(-0.05, 0.05, E, device="cuda")
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    cnt = torch.empty(E, dtype=torch.int32, device="cuda")
    dg, dl = torch.randn(T, k, device="cuda"), torch.empty_like(x)
    ws = K.route_workspace(E)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.normal_()
        K.route(x, r, idx, gate, bias=bias, expert_counts=cnt, ws=ws)
        K.route_bwd(x, r, idx, gate, dg, dl)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        K.route(x, r, idx, gate, bias=bias, expert_counts=cnt, ws=ws)
        K.route_bwd(x, r, idx, gate, dg, dl)
    for _ in range(3):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        i2, g2, c2 = run_route(K, x, c, bias)
        d2 = torch.empty_like(x)
        K.route_bwd(x, r, i2, g2, dg, d2)
        assert torch.equal(idx, i2) and torch.equal(gate, g2) and torch.equal(cnt, c2) and torch.equal(dl, d2)
