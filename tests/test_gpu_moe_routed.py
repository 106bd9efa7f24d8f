"""The expert layer on a given routing, and a training step that runs the
routing operators, the layer, and the clipping together.

  * with moe_fwd's own routing given back to it, the routed call's outputs,
    counts and positions are those of moe_fwd bit for bit;
  * with other routings, outputs and gradients against the layer in fp64 on
    the CPU: max|got - ref| <= 1e-2 max|ref|, the layer's tolerance (bf16 inputs,
    h and y each rounded once: 3 * 2^-8 of a value, averaged over the sums);
  * a routing that is none ends in INVALID_ARG with the token, and the
    workspace works again once it is initialised."""
import numpy as np
import pytest
import torch

from _helpers import kosmos, rel_err
from kosmos_inputs import moe_inputs
from test_gpu_moe import _split, dispatch_tables_np

pytestmark = pytest.mark.gpu
TOL = 1e-2


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kosmos()


class Layer:
    def __init__(self, K, P, T, H, E, k, I, seed):
        self.K, self.P, self.k = K, P, k
        self.inp = moe_inputs(T, H, E, I, seed)
        d = "cuda"
        self.x = [t.contiguous().to(d) for t in torch.chunk(self.inp["x"], P, 0)]
        self.w = [[w.to(d) for w in _split(self.inp[n], P)] for n in ("w_gate", "w_up", "w_down")]
        self.y = [torch.full((T // P, H), float("nan"), dtype=torch.bfloat16, device=d) for _ in range(P)]
        self.counts = torch.empty(E, dtype=torch.int32, device=d)
        self.pos = torch.empty(T, k, dtype=torch.int32, device=d)
        self.ws = K.moe_workspace(P, T, H, E, k, I)

    def routed(self, idx, gate):
        self.K.moe_fwd_routed(self.x, *self.w, self.y, idx, gate, self.counts, self.pos, self.ws)
        return self.K.status_sync(self.ws)

    def own(self, idx, gate):
        self.K.moe_fwd(self.x, self.inp["w_router"].cuda(), *self.w, self.y, idx, gate, self.counts, self.pos, self.ws,
                       self.k)
        self.K.check(self.ws, "moe_fwd")


def reference(x, wg, wu, wd, idx, gate):
    """The layer in fp64: y [T, H]."""
    y = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        t, s = torch.where(idx == e)
        if len(t):
            h = torch.nn.functional.silu(x[t] @ wg[e]) * (x[t] @ wu[e])
            y = y.index_add(0, t, (h @ wd[e]) * gate[t, s][:, None])
    return y


@pytest.mark.parametrize("P,T,H,E,k,I", [(1, 1, 256, 64, 1, 128), (2, 256, 256, 64, 4, 256), (1, 100, 256, 64, 8, 128),
                                         (4, 1200, 512, 128, 8, 128), (3, 387, 256, 192, 5, 128)])
def test_own_routing_given_back(K, P, T, H, E, k, I):
    a = Layer(K, P, T, H, E, k, I, 5)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    a.own(idx, gate)
    y, counts, pos = torch.cat(a.y).clone(), a.counts.clone(), a.pos.clone()
    i0, g0 = idx.clone(), gate.clone()
    for ws in (a.ws, K.moe_workspace(P, T, H, E, k, I)):  # the same workspace and a fresh one
        a.ws = ws
        for _ in range(2):
            for t in a.y + [a.counts, a.pos]:
                t.fill_(-1)
            assert a.routed(idx, gate) == (K.OK, -1)
            assert torch.equal(torch.cat(a.y), y) and torch.equal(a.counts, counts) and torch.equal(a.pos, pos)
            assert torch.equal(idx, i0) and torch.equal(gate, g0)


@pytest.mark.parametrize("kind", ["route", "one_expert_set", "random"])
def test_other_routings_and_their_gradients(K, kind):
    P, T, H, E, k, I = 2, 256, 256, 64, 4, 256
    a = Layer(K, P, T, H, E, k, I, 7)
    g = torch.Generator().manual_seed(3)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    if kind == "route":
        logits = torch.randn(T, E, generator=g).cuda()
        bias = (torch.randn(E, generator=g) * 0.05).cuda()
        K.route(logits, K.router(topk=k, score=K.SCORE_SIGMOID, n_groups=8, topk_groups=3, group_top=2, scale=2.5), idx,
                gate, bias=bias)
    elif kind == "one_expert_set":  # every token to the same experts, most experts without a token
        idx.copy_(torch.tensor([63, 0, 17, 5], dtype=torch.int32).expand(T, k))
        gate.copy_(torch.rand(T, k, generator=g))
    else:
        idx.copy_(torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int())
        gate.copy_(torch.randn(T, k, generator=g))
        gate[::3, 1] = 0.0
    assert a.routed(idx, gate) == (K.OK, -1)
    c, _, pos = dispatch_tables_np(idx.cpu().numpy(), E)
    assert np.array_equal(a.counts.cpu().numpy(), c) and np.array_equal(a.pos.cpu().numpy(), pos)
    x = self_x = torch.cat(a.x).cpu().double().requires_grad_(True)
    ws = [torch.cat(w).cpu().double().requires_grad_(True) for w in a.w]
    gd = gate.cpu().double().requires_grad_(True)
    ref = reference(x, *ws, idx.cpu().long(), gd)
    assert rel_err(torch.cat(a.y).float().cpu(), ref.detach()) <= TOL
    dy = torch.randn(T, H, generator=g).bfloat16()
    want = torch.autograd.grad((ref * dy.double()).sum(), [self_x, *ws, gd])
    dys = [t.contiguous().cuda() for t in torch.chunk(dy, P, 0)]
    dx = [torch.empty_like(t) for t in a.x]
    dw = [[torch.empty_like(t) for t in w] for w in a.w]
    dwr = torch.empty(H, E, device="cuda")
    bws = K.moe_bwd_workspace(P, T, H, E, k, I)
    K.moe_bwd(a.x, torch.zeros(H, E, dtype=torch.bfloat16, device="cuda"), *a.w, idx, gate, a.ws, dys, dx, dwr, *dw, bws)
    K.check(bws, "moe_bwd")
    dgate = K.moe_bwd_debug_view(K.MOE_BWD_VIEW_DGATE, P, T, H, E, k, I, bws).view(torch.float32).view(T, k)
    assert rel_err(torch.cat(dx).float().cpu(), want[0]) <= TOL
    for got, w in zip(dw, want[1:4]):
        assert rel_err(torch.cat(got).float().cpu(), w) <= TOL
    assert rel_err(dgate.cpu(), want[4]) <= TOL


def test_a_routing_that_is_none(K):
    P, T, H, E, k, I = 2, 300, 256, 64, 4, 128
    a = Layer(K, P, T, H, E, k, I, 9)
    g = torch.Generator().manual_seed(1)
    good = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    gate = torch.rand(T, k, device="cuda")
    for t, s, v in ((0, 0, -1), (299, 3, E), (150, 2, 1 << 30), (7, 3, None)):
        bad = good.clone()
        bad[t, s] = bad[t, 0] if v is None else v  # None: the same expert twice
        assert a.routed(bad, gate) == (K.ERR_INVALID_ARG, t)
        K.workspace_init(a.ws)
        assert a.routed(good, gate) == (K.OK, -1)
    ref = reference(torch.cat(a.x).cpu().double(), *[torch.cat(w).cpu().double() for w in a.w], good.cpu().long(),
                    gate.cpu().double())
    assert rel_err(torch.cat(a.y).float().cpu(), ref) <= TOL


def test_training_step(K):
    """The gradients of one step of the example against automatic
    differentiation in fp64, then twelve steps: the loss falls, the load evens
    out, and clipping holds the norm."""
    from comm_persistent_gemm_gb300 import routed_step as R
    layer = R.RoutedLayer(2, 256, 256, 64, 4, 256, n_groups=8, topk_groups=4, scale=1.5, seed=3)
    x, target = R.inputs(layer, 4)
    y = torch.cat(layer.forward(x))
    dy = torch.randn(256, 256, generator=torch.Generator().manual_seed(5)).bfloat16()
    dx = layer.backward(x, [t.contiguous().cuda() for t in dy.chunk(2)])
    layer.check()
    xd = torch.cat(x).cpu().double().requires_grad_(True)
    wr = layer.w_router.cpu().double().requires_grad_(True)
    ws = [torch.cat(layer.weights[n]).cpu().double().requires_grad_(True) for n in ("gate", "up", "down")]
    idx = layer.idx.cpu().long()
    p = torch.sigmoid(xd @ wr).gather(1, idx)
    ref = reference(xd, *ws, idx, 1.5 * p / p.sum(1, keepdim=True))
    assert rel_err(y.float().cpu(), ref.detach()) <= TOL
    want = torch.autograd.grad((ref * dy.double()).sum(), [xd, wr, *ws])
    assert rel_err(dx.cpu(), want[0]) <= TOL
    assert rel_err(layer.dw_router.cpu(), want[1]) <= TOL
    for n, w in zip(("gate", "up", "down"), want[2:]):
        assert rel_err(torch.cat(layer.grads[n]).float().cpu(), w) <= TOL
    before = [t.double() for t in layer.grad_set.grads]
    norm = float(torch.sqrt(sum((t * t).sum() for t in before)))
    layer.update(0.0, norm / 4, 0.0)
    assert abs(float(layer.norm) - norm) <= 34 * 2.0 ** -24 * norm
    for t, b in zip(layer.grad_set.grads, before):
        assert rel_err(t.double().cpu(), b.cpu() / 4) <= 2.0 ** -7
    losses = R.train(layer, 12, lr=2.0)
    assert losses[-1] < 0.9 * losses[0]
