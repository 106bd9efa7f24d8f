"""What the routing and gradient operators refuse, on the host and without a
GPU: nothing is launched for any of these."""
import ctypes as C

import pytest
import torch

from _helpers import kosmos


@pytest.fixture(scope="module")
def K():
    return kosmos()


@pytest.fixture(scope="module")
def base():
    buf = (C.c_uint8 * 8192)()
    yield (C.addressof(buf) + 15) // 16 * 16
    del buf


GOOD = dict(dtype=3, tokens=4, experts=64, ld=64, topk=4, score=0, n_groups=1, topk_groups=1, group_top=1, renorm=1,
            scale=1.0)
BAD = [dict(dtype=1), dict(dtype=7), dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(experts=0), dict(experts=1025, ld=2000),
       dict(ld=63), dict(topk=0), dict(topk=17), dict(experts=3, topk=4), dict(score=2), dict(score=-1),
       dict(n_groups=0), dict(n_groups=7), dict(n_groups=64), dict(n_groups=8, topk_groups=0),
       dict(n_groups=8, topk_groups=9), dict(n_groups=8, topk_groups=1, topk=9), dict(group_top=0), dict(group_top=3),
       dict(n_groups=32, experts=32, group_top=2, topk_groups=8), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
       dict(scale=float("nan"))]


def _router(K, a):
    r = K.Router()
    K.lib().kosmos_default_router(C.byref(r))
    for f in ("topk", "score", "n_groups", "topk_groups", "group_top", "renorm", "scale"):
        setattr(r, f, a[f])
    return r


def test_default_router(K):
    r = K.Router()
    K.lib().kosmos_default_router(C.byref(r))
    assert (r.score, r.topk, r.n_groups, r.topk_groups, r.group_top, r.renorm, r.scale) == (0, 1, 1, 1, 1, 1, 1.0)
    r = K.router(topk=8, score=K.SCORE_SIGMOID, n_groups=8, topk_groups=4, group_top=2, renorm=False, scale=2.5)
    assert (r.score, r.topk, r.n_groups, r.topk_groups, r.group_top, r.renorm, r.scale) == (1, 8, 8, 4, 2, 0, 2.5)


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_route_refuses(K, base, bad):
    a = {**GOOD, **bad}
    r = _router(K, a)
    L = K.lib()
    assert L.kosmos_route(base, a["dtype"], a["tokens"], a["experts"], a["ld"], C.byref(r), None, base, base, None, None,
                          0, None) == K.ERR_INVALID_ARG
    assert L.kosmos_route_bwd(base, a["dtype"], a["tokens"], a["experts"], a["ld"], C.byref(r), base, base, base, base,
                              a["ld"], None) == K.ERR_INVALID_ARG


def test_route_refuses_pointers_and_workspace(K, base):
    L, r = K.lib(), _router(K, GOOD)
    R = C.byref(r)
    need = K.lib().kosmos_route_workspace_bytes(64)
    assert need >= 256 + 4 * 64
    assert L.kosmos_route_workspace_bytes(0) == 0 and L.kosmos_route_workspace_bytes(1025) == 0

    def call(logits=base, router=R, bias=None, idx=base, gate=base, cnt=None, ws=None, n=0):
        return L.kosmos_route(logits, 3, 4, 64, 64, router, bias, idx, gate, cnt, ws, n, None)

    for kw in (dict(logits=None), dict(logits=base + 2), dict(router=None), dict(bias=base + 4), dict(idx=None),
               dict(idx=base + 4), dict(gate=None), dict(gate=base + 8), dict(cnt=base + 4, ws=base, n=need)):
        assert call(**kw) == K.ERR_INVALID_ARG, kw
    for kw in (dict(cnt=base), dict(cnt=base, ws=base, n=need - 1), dict(cnt=base, ws=base + 8, n=need)):
        assert call(**kw) == K.ERR_WORKSPACE, kw

    def bwd(logits=base, router=R, idx=base, gate=base, dg=base, dl=base, ldd=64):
        return L.kosmos_route_bwd(logits, 3, 4, 64, 64, router, idx, gate, dg, dl, ldd, None)

    for kw in (dict(logits=None), dict(logits=base + 2), dict(router=None), dict(idx=None), dict(gate=base + 4),
               dict(dg=None), dict(dl=None), dict(dl=base + 1), dict(ldd=63)):
        assert bwd(**kw) == K.ERR_INVALID_ARG, kw


def test_grad_refuses(K, base):
    L = K.lib()

    def lists(sizes, dtypes, ptrs=None):
        n = len(sizes)
        return ((C.c_void_p * n)(*(ptrs or [base] * n)), (C.c_int64 * n)(*sizes), (C.c_int32 * n)(*dtypes), n)

    def norm(sizes, dtypes, ptrs=None, out=base, each=None, ws=base, nb=1 << 20, n=None):
        p, s, d, m = lists(sizes, dtypes, ptrs)
        return L.kosmos_grad_norm(p, s, d, m if n is None else n, out, each, ws, nb, None)

    def clip(sizes, dtypes, ptrs=None, outs=None, mx=1.0, ws=base, nb=1 << 20):
        p, s, d, m = lists(sizes, dtypes, ptrs)
        o = (C.c_void_p * m)(*(outs or [base] * m))
        return L.kosmos_grad_clip(p, o, s, d, m, mx, base, ws, nb, None)

    for args in (([-1], [0]), ([4], [1]), ([4], [9]), ([1 << 46], [0]), ([1 << 45, 1 << 45], [0, 0])):
        assert norm(*args) == K.ERR_INVALID_ARG, args
        assert clip(*args) == K.ERR_INVALID_ARG, args
        _, s, d, m = lists(*args)
        assert L.kosmos_grad_workspace_bytes(s, d, m) == 0
    assert norm([4], [3], n=-1) == K.ERR_INVALID_ARG
    assert norm([4], [3], ptrs=[None]) == K.ERR_INVALID_ARG
    assert norm([4], [3], ptrs=[base + 2]) == K.ERR_INVALID_ARG
    assert norm([4], [0], ptrs=[base + 1]) == K.ERR_INVALID_ARG
    assert norm([4], [0], out=None) == K.ERR_INVALID_ARG
    assert norm([4], [0], each=base + 2) == K.ERR_INVALID_ARG
    assert clip([4], [0], outs=[base + 1]) == K.ERR_INVALID_ARG
    for mx in (-1.0, float("nan"), float("inf")):
        assert clip([4], [0], mx=mx) == K.ERR_INVALID_ARG
    need = L.kosmos_grad_workspace_bytes(*lists([40000, 3], [3, 0])[1:])
    assert need >= 512 + 8 * 11
    assert norm([40000, 3], [3, 0], nb=need - 1) == K.ERR_WORKSPACE
    assert clip([40000, 3], [3, 0], nb=need - 1) == K.ERR_WORKSPACE
    assert norm([4], [0], ws=None) == K.ERR_WORKSPACE
    assert norm([4], [0], ws=base + 4) == K.ERR_WORKSPACE


def test_moe_fwd_routed_refuses(K, base):
    L = K.lib()
    P, T, H, E, k, I = 2, 128, 256, 64, 4, 128
    ptr = (C.c_void_p * P)(base, base)
    bad = (C.c_void_p * P)(base, base + 2)

    def call(x=ptr, P=P, T=T, H=H, E=E, k=k, I=I, wg=ptr, wu=ptr, wd=ptr, idx=base, gate=base, y=ptr, cnt=base, pos=base,
             ws=base, nb=1 << 40, o=None):
        return L.kosmos_moe_fwd_routed(x, P, T, H, E, k, I, wg, wu, wd, idx, gate, y, cnt, pos, ws, nb,
                                       C.byref(o) if o else None, None)

    for kw in (dict(P=0), dict(P=3), dict(T=127), dict(H=100), dict(E=60), dict(E=512), dict(k=0), dict(k=9), dict(I=100),
               dict(x=None), dict(x=bad), dict(wg=None), dict(wu=bad), dict(wd=None), dict(idx=None), dict(idx=base + 4),
               dict(gate=None), dict(y=bad), dict(cnt=None), dict(pos=base + 8)):
        assert call(**kw) == K.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=base + 8), dict(nb=1024)):
        assert call(**kw) == K.ERR_WORKSPACE, kw
    for kw in (dict(sched=K.SCHED_UNFUSED), dict(sched=K.SCHED_FIXED), dict(inject=K.INJECT_IDENTITY_EXPERTS),
               dict(link_gbs=100)):
        assert call(o=K.opts(**kw)) == K.ERR_UNSUPPORTED, kw


def test_binding_refuses(K):
    """The binding's own checks: CPU tensors, types, shapes, strides."""
    x, r = torch.zeros(4, 8), K.router(topk=2)
    i, g = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        K.route(x, r, i, g)
    with pytest.raises(ValueError):
        K.route_bwd(x, r, i, g, g, x)
    with pytest.raises(ValueError):
        K.GradSet([x])
    with pytest.raises(ValueError):
        K.GradSet([], [x])
    with pytest.raises(K.KosmosError):
        K.route_workspace(4096)
