"""GPU parity of the global gradient norm and of clipping against 64-bit sums.

Tolerances, in units of u = 2^-24 (half a step of fp32).  Norm: at most 64
squares are summed in fp32 (each square and each addition half a step: 65 u
on the sum, half of that on its root) before fp64 takes over, and the result
is rounded once: 34 u.  Clipped values: the norm's 33 u, the factor's and the
product's rounding and the norm's epsilon in the denominator's own fp64: 36 u,
and half a step of the tensor's type (fp16 below 2^-14: half of 2^-24)."""
import math

import pytest
import torch

from _helpers import kosmos

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTS = (torch.bfloat16, torch.float32, torch.float16)


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return kosmos()


def ref_norms(grads):
    sq = [float((g.detach().cpu().double() ** 2).sum()) for g in grads]
    return math.sqrt(math.fsum(sq)), torch.tensor(sq, dtype=torch.float64).sqrt()


def run_norm(K, grads, ws=None):
    norm = torch.full((1,), -1.0, device="cuda")
    each = torch.full((len(grads),), -1.0, device="cuda")
    K.grad_norm(grads, norm, ws if ws is not None else K.grad_workspace(grads), tensor_norms=each)
    return norm, each


def check_norm(K, grads):
    norm, each = run_norm(K, grads)
    rn, re = ref_norms(grads)
    assert abs(float(norm) - rn) <= 34 * U * rn, (float(norm), rn)
    assert bool(((each.cpu().double() - re).abs() <= 34 * U * re).all())
    return norm, rn


def check_clip(K, grads, max_norm, outs=None):
    """Clips into outs (or in place) and compares."""
    src = [g.clone() for g in grads]
    ref, _ = ref_norms(src)
    coef = min(1.0, max_norm / (ref + 1e-6))
    norm = torch.empty(1, device="cuda")
    s = K.GradSet(grads, outs)
    K.grad_clip(s, max_norm, norm, K.grad_workspace(s))
    assert abs(float(norm) - ref) <= 34 * U * ref
    for a, o in zip(src, outs if outs is not None else grads):
        want = a.cpu().double() * coef
        tiny = 2.0 ** -25 if a.dtype == torch.float16 else 1e-38
        lim = (36 * U + torch.finfo(a.dtype).eps / 2 * (1 + 2 ** -6)) * want.abs() + tiny
        assert bool(((o.cpu().double() - want).abs() <= lim).all())
    if outs is not None:
        for a, g in zip(src, grads):
            assert torch.equal(a, g)


SIZES = [0, 1, 7, 8, 9, 31, 63, 64, 65, 255, 257, 4095, 4097, 8191, 8192, 8193, 16385, 100003, 0]


def ragged(seed, shift, sizes=SIZES):
    """Gradients of mixed types; tensor i starts (i * shift) % 8 elements into
    a buffer of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        off = (i * shift) % 8
        buf = torch.randn(n + off + 8, generator=g, device="cuda") * 10.0 ** (i % 5 - 3)
        out.append(buf.to(DTS[i % 3])[off:off + n])
    return out


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm_ragged(K, shift):
    check_norm(K, ragged(1 + shift, shift))


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 256, 257, 1000, 1001, 2100])
def test_norm_and_clip_many_tensors(K, n):
    grads = ragged(n + 7, 1, [1 + (i * 37) % 301 for i in range(n)])
    if n == 0:
        norm, each = run_norm(K, grads)
        assert float(norm) == 0.0
    else:
        check_norm(K, grads)
    check_clip(K, grads, 0.5)


@pytest.mark.parametrize("shift,out_shift", [(0, 0), (1, 1), (1, 0), (3, 5)])
@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0])
def test_clip_into_outputs(K, shift, out_shift, max_norm):
    grads = ragged(21, shift)
    outs = [torch.empty(g.numel() + 8, dtype=g.dtype, device="cuda")[(i * out_shift) % 8:][:g.numel()]
            for i, g in enumerate(grads)]
    check_clip(K, grads, max_norm, outs)


BIG = [0, 2500001, 31, 4000003, 1, 1800000, 700001]  # 23 MB: more than one launch holds


@pytest.mark.parametrize("shift,out_shift", [(0, 0), (1, 1), (1, 0), (3, 5)])
def test_clip_of_a_larger_set(K, shift, out_shift):
    grads = ragged(51, shift, BIG)
    outs = [torch.empty(g.numel() + 8, dtype=g.dtype, device="cuda")[(i * out_shift) % 8:][:g.numel()]
            for i, g in enumerate(grads)]
    check_clip(K, grads, 1.0, outs)
    check_clip(K, grads, 1.0)
    check_norm(K, grads)


def test_norm_and_clip_agree_and_share_a_workspace(K):
    """One workspace through calls of every kind, in turn."""
    for sizes in (SIZES, BIG):
        grads = ragged(61, 1, sizes)
        s = K.GradSet(grads, [torch.empty_like(g) for g in grads])
        ws, a, b = K.grad_workspace(s), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        for _ in range(3):
            K.grad_norm(s, a, ws)
            K.grad_clip(s, 1.0, b, ws)
            assert abs(float(a) - float(b)) <= 2 * U * float(a)
        assert K.status_sync(ws) == (K.OK, -1)


def test_clip_in_place_and_guards(K):
    bufs = [torch.full((n + 16,), 3.0, dtype=DTS[i % 3], device="cuda") for i, n in enumerate(SIZES)]
    grads = [b[8:8 + n] for b, n in zip(bufs, SIZES)]
    for i, g in enumerate(grads):
        g.normal_()
    check_clip(K, grads, 1.0)
    for b, n in zip(bufs, SIZES):
        assert bool((b[:8] == 3.0).all()) and bool((b[8 + n:] == 3.0).all())


def test_factor_one_leaves_every_bit(K):
    g = [torch.tensor([-0.0, 1e-40, 0.25], device="cuda"), torch.full((5000,), -0.01, dtype=torch.bfloat16, device="cuda")]
    before = [t.clone() for t in g]
    norm = torch.empty(1, device="cuda")
    K.grad_clip(g, 5.0, norm, K.grad_workspace(g))
    for a, b in zip(before, g):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mag", [1e-38, 1e-30, 1e-22, 1e-18, 1e17, 1e20, 1e30])
def test_squares_outside_fp32(K, dtype, mag):
    """Squares below or above fp32's range: sums stay those of 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.randn(5001, generator=g, device="cuda") * mag).to(dtype)
    y = torch.zeros(900, dtype=dtype, device="cuda")
    z = x.clone()
    z[100:] = 0
    z[-1] = mag
    for grads in ([x], [y, x, y], [z], [x, torch.ones(1, device="cuda")]):
        norm, each = run_norm(K, grads)
        rn, re = ref_norms(grads)
        assert abs(float(norm) - rn) <= 34 * U * rn + 2.0 ** -149
        assert bool(((each.cpu().double() - re).abs() <= 34 * U * re + 2.0 ** -149).all())


def test_zero_nan_and_infinite(K):
    z = [torch.zeros(1000, device="cuda"), torch.zeros(77, dtype=torch.bfloat16, device="cuda")]
    norm, each = run_norm(K, z)
    assert float(norm) == 0.0 and bool((each == 0).all())
    check_clip(K, z, 1.0)
    for bad in (math.nan, math.inf):
        for dt in DTS:
            g = [torch.ones(300, dtype=dt, device="cuda"), torch.ones(40001, dtype=dt, device="cuda")]
            g[1][40000] = bad
            norm, each = run_norm(K, g)
            assert float(each[0]) == pytest.approx(math.sqrt(300))
            for v in (float(norm), float(each[1])):
                assert math.isnan(v) if math.isnan(bad) else v == math.inf
            K.grad_clip(g, 1.0, norm, K.grad_workspace(g))
            if math.isnan(bad):
                assert bool(torch.isnan(g[0]).all()) and bool(torch.isnan(g[1]).all())
            else:
                assert bool((g[0] == 0).all()) and bool((g[1][:-1] == 0).all()) and math.isnan(float(g[1][-1]))


def test_norm_beyond_fp32_is_infinite(K):
    g = [torch.full((8,), 3e38, device="cuda")]
    norm, _ = run_norm(K, g)
    assert float(norm) == math.inf


def test_more_elements_than_32_bits(K):
    n = (1 << 32) + 5
    x = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    norm, each = run_norm(K, [x])
    want = math.sqrt(n) * 2.0 ** -10
    assert abs(float(norm) - want) <= 34 * U * want
    K.grad_clip([x], 1.0, norm, K.grad_workspace([x]))
    v = x[[0, 1 << 20, (1 << 31) + 3, n - 1]].float().cpu().double()
    assert bool(((v - 2.0 ** -10 / want).abs() <= (36 * U + 2.0 ** -8) * 2.0 ** -10 / want).all())
    assert bool((x[:1 << 28] == x[0]).all()) and bool((x[-(1 << 28):] == x[0]).all())


def test_reruns_are_bit_identical(K):
    grads = ragged(31, 1, [1 << 20, 99999, 5, 300000, 1 << 21])
    s = K.GradSet(grads)
    ws = K.grad_workspace(s)
    a = run_norm(K, s.grads, ws)
    for _ in range(20):
        b = run_norm(K, s.grads, ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_side_stream_and_graph(K):
    grads = ragged(41, 1)
    outs = [torch.empty_like(g) for g in grads]
    s = K.GradSet(grads, outs)
    ws, norm = K.grad_workspace(s), torch.empty(1, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        grads[3].mul_(3.0)
        K.grad_clip(s, 1.0, norm, ws)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        K.grad_clip(s, 1.0, norm, ws)
    for f in (2.0, 0.25):
        for g in grads:
            g.mul_(f)
        graph.replay()
        torch.cuda.synchronize()
        n2 = torch.empty(1, device="cuda")
        o2 = [torch.empty_like(g) for g in grads]
        s2 = K.GradSet(grads, o2)
        K.grad_clip(s2, 1.0, n2, K.grad_workspace(s2))
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, o2))
