"""Group norm with an activation on the GPU against the formula in 64 bits.

y, dgate and a bf16 dx are rounded once from fp32: at most 2^-8 of the value,
and fp32 sums over at most 1,024 channels before that (2e-6).  An fp32 dx: the
sums alone.  dweight and dbias: fp32 sums over the rows, 1e-5 of their terms'
2-norm."""
import pytest
import torch

import linear_attention_simple_b200 as gla
from delta_reference import norm, rel

pytestmark = pytest.mark.gpu
U = 2.0 ** -8

CASES = [  # M, G, d, dtype, gate, center, shared, weight, bias, act
    (1, 1, 8, torch.bfloat16, True, True, False, True, True, True),
    (3, 5, 24, torch.float32, False, True, True, True, True, True),
    (37, 16, 192, torch.bfloat16, True, True, False, True, True, True),
    (37, 16, 128, torch.float32, True, False, True, True, False, True),
    (700, 2, 256, torch.bfloat16, True, False, False, False, False, True),
    (65, 3, 264, torch.bfloat16, False, True, False, True, True, False),
    (9, 1, 1024, torch.float32, True, True, False, True, True, True),
    (5, 2, 776, torch.bfloat16, True, False, True, True, True, True),
    (5001, 7, 40, torch.bfloat16, True, True, True, True, True, True),
    (130, 33, 8, torch.float32, True, True, False, False, True, False),
]


def make(M, G, d, dtype, gate, shared, weight, bias, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda")

    ws = (d,) if shared else (G, d)
    return ((0.3 * rnd(M, G, d) + 0.2).to(dtype), 1 + 0.2 * rnd(*ws) if weight else None,
            0.2 * rnd(*ws) if bias else None, rnd(M, G, d).bfloat16() if gate else None, rnd(M, G, d).bfloat16())


@pytest.mark.parametrize("M,G,d,dtype,gate,center,shared,weight,bias,act", CASES)
def test_forward_and_gradients(M, G, d, dtype, gate, center, shared, weight, bias, act):
    x, w, b, z, dy = make(M, G, d, dtype, gate, shared, weight, bias, 1 + d)
    y = gla.group_norm_silu(x, w, b, z, center=center, act=act)
    got = gla.group_norm_silu_bwd(x, dy, w, b, z, center=center, act=act)
    leaves = [t.double().requires_grad_(True) if t is not None else None for t in (x, z, w, b)]
    ref = norm(leaves[0], leaves[2], leaves[3], leaves[1], center, act, 1e-5)
    assert y.dtype == torch.bfloat16 and rel(y, ref) <= U
    want = iter(torch.autograd.grad(ref, [t for t in leaves if t is not None], dy.double()))
    for n, t, g in zip(("dx", "dgate", "dweight", "dbias"), leaves, got):
        assert (t is None) == (g is None)
        if t is None:
            continue
        r = next(want)
        tol = 1e-5 if g.dtype == torch.float32 else U
        if n == "dx" and d == 8:
            tol *= 4            # centred groups of eight: dx is a difference of terms a few times its size
        assert rel(g, r) <= tol, (n, rel(g, r))
    again = gla.group_norm_silu_bwd(x, dy, w, b, z, center=center, act=act)
    for p, q in zip(got, again):
        assert p is None or torch.equal(p, q)


def test_rows_that_are_constant_or_zero():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[1:3] = 3.0
    y = gla.group_norm_silu(x, act=False)
    assert bool((y == 0).all())
    dx, _, _, _ = gla.group_norm_silu_bwd(x, torch.ones_like(x), act=False)
    assert bool(torch.isfinite(dx).all())


def test_no_rows():
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(4, 64, device="cuda")
    assert gla.group_norm_silu(x, w).shape == x.shape
    assert bool((gla.group_norm_silu_bwd(x, x, w)[2] == 0).all())


def test_slices_other_stream_and_graph():
    x, w, b, z, dy = make(50, 4, 96, torch.bfloat16, True, False, True, True, 3)
    buf = torch.full((50, 3 * 4 * 96 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, 384:768], buf[:, 768:1152] = x.flatten(1), z.flatten(1)
    xs, zs = buf[:, 384:768].unflatten(-1, (4, 96)), buf[:, 768:1152].unflatten(-1, (4, 96))
    want = (gla.group_norm_silu(x, w, b, z),) + gla.group_norm_silu_bwd(x, dy, w, b, z)
    got = (gla.group_norm_silu(xs, w, b, zs),) + gla.group_norm_silu_bwd(xs, dy, w, b, zs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rep = (gla.group_norm_silu(x, w, b, z),) + gla.group_norm_silu_bwd(x, dy, w, b, z)
    graph.replay()
    torch.cuda.synchronize()
    for p, q, r in zip(want, got, rep):
        assert torch.equal(p, q) and torch.equal(p, r)


def test_offsets_past_32_bits():
    M, G, d = 70_000, 32, 1024
    x = torch.zeros(M, G, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    end = make(40, G, d, torch.bfloat16, False, False, True, False, 7)
    x[-40:] = end[0]
    y = gla.group_norm_silu(x, end[1])
    assert torch.equal(y[-40:], gla.group_norm_silu(end[0], end[1]))
    dx = gla.group_norm_silu_bwd(x, x, end[1])[0]
    assert torch.equal(dx[-40:], gla.group_norm_silu_bwd(end[0], end[0], end[1])[0])


def test_gradients_against_differences():
    """fp32 x, identity activation: the loss <n, c> along random directions.
    Central differences with a step of 2^-6 of x's size leave third-order terms
    (2^-12) and fp32 roundings of y... y is bf16, so the loss is taken from the
    formula in 64 bits and only the gradient from the kernel."""
    x, w, b, z, dy = make(20, 3, 64, torch.float32, True, False, True, True, 5)
    got = gla.group_norm_silu_bwd(x, dy, w, b, z)
    g = torch.Generator(device="cuda").manual_seed(6)
    h = 2.0 ** -12
    for i, grad in ((0, got[0]), (3, got[1]), (1, got[2]), (2, got[3])):
        ins = [t.double() for t in (x, w, b, z)]
        v = torch.randn(ins[i].shape, generator=g, device="cuda").double()
        side = []
        for s in (1, -1):
            e = list(ins)
            e[i] = ins[i] + s * h * v
            side.append(float((norm(e[0], e[1], e[2], e[3], True, True, 1e-5) * dy.double()).sum()))
        diff, want = (side[0] - side[1]) / (2 * h), float((grad.double() * v).sum())
        assert abs(diff - want) <= 2 * U * float((grad.double() * v).norm()), (i, diff, want)


@pytest.mark.parametrize("M,G,d", [(37, 16, 192), (1000, 16, 192), (7, 3, 40), (601, 1, 1024)])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_eps_of_zero(M, G, d, gate, center):
    """Numbers of rows that the CTAs do not divide: the seats behind the last row
    hold zeros, whose norm is undefined at eps = 0, and add nothing.  Tolerances as
    above (every group's variance is some 0.09, far from zero)."""
    x, w, b, z, dy = make(M, G, d, torch.bfloat16, gate, False, True, True, 11)
    y = gla.group_norm_silu(x, w, b, z, center=center, eps=0.0)
    got = gla.group_norm_silu_bwd(x, dy, w, b, z, center=center, eps=0.0)
    leaves = [t.double().requires_grad_(True) if t is not None else None for t in (x, z, w, b)]
    ref = norm(leaves[0], leaves[2], leaves[3], leaves[1], center, True, 0.0)
    assert rel(y, ref) <= U
    want = iter(torch.autograd.grad(ref, [t for t in leaves if t is not None], dy.double()))
    for n, t, g in zip(("dx", "dgate", "dweight", "dbias"), leaves, got):
        if t is not None:
            r = next(want)
            assert rel(g, r) <= (1e-5 if g.dtype == torch.float32 else U), (n, rel(g, r))


@pytest.mark.parametrize("shape", [(3, 0, 64), (0, 4, 64)])
def test_shared_parameters_of_no_groups_and_of_no_rows_have_gradients_of_zero(shape):
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    assert gla.group_norm_silu(x, w, b).shape == x.shape
    grads = (torch.empty_like(x), None, torch.full_like(w, 7), torch.full_like(b, 7))
    _, _, gw, gb = gla.group_norm_silu_bwd(x, x, w, b, grads=grads)
    assert bool((gw == 0).all()) and bool((gb == 0).all())


def test_parameters_per_group_of_no_groups():
    x, w = torch.zeros(3, 0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(0, 64, device="cuda")
    assert gla.group_norm_silu_bwd(x, x, w)[2].shape == (0, 64)
