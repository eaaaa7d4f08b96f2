"""The gated delta rule on the GPU against the token recurrence in 64 bits.

Tolerances (relative 2-norm), from the roundings on each path; a bf16 rounding
is off by at most U = 2^-8 of the value, a pair of bf16 terms by 2^-17:
  o         rounded itself, and S, P and V' each once before their products:
            four independent roundings, sqrt(4) U = 2 U.
  dq, dk    rounded, and dO or dv, V' (twice) and the state each once: 2.5 U.
  dv        computed from pairs, rounded once: U, and 2^-14 for the pairs.
  S_T, dS0, dbeta   a pair for each operand of the four products on a chunk's
            path, and 2^-17 of what the chunk before left: 8 x 2^-17.
  da        sums of up to 64 tokens' terms of either sign: sqrt(64) = 8 times
            that of its terms (2 x 2^-17, three terms elsewhere): 16 x 2^-17.
            Under strong decays the terms themselves (o.dO) are up to 8 times
            the sums, so the error is taken against the larger of the two.
"""
import pytest
import torch

import linear_attention_simple_b200 as gla
from delta_reference import backward, forward, recurrence, rel

pytestmark = pytest.mark.gpu

U, P = 2.0 ** -8, 2.0 ** -17
TOL_O, TOL_QK, TOL_V, TOL_S, TOL_DA = 2 * U, 2.5 * U, U + 2.0 ** -14, 8 * P, 16 * P


def make(lead, Hk, H, dk, dv, seed, decay="usual", dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda")

    q, k = rnd(*lead, Hk, dk), rnd(*lead, Hk, dk) + 0.5 * rnd(*(1,) * len(lead), Hk, dk)
    a = {"usual": lambda: torch.nn.functional.logsigmoid(rnd(*lead, H) + 3),
         "slow": lambda: -0.002 * torch.rand((*lead, H), generator=g, device="cuda"),
         "none": lambda: torch.zeros((*lead, H), device="cuda"),
         "strong": lambda: -8 * torch.rand((*lead, H), generator=g, device="cuda"),
         "resets": lambda: torch.where(torch.rand((*lead, H), generator=g, device="cuda") < 0.05, -1e4, -0.05)}[decay]()
    return dict(q=(q / q.norm(dim=-1, keepdim=True)).to(dtype), k=(k / k.norm(dim=-1, keepdim=True)).to(dtype),
                v=rnd(*lead, H, dv).to(dtype), a=a, beta=torch.sigmoid(rnd(*lead, H)))


def states(N, H, dk, dv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 0.1 * torch.randn((N, H, dk, dv), generator=g, device="cuda")


def cu_of(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def args(d):
    return d["q"], d["k"], d["v"], d["a"], d["beta"]


def check_fwd(d, s0, cu=None):
    dk, z = d["q"].shape[-1], s0
    if s0 is None:
        N = cu.numel() - 1 if cu is not None else d["q"].shape[0]
        z = torch.zeros(N, d["v"].shape[-2], dk, d["v"].shape[-1], device="cuda")
    o, s = gla.gated_delta_chunk_fwd(*args(d), s0=s0, cu_seqlens=cu)
    ro, rs = forward(d, z, dk ** -0.5, cu)
    assert rel(o, ro) <= TOL_O and rel(s, rs) <= TOL_S, (rel(o, ro), rel(s, rs))


def check_bwd(d, s0, dO, ds, cu=None, da_of_terms=False):
    dk = d["q"].shape[-1]
    N = cu.numel() - 1 if cu is not None else d["q"].shape[0]
    z = torch.zeros(N, d["v"].shape[-2], dk, d["v"].shape[-1], device="cuda")
    got = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, cu_seqlens=cu)
    ref = backward(d, z if s0 is None else s0, dO, z if ds is None else ds, dk ** -0.5, cu)
    for n, x, y, tol in zip(("dq", "dk", "dv", "da", "dbeta", "ds0"), got, ref,
                            (TOL_QK, TOL_QK, TOL_V, TOL_DA, TOL_S, TOL_S)):
        y = torch.zeros_like(x) if y is None else y
        if n == "da" and da_of_terms:
            o, _ = forward(d, z if s0 is None else s0, dk ** -0.5, cu)
            terms = float((o * dO.double()).sum(-1).norm())
            assert float((x - y).norm()) <= tol * max(terms, float(y.norm()))
            continue
        assert rel(x, y) <= tol, (n, rel(x, y), tol)
    return got


SHAPES = [  # N, T, Hk, H, dk, dv
    (1, 1, 1, 1, 96, 192), (2, 1, 2, 4, 64, 32), (1, 63, 1, 1, 64, 64), (2, 64, 1, 2, 96, 192), (1, 65, 2, 2, 128, 128),
    (3, 130, 2, 6, 128, 96), (1, 200, 16, 16, 96, 192), (2, 97, 1, 3, 128, 256), (1, 129, 3, 3, 64, 160),
    (1, 66, 1, 1, 96, 224), (140, 67, 1, 1, 96, 192), (12, 70, 4, 16, 64, 128),
]


@pytest.mark.parametrize("N,T,Hk,H,dk,dv", SHAPES)
@pytest.mark.parametrize("with_s0", [False, True])
def test_chunk_fwd(N, T, Hk, H, dk, dv, with_s0):
    check_fwd(make((N, T), Hk, H, dk, dv, 1 + T), states(N, H, dk, dv, 2) if with_s0 else None)


@pytest.mark.parametrize("N,T,Hk,H,dk,dv", SHAPES)
@pytest.mark.parametrize("with_states", [False, True])
def test_chunk_bwd(N, T, Hk, H, dk, dv, with_states):
    d = make((N, T), Hk, H, dk, dv, 3 + T)
    dO = make((N, T), Hk, H, dk, dv, 4 + T)["v"]
    s0, ds = (states(N, H, dk, dv, 5), states(N, H, dk, dv, 6)) if with_states else (None, None)
    check_bwd(d, s0, dO, ds)


def test_more_chunks_than_fit_at_once():
    """The gradients' kernel walks over the chunks: several rounds of it, dense and
    packed with sequences that are empty."""
    N, T, H, dk, dv = 300, 65, 8, 64, 32
    d, dO = make((N, T), H, H, dk, dv, 71), make((N, T), H, H, dk, dv, 72)["v"]
    check_bwd(d, states(N, H, dk, dv, 73), dO, states(N, H, dk, dv, 74))
    lens = [3, 0, 70, 0, 0, 1] * 60
    d, dO = make((sum(lens),), 4, 8, dk, dv, 75), make((sum(lens),), 4, 8, dk, dv, 76)["v"]
    got = gla.gated_delta_chunk_bwd(*args(d), dO, cu_seqlens=cu_of(lens))
    # the pattern of lengths repeats: a dense call on each of its sequences
    x = {n: t.view(60, 74, *t.shape[1:]) for n, t in dict(d, dO=dO).items()}
    out = [t.view(60, 74, *t.shape[1:]) for t in got[:5]]
    for b, e in ((0, 3), (3, 73), (73, 74)):
        part = {n: t[:, b:e].contiguous() for n, t in x.items()}
        want = gla.gated_delta_chunk_bwd(*args(part), part["dO"])
        for u, v in zip(out, want):
            assert torch.equal(u[:, b:e], v)


# few heads and long sequences: both directions cut them into segments
LONG = [(1, 1600, 1, 1, 96, 192, None), (2, 2100, 1, 2, 128, 128, None), (1, 1537, 2, 2, 64, 256, None),
        (1, 1793, 1, 1, 96, 160, None), (1, 0, 1, 2, 96, 192, [700, 0, 1200, 65]), (1, 0, 1, 1, 128, 32, [1, 1700]),
        (1, 769, 2, 2, 96, 192, None), (1, 0, 1, 1, 64, 64, [770, 3, 129])]


@pytest.mark.parametrize("N,T,Hk,H,dk,dv,lens", LONG)
@pytest.mark.parametrize("decay", ["usual", "slow", "resets"])
def test_segments(N, T, Hk, H, dk, dv, lens, decay):
    cu = cu_of(lens) if lens else None
    N = len(lens) if lens else N
    d = make((sum(lens),) if lens else (N, T), Hk, H, dk, dv, 50, decay)
    check_fwd(d, states(N, H, dk, dv, 51), cu)
    check_fwd(d, None, cu)


@pytest.mark.parametrize("N,T,Hk,H,dk,dv,lens", LONG)
@pytest.mark.parametrize("decay,with_states", [("usual", True), ("usual", False), ("slow", True), ("resets", True)])
def test_segments_bwd(N, T, Hk, H, dk, dv, lens, decay, with_states):
    cu = cu_of(lens) if lens else None
    N = len(lens) if lens else N
    lead = (sum(lens),) if lens else (N, T)
    d, dO = make(lead, Hk, H, dk, dv, 52, decay), make(lead, Hk, H, dk, dv, 53)["v"]
    s0, ds = (states(N, H, dk, dv, 54), states(N, H, dk, dv, 55)) if with_states else (None, None)
    check_bwd(d, s0, dO, ds, cu, da_of_terms=decay == "resets")


@pytest.mark.parametrize("decay", ["slow", "none", "strong", "resets"])
def test_decays(decay):
    d = make((2, 150), 2, 2, 96, 192, 7, decay)
    s0, ds, dO = states(2, 2, 96, 192, 8), states(2, 2, 96, 192, 9), make((2, 150), 2, 2, 96, 192, 10)["v"]
    check_fwd(d, s0)
    check_bwd(d, s0, dO, ds, da_of_terms=decay in ("strong", "resets"))


def test_a_minus_infinity_is_a_reset():
    d = make((1, 100), 1, 1, 96, 192, 11)
    d["a"][0, 40] = -float("inf")
    o, s = gla.gated_delta_chunk_fwd(*args(d))
    ro, rs = forward(d, torch.zeros(1, 1, 96, 192, device="cuda"), 96 ** -0.5)
    assert rel(o, ro) <= TOL_O and rel(s, rs) <= TOL_S


def test_a_nan_decay_is_not_taken_for_a_reset():
    d = make((2, 200), 1, 1, 96, 192, 11)
    d["a"][0, 40] = float("nan")
    o, s = gla.gated_delta_chunk_fwd(*args(d))
    assert bool(o[0, 40:].isnan().all()) and bool(s[0].isnan().all())
    assert bool(o[1].isfinite().all()) and bool(s[1].isfinite().all())


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
def test_write_strengths(beta):
    """beta = 0 (nothing written, dbeta still defined), 1 (the prediction replaced) and 2 (a reflection)."""
    d = make((1, 140), 1, 2, 96, 192, 12)
    d["beta"].fill_(beta)
    dO = make((1, 140), 1, 2, 96, 192, 13)["v"]
    s0, ds = states(1, 2, 96, 192, 14), states(1, 2, 96, 192, 15)
    check_fwd(d, s0)
    got = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds)
    ref = backward(d, s0, dO, ds, 96 ** -0.5)
    for x, y, tol in zip(got, ref, (TOL_QK, TOL_QK, TOL_V, TOL_DA, TOL_S, TOL_S)):
        if not float(y.norm()):
            assert float(x.float().norm()) <= 1e-25         # dv = 0: beta stands at 1e-30
        else:
            assert rel(x, y) <= tol, rel(x, y)


def test_keys_that_repeat_and_keys_of_zero():
    d = make((1, 128), 1, 1, 96, 192, 16)
    d["k"][:, :64] = d["k"][:, :1]
    d["k"][:, 100:110] = 0
    d["q"][:, 5] = 0
    check_fwd(d, None)
    check_bwd(d, None, make((1, 128), 1, 1, 96, 192, 17)["v"], None)


@pytest.mark.parametrize("lens", [[1], [0], [64, 64], [5, 0, 1, 130, 63, 65], [0, 0, 200, 0], [3] * 40])
def test_packed(lens):
    cu = cu_of(lens)
    T, N = int(cu[-1]), len(lens)
    d = make((T,), 2, 4, 96, 192, 18)
    s0, ds, dO = states(N, 4, 96, 192, 19), states(N, 4, 96, 192, 20), make((T,), 2, 4, 96, 192, 21)["v"]
    if T == 0:
        o, s = gla.gated_delta_chunk_fwd(*args(d), s0=s0, cu_seqlens=cu)
        got = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, cu_seqlens=cu)
        assert torch.equal(s, s0) and torch.equal(got[5], ds)
        return
    check_fwd(d, s0, cu)
    check_bwd(d, s0, dO, ds, cu)


def test_rows_outside_every_sequence_stay():
    cu = torch.tensor([7, 80, 150], dtype=torch.int32, device="cuda")
    d = make((160,), 1, 2, 96, 192, 22)
    dO = make((160,), 1, 2, 96, 192, 23)["v"]
    o = torch.full_like(d["v"], 5.0)
    gla.gated_delta_chunk_fwd(*args(d), cu_seqlens=cu, o=o)
    grads = [torch.full_like(x, 5.0) for x in args(d)] + [None]
    gla.gated_delta_chunk_bwd(*args(d), dO, cu_seqlens=cu, grads=grads)
    ro, _ = forward(d, torch.zeros(2, 2, 96, 192, device="cuda"), 96 ** -0.5, cu)
    assert rel(o[7:150], ro) <= TOL_O
    for x in [o] + grads[:5]:
        assert bool((x[:7] == 5).all()) and bool((x[150:] == 5).all())


def test_what_is_not_finite_stays_in_its_sequence():
    """Packed neighbours share tiles' tails: NaN and infinities in one sequence
    reach no other's outputs, and dense batches' rows keep apart too."""
    lens = [70, 33, 100, 1, 64]
    cu = cu_of(lens)
    d, dO = make((sum(lens),), 1, 2, 96, 192, 60), make((sum(lens),), 1, 2, 96, 192, 61)["v"]
    s0, ds = states(5, 2, 96, 192, 62), states(5, 2, 96, 192, 63)
    b, e = int(cu[1]), int(cu[2])

    def run():
        return gla.gated_delta_chunk_fwd(*args(d), s0=s0, cu_seqlens=cu) + \
            gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, cu_seqlens=cu)

    want = run()
    for n, bad in (("q", float("inf")), ("k", float("nan")), ("v", float("inf")), ("beta", float("nan"))):
        d[n][b:e] = bad
    dO[b:e] = float("nan")
    s0[1], ds[1] = float("nan"), float("inf")
    for i, (x, y) in enumerate(zip(run(), want)):
        if i in (1, 7):                                     # states: [sequence, ...]
            assert all(torch.equal(x[j], y[j]) for j in (0, 2, 3, 4)), i
        else:
            assert torch.equal(x[:b], y[:b]) and torch.equal(x[e:], y[e:]), i


@pytest.mark.parametrize("T", [100, 1700])
def test_states_in_place(T):
    """s_final may be s0 and grad_s0 ds_final, in one piece and in segments."""
    d, dO = make((1, T), 1, 1, 96, 192, 64), make((1, T), 1, 1, 96, 192, 65)["v"]
    s0, ds = states(1, 1, 96, 192, 66), states(1, 1, 96, 192, 67)
    o, s = gla.gated_delta_chunk_fwd(*args(d), s0=s0)
    grads = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds)
    o2, s2 = gla.gated_delta_chunk_fwd(*args(d), s0=s0.clone(), s_final=(c := s0.clone()))
    o3, s3 = gla.gated_delta_chunk_fwd(*args(d), s0=c.copy_(s0), s_final=c)
    again = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, grads=[torch.empty_like(x) for x in args(d)] + [ds])
    for x, y in zip((o, s, o, s) + tuple(grads), (o2, s2, o3, s3) + tuple(again)):
        assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """A sequence with more than 2^31 values of v, its end against a call on the
    end alone (a reset before it), and a pool with more than 2^31."""
    T, H, dv, tail = 150_000, 60, 256, 130
    d = make((1, T), 1, H, 64, dv, 68)
    assert d["v"].numel() > 2 ** 31
    d["a"][:, T - tail] = -1e4
    end = {n: x[:, T - tail:].contiguous() for n, x in d.items()}
    o, s = gla.gated_delta_chunk_fwd(*args(d))
    o2, s2 = gla.gated_delta_chunk_fwd(*args(end))
    # the chunks begin elsewhere: not the same bits
    assert rel(o[:, T - tail:], o2) <= TOL_O and rel(s, s2) <= TOL_S
    del o, s, d
    slots = 2 ** 31 // (H * 64 * dv) + 5
    pool = torch.zeros(slots, H, 64, dv, device="cuda")
    one = make((1, 1), 1, H, 64, dv, 69)
    pool[-1] = states(1, H, 64, dv, 70)[0]
    before = pool[-1:].clone()
    o = gla.gated_delta_decode_step(pool, *args(one), slot_idx=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    ro, rs = forward(one, before, 64 ** -0.5)
    assert rel(o, ro) <= 2e-6 and rel(pool[-1:], rs) <= 2e-6


def test_offsets_outside_the_rows_are_reported():
    d = make((100,), 1, 1, 96, 192, 24)
    gla.gla_get_device_status()
    for bad in ([0, 50, 120], [0, 60, 40], [-5, 50, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        gla.gated_delta_chunk_fwd(*args(d), cu_seqlens=cu)
        assert gla.gla_get_device_status() == 1
        gla.gated_delta_chunk_bwd(*args(d), d["v"], cu_seqlens=cu)
        assert gla.gla_get_device_status() == 1
    check_fwd(make((1, 100), 1, 1, 96, 192, 24), None)


def test_views_into_a_fused_projection():
    N, T, Hk, H, dk, dv = 2, 90, 2, 4, 96, 192
    d = make((N, T), Hk, H, dk, dv, 25)
    buf = torch.full((N, T, 2 * Hk * dk + H * dv + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    at, views = 0, {}
    for n, h, w in (("q", Hk, dk), ("k", Hk, dk), ("v", H, dv)):
        buf[..., at:at + h * w] = d[n].reshape(N, T, -1)
        views[n] = buf[..., at:at + h * w].unflatten(-1, (h, w))
        at += h * w
    e = dict(d, **views)
    dO, s0 = make((N, T), Hk, H, dk, dv, 26)["v"], states(N, H, dk, dv, 27)
    for x, y in zip(gla.gated_delta_chunk_fwd(*args(e), s0=s0), gla.gated_delta_chunk_fwd(*args(d), s0=s0)):
        assert torch.equal(x, y)
    for x, y in zip(gla.gated_delta_chunk_bwd(*args(e), dO, s0=s0), gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0)):
        assert torch.equal(x, y)
    st = states(2, H, dk, dv, 28)
    st2 = st.clone()
    assert torch.equal(gla.gated_delta_decode_step(st, *args(e)), gla.gated_delta_decode_step(st2, *args(d)))
    assert torch.equal(st, st2)


def test_workspace_contents_do_not_matter_and_calls_repeat():
    d = make((2, 333), 2, 4, 96, 192, 29)
    dO, s0, ds = make((2, 333), 2, 4, 96, 192, 30)["v"], states(2, 4, 96, 192, 31), states(2, 4, 96, 192, 32)
    outs = []
    for fill in (0, 255):
        wf = torch.full((gla.gated_delta_chunk_workspace_bytes(2, 333, 4),), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((gla.gated_delta_chunk_workspace_bytes(2, 333, 4, for_bwd=True),), fill, dtype=torch.uint8,
                        device="cuda")
        outs.append(gla.gated_delta_chunk_fwd(*args(d), s0=s0, ws=wf) +
                    gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, ws=wb))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_other_stream_and_graph_replay():
    d = make((1, 130), 1, 2, 96, 192, 33)
    dO, s0 = make((1, 130), 1, 2, 96, 192, 34)["v"], states(1, 2, 96, 192, 35)
    want = gla.gated_delta_chunk_fwd(*args(d), s0=s0) + gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gla.gated_delta_chunk_fwd(*args(d), s0=s0) + gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gla.gated_delta_chunk_fwd(*args(d), s0=s0) + gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0)
    new = make((1, 130), 1, 2, 96, 192, 36)
    for n in d:
        d[n].copy_(new[n])
    graph.replay()
    torch.cuda.synchronize()
    want = gla.gated_delta_chunk_fwd(*args(new), s0=s0) + gla.gated_delta_chunk_bwd(*args(new), dO, s0=s0)
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dk,dv", [(64, 64), (96, 192)])
def test_calls_that_overlap(dk, dv):
    """Forward and backward on two streams at once, each with buffers of its own."""
    d = make((2, 900), 4, 4, dk, dv, 77)
    dO, s0, ds = make((2, 900), 4, 4, dk, dv, 78)["v"], states(2, 4, dk, dv, 79), states(2, 4, dk, dv, 80)

    def fwd():
        return gla.gated_delta_chunk_fwd(*args(d), s0=s0)

    def bwd():
        return gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds)

    want = fwd() + tuple(bwd())
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        with torch.cuda.stream(a):
            x = fwd()
        with torch.cuda.stream(b):
            y = bwd()
        got.append(x + tuple(y))
    torch.cuda.synchronize()
    for g in got:
        for x, y in zip(g, want):
            assert torch.equal(x, y)


def test_gradients_against_differences():
    """Central differences of the loss along random directions, by the GPU's own
    forward: the loss in fp32 from S_T and the step's fp32 outputs (bf16 o would
    drown the difference).  Second-order terms cancel; third-order ones and the
    2^-17 of the states over a step of 2^-4 bound the error by 1%."""
    N, T, H, dk, dv, h = 1, 70, 1, 96, 192, 2.0 ** -4
    d = make((N, T), H, H, dk, dv, 37)
    ds, zero = states(N, H, dk, dv, 38), torch.zeros(N, H, dk, dv, device="cuda")
    dO = torch.zeros_like(d["v"])
    got = gla.gated_delta_chunk_bwd(*args(d), dO, ds_final=ds)
    g = torch.Generator(device="cuda").manual_seed(39)
    for n, grad in zip(("a", "beta"), got[3:5]):
        x = torch.randn(d[n].shape, generator=g, device="cuda")
        side = []
        for sign in (1, -1):
            e = dict(d)
            e[n] = d[n] + sign * h * x
            side.append(float((gla.gated_delta_chunk_fwd(*args(e), s0=zero)[1].double() * ds).sum()))
        diff, want = (side[0] - side[1]) / (2 * h), float((grad.double() * x).sum())
        scale = float((grad.double() * x).abs().sum())
        assert abs(diff - want) <= 1e-2 * scale, (n, diff, want)


# ---------------------------------------------------------------- step
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T,Hk,H,dk,dv", [(1, 1, 1, 1, 96, 192), (3, 1, 16, 16, 96, 192), (2, 5, 2, 4, 128, 256),
                                            (5, 2, 1, 3, 64, 32), (40, 3, 8, 16, 128, 128), (30, 1, 16, 16, 64, 160)])
def test_step(N, T, Hk, H, dk, dv, dtype):
    """All fp32: a few hundred additions at 2^-24 each, 2e-6 in the 2-norm."""
    d = make((N, T), Hk, H, dk, dv, 40, dtype=dtype)
    slots = N + 3
    st = states(slots, H, dk, dv, 41)
    before = st.clone()
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(42))[:N].to(torch.int32).cuda()
    o = gla.gated_delta_decode_step(st, *args(d), slot_idx=idx)
    ro, rs = forward(d, before[idx.long()], dk ** -0.5)
    assert o.dtype == torch.float32 and rel(o, ro) <= 2e-6 and rel(st[idx.long()], rs) <= 2e-6
    rest = [i for i in range(slots) if i not in idx.tolist()]
    assert torch.equal(st[rest], before[rest])
    if T == 1:
        st2 = before.clone()
        o2 = gla.gated_delta_decode_step(st2, *[d[n][:, 0] for n in ("q", "k", "v", "a", "beta")], slot_idx=idx)
        assert torch.equal(o2, o[:, 0]) and torch.equal(st2, st)


def test_step_skips_slots_outside_the_pool():
    d = make((4, 1), 2, 2, 96, 192, 43)
    st = states(3, 2, 96, 192, 44)
    before = st.clone()
    gla.gla_get_device_status()
    o = torch.full((4, 1, 2, 192), 7.0, device="cuda")
    idx = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device="cuda")
    gla.gated_delta_decode_step(st, *args(d), slot_idx=idx, o=o)
    assert gla.gla_get_device_status() == 1
    assert torch.equal(st[1], before[1]) and bool((o[1:3] == 7).all())
    pick = {n: x[[0, 3]] for n, x in d.items()}
    ro, rs = forward(pick, before[[2, 0]], 96 ** -0.5)
    assert rel(o[[0, 3]], ro) <= 2e-6 and rel(st[[2, 0]], rs) <= 2e-6


def test_prefill_decode_and_norm_together():
    """A serving step as it is used: packed prefill into states, then decoded
    tokens in the pool, each followed by the gated norm; against one recurrence
    over all tokens."""
    lens, H, dk, dv = [70, 5, 129], 4, 96, 192
    cu, more = cu_of(lens), 6
    d, tail = make((sum(lens),), 2, H, dk, dv, 45), make((3, more), 2, H, dk, dv, 46)
    gate, gate2 = make((sum(lens),), 2, H, dk, dv, 47)["v"], make((3, more), 2, H, dk, dv, 48)["v"]
    w = 1 + 0.1 * torch.randn(H, dv, generator=torch.Generator().manual_seed(49)).cuda()
    o, s = gla.gated_delta_chunk_fwd(*args(d), cu_seqlens=cu)
    y = gla.group_norm_silu(o, w, gate=gate)
    pool = torch.zeros(5, H, dk, dv, device="cuda")
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[idx.long()] = s
    ys = []
    for t in range(more):
        od = gla.gated_delta_decode_step(pool, *[tail[n][:, t].contiguous() for n in tail], slot_idx=idx)
        ys.append(gla.group_norm_silu(od, w, gate=gate2[:, t]))
    from delta_reference import norm
    zero = torch.zeros(1, H, dk, dv, dtype=torch.float64, device="cuda")
    for i, (b, e) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        whole = {n: torch.cat([d[n][b:e], tail[n][i]])[None].double() for n in d}
        ro, rs = recurrence(*args(whole), zero, dk ** -0.5)
        gates = torch.cat([gate[b:e], gate2[i]])[None].double()
        # the norm passes o's relative error on, and rounds once more
        ref = norm(ro, w.double(), None, gates, True, True, 1e-5)[0]
        assert rel(y[b:e], ref[:e - b]) <= TOL_O + 2 * U
        assert rel(torch.stack([x[i] for x in ys]), ref[e - b:]) <= 2 * U
        assert rel(pool[idx[i].long()], rs[0]) <= TOL_S


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -60])
@pytest.mark.parametrize("lens", [None, [130, 0, 1700]])
def test_small_gradients_at_write_strengths_of_zero(size, lens):
    """beta of zero and next to it, gradients as small as a mean over many tokens
    makes them: dbeta is <dV' ..., z>, which does not get smaller with beta, and dv
    is beta times that.  The tolerances are relative and do not change."""
    cu = cu_of(lens) if lens else None
    lead, N = ((sum(lens),), len(lens)) if lens else ((2, 140), 2)
    d = make(lead, 1, 2, 96, 192, 81)
    flat = d["beta"].view(-1, 2)
    flat[3::5] = 0.0
    flat[4::25] = 1e-35
    flat[9::25] = 1e-20
    flat[14::25] = 1e-11
    flat[19::25] = -1e-20
    dO, ds = make(lead, 1, 2, 96, 192, 82)["v"] * size, states(N, 2, 96, 192, 83) * size
    got = check_bwd(d, states(N, 2, 96, 192, 84), dO, ds, cu)
    ref = backward(d, states(N, 2, 96, 192, 84), dO, ds, 96 ** -0.5, cu)
    (gv, gb), (rv, rb) = ((x[2].flatten(0, -3), x[4].flatten(0, -2)) for x in (got, ref))
    assert bool((gv[3::5] == 0).all())
    assert rel(gb[3::5], rb[3::5]) <= TOL_S
    for first in (4, 9, 14, 19):
        assert rel(gb[first::25], rb[first::25]) <= TOL_S
        if float(rv[first::25].abs().mean()) > 2.0 ** -100:      # else its values are not normal numbers
            assert rel(gv[first::25], rv[first::25]) <= TOL_V


def test_write_strengths_of_zero_leave_a_state_of_zeros():
    d = make((2, 100), 1, 2, 96, 192, 85)
    d["beta"].zero_()
    o, s = gla.gated_delta_chunk_fwd(*args(d))
    assert bool((o == 0).all()) and bool((s == 0).all())
    got = gla.gated_delta_chunk_bwd(*args(d), make((2, 100), 1, 2, 96, 192, 86)["v"])
    for n, x in zip(("dq", "dk", "dv"), got):
        assert bool((x == 0).all()), n
    # beta stands at 2^-40 in da's sums of up to 128 x 192 terms of size 1, of either sign
    assert float(got[3].abs().max()) <= 2.0 ** -40 * (128 * 192) ** 0.5 * 8


def test_a_short_wait_limit_still_lets_copies_land():
    """A block that gives up waits for its own copies in flight, within the same
    limit: so limits of less than a millisecond count as one."""
    d, dO = make((2, 200), 2, 2, 96, 192, 87), make((2, 200), 2, 2, 96, 192, 88)["v"]
    want = gla.gated_delta_chunk_fwd(*args(d)) + gla.gated_delta_chunk_bwd(*args(d), dO)
    gla.gla_get_device_status()
    gla.gla_set_wait_limit_ns(1)
    try:
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        gla.gla_selftest_wait_timeout()
        end.record()
        assert gla.gla_get_device_status() == 5
        assert 0.9 <= start.elapsed_time(end) <= 500
        got = gla.gated_delta_chunk_fwd(*args(d)) + gla.gated_delta_chunk_bwd(*args(d), dO)
        assert gla.gla_get_device_status() == 0
    finally:
        gla.gla_set_wait_limit_ns(0)
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def beyond_rounding(x, ref):
    """By how much the elements of a bf16 x are off beyond a rounding of ref, at
    most, against the root mean square of ref's rows."""
    ref = ref.double()
    over = (x.double() - ref).abs() - U * ref.abs()
    rms = ref.square().mean(-1, keepdim=True).sqrt().clamp_min(1e-300)
    return float((over / rms).max())


# What o's own rounding does not account for, per element: pairs of bf16 terms leave 8 P
# of the terms' root mean square (TOL_S), whose largest of some 10^6 is five times that;
# the two parts of o (state, chunk) are up to 1.5 times their sum.  One term in a pair's
# place leaves 2^-10 of the root mean square and more.
TOL_ROUNDED = 8 * P * 5 * 1.5


@pytest.mark.parametrize("decay", ["usual", "slow", "strong"])
@pytest.mark.parametrize("N,T,Hk,H,dk,dv", [(2, 1, 1, 2, 96, 192), (2, 300, 2, 4, 96, 192), (2, 130, 1, 2, 128, 128),
                                            (2, 130, 1, 2, 64, 64), (1, 900, 1, 1, 96, 160), (1, 100, 1, 1, 64, 256)])
def test_o_is_off_by_its_own_rounding(N, T, Hk, H, dk, dv, decay):
    d, s0 = make((N, T), Hk, H, dk, dv, 90, decay), states(N, H, dk, dv, 91)
    o, _ = gla.gated_delta_chunk_fwd(*args(d), s0=s0)
    assert beyond_rounding(o, forward(d, s0, dk ** -0.5)[0]) <= TOL_ROUNDED


# One bf16 rounding of values of any mantissa alike is off by U sqrt((1 - 1/4) / (6 ln 2)),
# 0.425 U, in the relative 2-norm.  dq is rounded, and where it comes from the state that
# is rounded too: sqrt(2) of it at most; dk's part from a state has a second rounded
# factor (dv): sqrt(3).  With the usual decays and no states at either end at most half of
# dk is that part: sqrt(1 + 2/2).  Pairs (A, B, V') add 2^-17, lost in the 2% that are left.
ONE = 0.425 * 1.02 * U


@pytest.mark.parametrize("decay,with_states", [("usual", False), ("usual", True), ("slow", True), ("strong", True)])
@pytest.mark.parametrize("N,T,Hk,H,dk,dv", [(2, 300, 2, 4, 96, 192), (2, 140, 1, 3, 128, 96), (2, 130, 1, 2, 64, 64),
                                            (1, 900, 1, 1, 96, 160), (1, 100, 1, 1, 64, 256)])
def test_dq_and_dk_are_off_by_their_roundings(N, T, Hk, H, dk, dv, decay, with_states):
    d, dO = make((N, T), Hk, H, dk, dv, 92, decay), make((N, T), Hk, H, dk, dv, 93)["v"]
    s0, ds = (states(N, H, dk, dv, 94), states(N, H, dk, dv, 95)) if with_states else (None, None)
    got = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds)
    zero = torch.zeros(N, H, dk, dv, device="cuda")
    ref = backward(d, zero if s0 is None else s0, dO, zero if ds is None else ds, dk ** -0.5)
    assert rel(got[0], ref[0]) <= 2 ** 0.5 * ONE, rel(got[0], ref[0]) / U
    assert rel(got[1], ref[1]) <= (3 if with_states else 2) ** 0.5 * ONE, rel(got[1], ref[1]) / U


@pytest.mark.parametrize("lens", [None, [1, 70, 0, 1, 130]])
def test_the_first_decay_of_a_sequence_without_a_state_has_no_gradient(lens):
    """e^a S with S = 0: exactly 0, whatever gradient the states have; with an s0
    it is <E, e^a s0>."""
    cu, lead = (cu_of(lens), (sum(lens),)) if lens else (None, (3, 1))
    N = len(lens) if lens else 3
    d, dO = make(lead, 1, 2, 96, 192, 96), make(lead, 1, 2, 96, 192, 97)["v"]
    s0, ds = states(N, 2, 96, 192, 98), states(N, 2, 96, 192, 99)
    first = [int(b) for b, n in zip(cu.tolist(), lens) if n] if lens else slice(None)
    got = gla.gated_delta_chunk_bwd(*args(d), dO, ds_final=ds, cu_seqlens=cu)[3]
    assert bool((got[first] == 0).all())
    got = gla.gated_delta_chunk_bwd(*args(d), dO, s0=s0, ds_final=ds, cu_seqlens=cu)[3]
    want = backward(d, s0, dO, ds, 96 ** -0.5, cu)[3]
    assert rel(got[first], want[first]) <= TOL_DA
