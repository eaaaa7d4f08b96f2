"""Refusals of the gated delta rule's and the group norm's entry points: host
validation with fake pointers (never dereferenced, validation fails first) and
the binding's own checks.  No GPU."""
import ctypes

import pytest
import torch

import linear_attention_simple_b200 as gla

OK, INVALID, UNSUPPORTED, MISALIGNED = range(4)
P = ctypes.c_void_p
PTR = dict(q=0x10000, k=0x20000, v=0x30000, a=0x40000, beta=0x50000)


@pytest.fixture(scope="module")
def L():
    from linear_attention_simple_b200 import build
    build.build()
    return gla.lib()


def fwd(L, cu=None, s0=None, o=0x60000, sf=None, ws=0x70000, wsb=1 << 40, N=1, T=64, Hk=1, H=1, dk=96, dv=192, ld=0,
        scale=0.1, dt=0, **ptr):
    x = dict(PTR, **ptr)
    return L.gated_delta_chunk_fwd(P(x["q"]), P(x["k"]), P(x["v"]), P(x["a"]), P(x["beta"]), P(cu), P(s0), P(o), P(sf),
                                   P(ws), wsb, N, T, Hk, H, dk, dv, ld, scale, dt, None)


def bwd(L, cu=None, dO=0x60000, grads=(0x70000,) * 5, gs=None, ws=0x80000, wsb=1 << 40, N=1, T=64, Hk=1, H=1, dk=96,
        dv=192, ld=0, scale=0.1, dt=0, **ptr):
    x = dict(PTR, **ptr)
    return L.gated_delta_chunk_bwd(P(x["q"]), P(x["k"]), P(x["v"]), P(x["a"]), P(x["beta"]), P(cu), None, P(dO), None,
                                   *map(P, grads), P(gs), P(ws), wsb, N, T, Hk, H, dk, dv, ld, scale, dt, None)


def step(L, state=0x90000, idx=None, ns=4, o=0x60000, N=4, T=1, Hk=1, H=1, dk=96, dv=192, ld=0, scale=0.1, dt=0, **ptr):
    x = dict(PTR, **ptr)
    return L.gated_delta_decode_step(P(state), P(idx), ns, P(x["q"]), P(x["k"]), P(x["v"]), P(x["a"]), P(x["beta"]),
                                     P(o), N, T, Hk, H, dk, dv, ld, scale, dt, None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_shared_refusals(L, call):
    for n in PTR:
        assert call(L, **{n: None}) == INVALID
        assert call(L, **{n: PTR[n] + 4}) == MISALIGNED
    for bad in (dict(N=-1), dict(T=-1), dict(H=-1), dict(Hk=-1), dict(Hk=0), dict(Hk=2, H=3), dict(Hk=4, H=2), dict(dk=0),
                dict(dv=-32), dict(ld=-8), dict(ld=8), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(dt=7)):
        assert call(L, **bad) == INVALID, bad
    for bad in (dict(dk=80), dict(dk=256), dict(dv=16), dict(dv=200), dict(dv=288), dict(H=70000, Hk=70000),
                dict(N=1 << 20, H=1 << 14, Hk=1), dict(N=1 << 15, T=1 << 30)):
        assert call(L, **dict(dict(ns=1 << 30) if call is step else {}, **bad)) == UNSUPPORTED, bad
    assert call(L, ld=196) == MISALIGNED
    assert call(L, N=0) == OK
    assert call(L, H=0, Hk=0) == OK


def test_chunk_refusals(L):
    assert fwd(L, dt=1) == UNSUPPORTED and bwd(L, dt=1) == UNSUPPORTED
    assert fwd(L, o=None) == INVALID and fwd(L, o=0x60008) == MISALIGNED
    assert fwd(L, ws=None) == INVALID and fwd(L, ws=0x70010, wsb=100) == INVALID and fwd(L, ws=0x70004) == MISALIGNED
    assert fwd(L, s0=0x8) == MISALIGNED and fwd(L, sf=0x8) == MISALIGNED and fwd(L, cu=0x4) == MISALIGNED
    assert bwd(L, dO=None) == INVALID and bwd(L, dO=0x60002) == MISALIGNED
    for i in range(5):
        g = [0x70000] * 5
        g[i] = None
        assert bwd(L, grads=g) == INVALID
        g[i] = 0x70004
        assert bwd(L, grads=g) == MISALIGNED
    assert bwd(L, gs=0x4) == MISALIGNED
    need = gla.gated_delta_chunk_workspace_bytes(2, 100, 4, for_bwd=True)
    assert bwd(L, N=2, T=100, H=4, Hk=2, wsb=need - 1) == INVALID


def test_workspace_query(L):
    f = gla.gated_delta_chunk_workspace_bytes
    assert f(0, 64, 1) == f(1, 0, 1) == f(1, 64, 0) == f(1, 64, 1, dk=80) == f(1, 64, 1, dv=16) == 0
    assert 0 < f(1, 64, 1) == f(1, 1, 1) < f(1, 65, 1) < f(1, 65, 1, for_bwd=True)
    assert f(3, 100, 2, packed=True) >= f(1, 100, 2, packed=True) > 0


def test_step_refusals(L):
    assert step(L, state=None) == INVALID and step(L, state=0x90004) == MISALIGNED
    assert step(L, ns=3) == INVALID and step(L, ns=-1) == INVALID
    assert step(L, o=None) == INVALID and step(L, o=0x60004) == MISALIGNED and step(L, idx=0x4) == MISALIGNED
    assert step(L, T=0) == OK
    assert step(L, dt=1, ld=194) == MISALIGNED


def norm(L, x=0x1000, gate=0x2000, w=0x3000, b=0x4000, y=0x5000, M=3, G=2, d=64, ldx=0, ldg=0, eps=1e-5, dt=0):
    return L.group_norm_silu(P(x), P(gate), P(w), P(b), P(y), M, G, d, ldx, ldg, 0, 1, 1, eps, dt, None)


def norm_bwd(L, x=0x1000, gate=0x2000, w=0x3000, b=0x4000, y=0x5000, gx=0x6000, gg=0x7000, gw=0x8000, gb=0x9000,
             ws=0xA000, wsb=1 << 40, M=3, G=2, d=64, ldx=0, ldg=0, eps=1e-5, dt=0):
    return L.group_norm_silu_bwd(P(x), P(gate), P(w), P(b), P(y), P(gx), P(gg), P(gw), P(gb), P(ws), wsb, M, G, d, ldx,
                                 ldg, 0, 1, 1, eps, dt, None)


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_refusals(L, call):
    for bad in (dict(M=-1), dict(G=-1), dict(d=0), dict(ldx=-1), dict(ldg=-8), dict(ldx=64), dict(ldg=120), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(dt=5), dict(x=None), dict(y=None)):
        assert call(L, **bad) == INVALID, bad
    for bad in (dict(d=12), dict(d=1032), dict(G=1 << 15)):
        assert call(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(x=0x1008), dict(gate=0x2002), dict(w=0x3004), dict(b=0x4004), dict(y=0x5004), dict(ldx=132),
                dict(ldg=132), dict(ldx=130, dt=1)):
        assert call(L, **bad) == MISALIGNED, bad
    assert call(L, G=0) == OK


def test_norm_bwd_refusals(L):
    assert norm_bwd(L, gx=None) == INVALID and norm_bwd(L, gg=None) == INVALID
    assert norm_bwd(L, ws=None) == INVALID and norm_bwd(L, wsb=4) == INVALID
    for n in ("gx", "gg", "gw", "gb", "ws"):
        assert norm_bwd(L, **{n: 0x6004}) == MISALIGNED
    f = gla.group_norm_silu_bwd_workspace_bytes
    assert f(0, 2, 64) == f(3, 0, 64) == f(3, 2, 12) == f(3, 2, 2048) == 0 < f(1, 2, 64) <= f(9, 2, 64)


def test_binding_refuses_before_the_library_is_called():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    q, v, a = z(2, 8, 1, 96), z(2, 8, 2, 192), z(2, 8, 2, t=torch.float32)
    with pytest.raises(ValueError):                     # host tensors
        gla.gated_delta_chunk_fwd(q, q, v, a, a)
    with pytest.raises(ValueError):                     # packed shapes without cu_seqlens
        gla.gated_delta_chunk_fwd(q[0], q[0], v[0], a[0], a[0])
    with pytest.raises(TypeError):
        gla.gated_delta_chunk_fwd(q.float(), q, v, a, a)
    with pytest.raises(ValueError):
        gla.group_norm_silu(v)
    with pytest.raises(ValueError):
        gla.group_norm_silu(z(4))


def test_row_strides_of_views():
    f = lambda x: gla._rows_stride(x, "x")  # noqa: E731
    b = torch.zeros(2, 5, 40)
    assert f(b[..., 8:32].unflatten(-1, (3, 8))) == 40
    assert f(b[:1, :1, 8:32].unflatten(-1, (3, 8))) == 24
    assert f(b[:, :1, 8:32].unflatten(-1, (3, 8))) == 200
    for bad in (b[:, :4, :24].unflatten(-1, (3, 8)), b[..., :30].unflatten(-1, (3, 10))[..., :8],
                b[..., :24].unflatten(-1, (8, 3)).transpose(-1, -2), b[:1, :1].expand(2, 5, 40).unflatten(-1, (5, 8))):
        with pytest.raises(ValueError):
            f(bad)


@pytest.mark.parametrize("name", ["gated_delta_sweep_fwd.cu", "gated_delta_sweep_bwd.cu", "gated_delta_grad.cu"])
def test_every_load_is_waited_for_before_its_block_ends(name):
    """A wait that runs out ends a kernel's work early.  What no input brings about is
    read from the source: each barrier that asynchronous loads complete on has a wait
    in the lines behind a note that no copy may be in flight when the block ends."""
    import os
    import re
    with open(os.path.join(os.path.dirname(gla.__file__), "csrc", name)) as f:
        text = f.read()
    loads = set(re.findall(r"(?:bulk_load|tma_load_2d)\([^;]*?&B\.(\w+)", text)) | set(re.findall(r"= tile\(\w+, &B\.(\w+)", text))
    drained = set()
    for part in text.split("no copy may be in flight when the block ends")[1:]:
        drained |= set(re.findall(r"(?:mbar|warp)_wait\(&B\.(\w+)", "\n".join(part.split("\n")[:8])))
    if "kq" in loads:                                  # behind what is on its way out of the same place
        assert re.search(r"tma_store_wait_read\(\);\s*if \(step > 0\) mbar_wait\(&B\.kq,", text)
        drained.add("kq")
    assert len(loads) >= 3 and loads <= drained, loads - drained


@pytest.mark.parametrize("shape", [(1 << 31, 1, 8), (1 << 16, (1 << 16) + 5, 1, 8)])
def test_binding_refuses_more_rows_than_the_abi_counts(shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    for call in (lambda: gla.group_norm_silu(x), lambda: gla.group_norm_silu_bwd(x, x)):
        with pytest.raises(ValueError, match="rows, more than"):
            call()
