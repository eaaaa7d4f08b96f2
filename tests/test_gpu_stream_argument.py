"""Calls that are given `stream=`, while the current stream is another one.

What the binding allocates for such a call belongs to the stream that the kernels
run on: the caching allocator hands out blocks in the order of a stream's own work.
Two ways in which a block of the current stream goes wrong:
  - it was freed there with work on it still to come: that work then lands in the
    call's output;
  - it is free again as soon as the binding returns (a workspace), and the current
    stream writes into it while the kernels still read it.
Both are made to happen here: the first by a wait on the current stream before the
pending write, the second by writes to blocks of the workspace's size all through
the call.  Results have to be the same bits as on the current stream."""
import pytest
import torch

import linear_attention_simple_b200 as gla

pytestmark = pytest.mark.gpu
LONG = 20_000_000                       # cycles of a wait: some 10 ms


def rnd(*shape, seed, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def delta(N, T, H, dk=96, dv=192):
    q, k = rnd(N, T, H, dk, seed=1), rnd(N, T, H, dk, seed=2)
    return dict(q=q / q.norm(dim=-1, keepdim=True), k=k / k.norm(dim=-1, keepdim=True), v=rnd(N, T, H, dv, seed=3),
                a=torch.nn.functional.logsigmoid(rnd(N, T, H, seed=4, dtype=torch.float32) + 3),
                beta=torch.sigmoid(rnd(N, T, H, seed=5, dtype=torch.float32)))


def delta_calls():
    d = delta(4, 1024, 16)
    s0, dO = rnd(4, 16, 96, 192, seed=6, dtype=torch.float32, std=0.1), rnd(4, 1024, 16, 192, seed=7)
    x, z, w = rnd(2000, 16, 192, seed=8), rnd(2000, 16, 192, seed=9), rnd(16, 192, seed=10, dtype=torch.float32)
    one, pools = {n: t[:, 0].contiguous() for n, t in d.items()}, [s0.clone() for _ in range(8)]
    return {
        "gated_delta_chunk_fwd": lambda **kw: gla.gated_delta_chunk_fwd(**d, s0=s0, **kw),
        "gated_delta_chunk_bwd": lambda **kw: gla.gated_delta_chunk_bwd(**d, dO=dO, s0=s0, **kw),
        "gated_delta_decode_step": lambda **kw: (gla.gated_delta_decode_step(pools.pop(), **one, **kw),),
        "group_norm_silu": lambda **kw: (gla.group_norm_silu(x, w, gate=z, **kw),),
        "group_norm_silu_bwd": lambda **kw: gla.group_norm_silu_bwd(x, z, w, gate=z, **kw),
    }


def workspace_bytes(name):
    if name.startswith("gated_delta_chunk"):
        return gla.gated_delta_chunk_workspace_bytes(4, 1024, 16, for_bwd=name.endswith("bwd"))
    return gla.group_norm_silu_bwd_workspace_bytes(2000, 16, 192) if name == "group_norm_silu_bwd" else 0


DELTA = ["gated_delta_chunk_fwd", "gated_delta_chunk_bwd", "gated_delta_decode_step", "group_norm_silu",
         "group_norm_silu_bwd"]


def check_outputs(call):
    """Work that the current stream still has to do on a block it freed does not
    reach the call's outputs."""
    want = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i, ref in enumerate(want):
        torch.cuda.synchronize()
        torch.cuda._sleep(LONG)
        held = [torch.empty_like(ref) for _ in range(4)]
        for t in held:
            t.fill_(7)
        del held, t
        got = [t for t in call(stream=side) if t is not None]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i


def check_workspace(call, need):
    """Writes of the current stream into blocks of the workspace's size, all
    through the call, do not reach the workspace."""
    want = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = [t for t in call(stream=side) if t is not None]
        for _ in range(40):
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", DELTA)
def test_outputs_of_the_delta_rule_and_the_norm(name):
    check_outputs(delta_calls()[name])


@pytest.mark.parametrize("name", ["gated_delta_chunk_fwd", "gated_delta_chunk_bwd", "group_norm_silu_bwd"])
def test_workspaces_of_the_delta_rule_and_the_norm(name):
    check_workspace(delta_calls()[name], workspace_bytes(name))


@pytest.mark.parametrize("name", DELTA)
def test_an_output_dropped_here_is_not_reused_there(name):
    """An output read on the current stream and dropped: the next call on the other
    stream does not write into it before the read is done."""
    call = delta_calls()[name]
    want = [t for t in call() if t is not None]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    got = [t for t in call(stream=side) if t is not None]
    here.wait_stream(side)
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full(s, 3, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(copies, want)) and len(over) == len(want)


# ---------------------------------------------------------------- the other entry points
def mixer_calls():
    B, T, H, D = 8, 1024, 16, 1024
    d = dict(q=rnd(B, T, H, 96, seed=21), k=rnd(B, T, H, 96, seed=22), v=rnd(B, T, H, 192, seed=23),
             a=torch.nn.functional.logsigmoid(rnd(B, T, H, seed=24, dtype=torch.float32) + 3))
    dO, s0 = rnd(B, T, H, 192, seed=25), rnd(B, H, 96, 192, seed=26, dtype=torch.float32, std=0.1)
    saved = gla.gla_chunk_fwd_train(**d)[2]
    flat = {n: t.flatten(0, 1) for n, t in d.items()}
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    one, pools = {n: t[:, 0].contiguous() for n, t in d.items()}, [s0.clone() for _ in range(8)]
    g = -rnd(B, H, seed=27, dtype=torch.float32).abs()
    x, dy, w = rnd(4, 2048, D, seed=28), rnd(4, 2048, D, seed=29), rnd(D, 4, seed=30, dtype=torch.float32, std=0.5)
    histories, x1 = [rnd(64, 3, D, seed=31, dtype=torch.float32) for _ in range(8)], rnd(64, D, seed=32)
    return {
        "gla_chunk_fwd": lambda **kw: gla.gla_chunk_fwd(**d, s0=s0, **kw),
        "gla_chunk_fwd_noalloc": lambda **kw: gla.gla_chunk_fwd_noalloc(**{n: t[:1, :128] for n, t in d.items()}, **kw),
        "gla_chunk_fwd_varlen": lambda **kw: gla.gla_chunk_fwd_varlen(**flat, cu_seqlens=cu, **kw),
        "gla_chunk_fwd_train": lambda **kw: gla.gla_chunk_fwd_train(**d, s0=s0, **kw)[:2],
        "gla_chunk_bwd": lambda **kw: gla.gla_chunk_bwd(**d, dO=dO, s0=s0, **kw),
        "gla_chunk_bwd_saved": lambda **kw: gla.gla_chunk_bwd_saved(**d, saved=saved, dO=dO, **kw),
        "gla_decode_step": lambda **kw: (gla.gla_decode_step(pools.pop(), **one, **kw),),
        "gla_segment_state_fwd": lambda **kw: gla.gla_segment_state_fwd(d["k"], d["v"], d["a"], **kw),
        "gla_segment_state_bwd": lambda **kw: gla.gla_segment_state_bwd(d["q"], dO, d["a"], want_decay=True, **kw),
        "gla_state_fold": lambda **kw: (gla.gla_state_fold(s0, g, **kw),),
        "conv1d_silu_causal": lambda **kw: (gla.conv1d_silu_causal(x, w, **kw),),
        "conv1d_silu_causal_bwd": lambda **kw: tuple(gla.conv1d_silu_causal_bwd(x, w, dy, **kw).values()),
        "conv1d_silu_decode_step": lambda **kw: (gla.conv1d_silu_decode_step(x1, w, histories.pop(), **kw),),
    }


MIXER = ["gla_chunk_fwd", "gla_chunk_fwd_noalloc", "gla_chunk_fwd_varlen", "gla_chunk_fwd_train", "gla_chunk_bwd",
         "gla_chunk_bwd_saved", "gla_decode_step", "gla_segment_state_fwd", "gla_segment_state_bwd", "gla_state_fold",
         "conv1d_silu_causal", "conv1d_silu_causal_bwd", "conv1d_silu_decode_step"]


@pytest.mark.parametrize("name", MIXER)
def test_outputs_of_the_mixer_and_its_front_end(name):
    check_outputs(mixer_calls()[name])


@pytest.mark.parametrize("name", ["gla_chunk_bwd", "gla_chunk_bwd_saved", "gla_segment_state_fwd",
                                  "gla_segment_state_bwd", "conv1d_silu_causal_bwd"])
def test_workspaces_of_the_mixer_and_its_front_end(name):
    need = {"gla_chunk_bwd": lambda: gla.gla_chunk_workspace_bytes(8, 1024, 16, for_bwd=True),
            "gla_chunk_bwd_saved": lambda: gla.gla_chunk_workspace_bytes(8, 1024, 16, for_bwd=True, from_saved=True),
            "conv1d_silu_causal_bwd": lambda: gla.conv1d_silu_causal_bwd_workspace_bytes(4, 2048, 1024),
            }.get(name, lambda: gla.gla_segment_workspace_bytes(8, 1024, 16))()
    assert need > 0
    check_workspace(mixer_calls()[name], need)


@pytest.mark.parametrize("name", DELTA)
def test_a_captured_call_that_is_given_the_captures_own_stream(name):
    call = delta_calls()[name]
    want = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [t for t in call(stream=torch.cuda.current_stream()) if t is not None]
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_threads_with_a_stream_each():
    """Host threads that call at once, each on a stream of its own and with what the
    binding allocates."""
    import threading
    calls, wants, errors = delta_calls(), {}, []
    names = [n for n in DELTA if n != "gated_delta_decode_step"]
    for n in names:
        wants[n] = [t for t in calls[n]() if t is not None]
    torch.cuda.synchronize()

    def work(n):
        side = torch.cuda.Stream()
        for _ in range(6):
            got = [t for t in calls[n](stream=side) if t is not None]
            side.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(got, wants[n])):
                errors.append(n)

    threads = [threading.Thread(target=work, args=(n,)) for n in names]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads)
