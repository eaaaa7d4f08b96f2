"""What the checking build (GLA_DEBUG_BOUNDS) scans of the gated delta rule's
inputs, in a child process that loads it: every tensor that a call reads is
scanned, and nothing that it does not read."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = r'''
import torch
import linear_attention_simple_b200 as gla
assert gla.gla_build_flags() == gla.GLA_BUILD_DEBUG_BOUNDS, "the checking build is not the one loaded"
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
NAMES = ("q", "k", "v", "a", "beta")

def make(lead, Hk, H, dk, dv, dt):
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)
    return dict(q=unit(rnd(*lead, Hk, dk)), k=unit(rnd(*lead, Hk, dk)), v=rnd(*lead, H, dv).to(dt),
                a=-rnd(*lead, H).abs(), beta=torch.sigmoid(rnd(*lead, H)))

def spoil(x, *at, to=float("nan")):
    x = x.clone()
    x[at] = to
    return x

def status(what, want):
    got = gla.gla_get_device_status()
    assert got == want, "%s: status %d, expected %d" % (what, got, want)

# the step, both types: inputs, decays, strengths, and the states it addresses
for dt in (torch.bfloat16, torch.float32):
    for tokens in (1, 3):
        d = make((4, tokens), 1, 2, 64, 32, dt)
        pool, idx = 0.1 * rnd(7, 2, 64, 32), torch.tensor([5, 0, 3, 6], dtype=torch.int32, device="cuda")
        step = lambda pool, **kw: gla.gated_delta_decode_step(pool.clone(), *[dict(d, **kw)[n] for n in NAMES], slot_idx=idx)
        step(pool)
        status("step", 0)
        for n in NAMES:
            step(pool, **{n: spoil(d[n], 3, tokens - 1, 0)})
            status("step: NaN in %s, %s" % (n, dt), 1)
        step(pool, a=spoil(d["a"], 0, 0, 1, to=0.5))
        status("step: a > 0", 1)
        step(spoil(pool, 6, 1, 63, 31))
        status("step: NaN in an addressed state", 1)
        step(spoil(spoil(pool, 1), 4, to=float("inf")))
        status("step: NaN in slots of other sequences", 0)
        step(spoil(pool, 2), q=d["q"])
        status("step: NaN in another slot", 0)
# views into a fused projection: what lies between the rows is not read
d = make((4, 3), 1, 2, 64, 64, torch.float32)
buf = torch.full((4, 3, 64 + 64 + 128 + 8), float("nan"), device="cuda")
views, at = {}, 0
for n in ("q", "k", "v"):
    w = d[n].shape[-1] * d[n].shape[-2]
    buf[..., at:at + w] = d[n].flatten(-2)
    views[n] = buf[..., at:at + w].unflatten(-1, d[n].shape[-2:])
    at += w
gla.gated_delta_decode_step(0.1 * rnd(4, 2, 64, 64), *[dict(d, **views)[n] for n in NAMES])
status("step: views", 0)
buf[3, 2, 64 + 5] = float("inf")
gla.gated_delta_decode_step(0.1 * rnd(4, 2, 64, 64), *[dict(d, **views)[n] for n in NAMES])
status("step: inf in a view", 1)
# a slot outside the pool: reported by the step itself, and its state not read
d = make((2, 1), 1, 1, 64, 32, torch.bfloat16)
gla.gated_delta_decode_step(0.1 * rnd(2, 1, 64, 32), *[d[n] for n in NAMES],
                            slot_idx=torch.tensor([-1, 2], dtype=torch.int32, device="cuda"))
status("step: slots outside the pool", 1)

# the chunked calls
d, s0, ds = make((2, 70), 1, 2, 64, 32, torch.bfloat16), 0.1 * rnd(2, 2, 64, 32), 0.1 * rnd(2, 2, 64, 32)
dO = rnd(2, 70, 2, 32).bfloat16()
ins = lambda **kw: [dict(d, **kw)[n] for n in NAMES]
gla.gated_delta_chunk_fwd(*ins(), s0=s0)
gla.gated_delta_chunk_bwd(*ins(), dO, s0=s0, ds_final=ds)
status("chunked", 0)
for n in NAMES:
    bad = spoil(d[n], 1, 69, 0)
    gla.gated_delta_chunk_fwd(*ins(**{n: bad}), s0=s0)
    status("forward: NaN in " + n, 1)
    gla.gated_delta_chunk_bwd(*ins(**{n: bad}), dO, s0=s0)
    status("backward: NaN in " + n, 1)
gla.gated_delta_chunk_fwd(*ins(), s0=spoil(s0, 1, 1, 63, 31))
status("forward: NaN in s0", 1)
gla.gated_delta_chunk_bwd(*ins(), spoil(dO, 1, 69, 1, 31), s0=s0, ds_final=ds)
status("backward: NaN in dO", 1)
gla.gated_delta_chunk_bwd(*ins(), dO, s0=s0, ds_final=spoil(ds, 1, 1, 63, 31, to=float("inf")))
status("backward: inf in ds_final", 1)

# packed: rows outside every sequence may hold anything
d, dO = make((160,), 1, 2, 64, 32, torch.bfloat16), rnd(160, 2, 32).bfloat16()
cu = torch.tensor([7, 80, 80, 150], dtype=torch.int32, device="cuda")
for n in NAMES:
    for row, want in ((6, 0), (150, 0), (159, 0), (7, 1), (149, 1)):
        gla.gated_delta_chunk_fwd(*ins(**{n: spoil(d[n], row)}), cu_seqlens=cu)
        status("packed forward: NaN in %s of row %d" % (n, row), want)
for row, want in ((6, 0), (150, 0), (7, 1), (149, 1)):
    gla.gated_delta_chunk_bwd(*ins(), spoil(dO, row), cu_seqlens=cu)
    status("packed backward: NaN in dO of row %d" % row, want)
# offsets outside the rows: reported, the scan keeps inside
for bad in ([0, 50, 200], [-5, 50, 100], [90, 20, 10]):
    gla.gated_delta_chunk_fwd(*ins(), cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"))
    status("offsets %s" % bad, 1)
gla.gated_delta_chunk_fwd(*ins(), cu_seqlens=cu)
status("afterwards", 0)
print("scans ok")
'''


@pytest.mark.gpu
def test_scans_of_the_gated_delta_rule():
    from linear_attention_simple_b200 import build
    build.build(debug=True)
    env = dict(os.environ, GLA_DEBUG_BOUNDS="1", PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", _CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    print(r.stdout[-2000:], r.stderr[-4000:])
    assert r.returncode == 0, r.stderr[-4000:]
    assert "scans ok" in r.stdout
