"""Cases of the gated delta rule and of the group norm with an activation.

For each case: its inputs, one pass through the operator (in a plain form of
elementary torch operations, or through this package's entry points), the bytes
and operations that a pass cannot do without, and the result in 64 bits.

Gated delta rule, per (sequence, head), with log-decay a_t <= 0 and write
strength beta_t:

    S'_t = exp(a_t) S_{t-1}
    S_t  = S'_t + k_t^T beta_t (v_t - k_t S'_t)       S: dk x dv
    o_t  = scale * q_t S_t

q and k have Hk heads, v has H; value head h reads q, k of head h // (H / Hk).

Group norm with an activation, per token row and group of d channels:

    n = (x - mean) * rstd * weight + bias     (mean taken as 0 when not centred)
    y = n * silu(gate), or silu(n) without a gate
"""
import math

import torch

own = False

CHUNK = 64


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one layer's prefill of a batch of prompts of 2,048 tokens
        dict(name="chunk_fwd_prefill", op="chunk_fwd", N=8, T=2048, H=16, Hk=16, dk=96, dv=192, packed=False, s0=False),
        # a serving step: seven prompts of uneven lengths packed together, continued from earlier states
        dict(name="chunk_fwd_packed", op="chunk_fwd", N=7, T=1205, H=16, Hk=16, dk=96, dv=192, packed=True, s0=True),
        # one long prompt, value heads that share q and k heads
        dict(name="chunk_fwd_long", op="chunk_fwd", N=1, T=16384, H=16, Hk=8, dk=128, dv=128, packed=False, s0=False),
        # the training step's backward
        dict(name="chunk_bwd_train", op="chunk_bwd", N=8, T=2048, H=16, Hk=16, dk=96, dv=192, packed=False, s0=False),
        # a short odd length, shared heads, gradients of the initial state too
        dict(name="chunk_bwd_odd", op="chunk_bwd", N=2, T=555, H=8, Hk=4, dk=128, dv=128, packed=False, s0=True),
        # documents of uneven lengths packed into one row
        dict(name="chunk_bwd_packed", op="chunk_bwd", N=5, T=2811, H=16, Hk=16, dk=96, dv=192, packed=True, s0=False),
        # one decoded token for three sequences: latency counts
        dict(name="step_few", op="step", N=3, T=1, H=16, Hk=16, dk=96, dv=192, dtype="bf16"),
        # one decoded token for 1,280 sequences
        dict(name="step_many", op="step", N=1280, T=1, H=16, Hk=16, dk=96, dv=192, dtype="bf16"),
        # four drafted tokens for each of 37 sequences, shared heads, fp32 inputs
        dict(name="step_drafted", op="step", N=37, T=4, H=16, Hk=8, dk=128, dv=128, dtype="f32"),
        # the mixer's output of a training batch: centred, gated
        dict(name="norm_fwd_train", op="norm_fwd", M=16384, G=16, d=192, dtype="bf16", gate=True, center=True, shared=False, bias=True),
        # the decode step's fp32 output: root mean square only, one weight for all heads
        dict(name="norm_fwd_step", op="norm_fwd", M=37, G=16, d=128, dtype="f32", gate=True, center=False, shared=True, bias=False),
        # its backward over the training batch
        dict(name="norm_bwd_train", op="norm_bwd", M=16384, G=16, d=192, dtype="bf16", gate=True, center=True, shared=False, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk_fwd", "chunk_bwd", "step", "norm_fwd", "norm_bwd"])
    if op.startswith("norm"):
        G, d = rng.choice([1, 2, 5, 8, 16, 32]), 8 * rng.randint(1, 32)
        M = _log(rng, 1, min(16384, 16384 * 16 * 192 // (G * d)))
        return dict(op=op, M=M, G=G, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), gate=rng.random() < 0.7,
                    center=rng.random() < 0.5, shared=rng.random() < 0.5, bias=rng.random() < 0.5)
    dk, dv = rng.choice([(96, 192), (96, 192), (128, 128), (64, 64), (64, 128), (96, 96), (128, 256)])
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 3]) if Hk < 16 else 16
    if op == "step":
        T = rng.choice([1, 1, 1, 2, 3, 5, 8])
        N = _log(rng, 1, max(1, 1280 * 16 * 96 * 192 // (H * dk * dv * T)))
        return dict(op=op, N=min(N, 1280), T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=rng.choice(["bf16", "bf16", "f32"]))
    N = _log(rng, 1, 12)
    most = 8 * 2048 * 16 * 96 * 192 // (N * H * dk * dv)
    T = _log(rng, 1, max(1, min(most, 8192)))
    return dict(op=op, N=N, T=T, H=H, Hk=Hk, dk=dk, dv=dv, packed=rng.random() < 0.5, s0=rng.random() < 0.5)


def _lengths(case):
    """Lengths of a packed batch, around T; the third is empty and the fourth a
    single token, as a serving step has them."""
    n, T = case["N"], case["T"]
    return [0 if i == 2 else 1 if i == 3 else max(1, T * (1 + 7 * i % 8) // 8) for i in range(n)]


# ---------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda")


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std + mean

    st = dict(case=dict(case))
    if case["op"].startswith("norm"):
        M, G, d = case["M"], case["G"], case["d"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = rnd(M, G, d, std=0.3, mean=0.05).to(dt)
        st["gate"] = rnd(M, G, d).bfloat16() if case["gate"] else None
        wshape = (d,) if case["shared"] else (G, d)
        st["weight"] = rnd(*wshape, mean=1.0, std=0.2)
        st["bias"] = rnd(*wshape, std=0.2) if case["bias"] else None
        if case["op"] == "norm_bwd":
            st["dy"] = rnd(M, G, d).bfloat16()
        return st
    N, T, H, Hk, dk, dv = (case[n] for n in ("N", "T", "H", "Hk", "dk", "dv"))
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    lead = (N, T)
    if case.get("packed"):
        lens = _lengths(case)
        st["lens"] = lens
        cu = [0]
        cu.extend(sum(lens[:i + 1]) for i in range(N))
        st["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        lead = (cu[-1],)

    def unit(x):  # the keys and queries of a delta rule have unit length
        return x / x.square().sum(-1, keepdim=True).sqrt()

    st["q"] = unit(rnd(*lead, Hk, dk)).to(dt)
    st["k"] = unit(rnd(*lead, Hk, dk) + 0.3 * rnd(*(1,) * len(lead), Hk, dk)).to(dt)
    st["v"] = rnd(*lead, H, dv).to(dt)
    st["a"] = torch.nn.functional.logsigmoid(rnd(*lead, H, mean=3.0))
    st["beta"] = torch.sigmoid(rnd(*lead, H))
    st["scale"] = dk ** -0.5
    if case["op"] == "step":
        # a pool with more slots than sequences, each sequence at a slot of its own
        slots = N + max(1, N // 8)
        st["state"] = rnd(slots, H, dk, dv, std=0.1)
        st["slot_idx"] = torch.randperm(slots, generator=g, device=dev)[:N].to(torch.int32)
        return st
    st["s0"] = rnd(N, H, dk, dv, std=0.1) if case["s0"] else None
    if case["op"] == "chunk_bwd":
        st["dO"] = rnd(*lead, H, dv).bfloat16()
        st["ds_final"] = rnd(N, H, dk, dv, std=0.1) if case["s0"] else None
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import linear_attention_simple_b200 as L
    case = st["case"]
    op = case["op"]
    if op == "norm_fwd":
        return L.group_norm_silu(st["x"], st["weight"], st["bias"], st["gate"], center=case["center"])
    if op == "norm_bwd":
        return _present(L.group_norm_silu_bwd(st["x"], st["dy"], st["weight"], st["bias"], st["gate"],
                                              center=case["center"]))
    ins = (st["q"], st["k"], st["v"], st["a"], st["beta"])
    if op == "step":
        o = L.gated_delta_decode_step(st["state"], *ins, slot_idx=st["slot_idx"], scale=st["scale"])
        return o, st["state"]
    cu = st.get("cu_seqlens")
    if op == "chunk_fwd":
        return L.gated_delta_chunk_fwd(*ins, s0=st["s0"], cu_seqlens=cu, scale=st["scale"])
    return _present(L.gated_delta_chunk_bwd(*ins, st["dO"], s0=st["s0"], ds_final=st["ds_final"], cu_seqlens=cu,
                                            scale=st["scale"], want_grad_s0=st["s0"] is not None))


def _present(outs):
    return [x for x in outs if x is not None]


def _run_plain(st):
    op = st["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm(st, st["x"].float(), *_norm_leaves(st, False)).bfloat16()
    if op == "norm_bwd":
        x = st["x"].float().requires_grad_(True)
        leaves = _norm_leaves(st, True)
        y = _plain_norm(st, x, *leaves)
        wanted = [x, leaves[2], leaves[0], leaves[1]]
        grads = torch.autograd.grad(y, _present(wanted), st["dy"].float())
        types = [st["x"].dtype] + ([torch.bfloat16] if st["gate"] is not None else []) + [torch.float32] * 2
        return [g.to(t) for g, t in zip(grads, types)]
    if op == "step":
        return _plain_step(st)
    if op == "chunk_fwd":
        o, s = _plain_chunked(st, *[st[n].float() for n in ("q", "k", "v", "a", "beta")], st["s0"])
        return o.bfloat16(), s
    ins = [st[n].float().detach().clone().requires_grad_(True) for n in ("q", "k", "v", "a", "beta")]
    s0 = st["s0"].detach().clone().requires_grad_(True) if st["s0"] is not None else None
    o, s = _plain_chunked(st, *ins, s0)
    outs, gos = [o], [st["dO"].float()]
    if st["ds_final"] is not None:
        outs, gos = outs + [s], gos + [st["ds_final"]]
    grads = torch.autograd.grad(outs, _present(ins + [s0]), gos)
    return [g.bfloat16() for g in grads[:3]] + list(grads[3:])


def _norm_leaves(st, grad):
    return [None if st[n] is None else st[n].float().detach().clone().requires_grad_(grad)
            for n in ("weight", "bias", "gate")]


def _plain_norm(st, x, weight, bias, gate):
    mean = x.mean(-1, keepdim=True) if st["case"]["center"] else 0.0
    c = x - mean
    n = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5) * weight
    if bias is not None:
        n = n + bias
    return n * torch.sigmoid(n) if gate is None else n * (gate * torch.sigmoid(gate))


def _plain_step(st):
    rep = st["case"]["H"] // st["case"]["Hk"]
    q = st["q"].float().repeat_interleave(rep, 2)
    k = st["k"].float().repeat_interleave(rep, 2)
    v, e, beta = st["v"].float(), torch.exp(st["a"]), st["beta"]
    at = st["slot_idx"].long()
    S, outs = st["state"][at], []
    for t in range(q.shape[1]):  # the tokens of a sequence are in order
        S = S * e[:, t, :, None, None]
        u = (v[:, t] - (k[:, t, :, None] @ S)[:, :, 0]) * beta[:, t, :, None]
        S = S + k[:, t, :, :, None] * u[:, :, None]
        outs.append((q[:, t, :, None] @ S)[:, :, 0] * st["scale"])
    st["state"][at] = S
    return torch.stack(outs, 1), st["state"]


def _rows_of(st, T):
    """For a packed batch: the row of each (sequence, token) and whether there is one."""
    cu = st["cu_seqlens"].long()
    t = torch.arange(T, device=cu.device)
    inside = t[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(inside, cu[:-1, None] + t[None], 0), inside


def _inverse(M):
    """The inverse of unit lower triangular matrices, by halves."""
    n = M.shape[-1]
    if n == 1:
        return torch.ones_like(M)
    h = n // 2
    a, b = _inverse(M[..., :h, :h]), _inverse(M[..., h:, h:])
    low = -(b @ M[..., h:, :h] @ a)
    return torch.cat([torch.cat([a, torch.zeros_like(low.mT)], -1), torch.cat([low, b], -1)], -2)


def _plain_chunked(st, q, k, v, a, beta, s0):
    case = st["case"]
    N, H, dk, dv = (case[n] for n in ("N", "H", "dk", "dv"))
    packed = case["packed"]
    T = max(st["lens"]) if packed else case["T"]
    nc = -(-T // CHUNK)
    Tp = nc * CHUNK
    if packed:
        rows, inside = _rows_of(st, Tp)

    def lay(x, heads):  # [N, H, chunks, CHUNK, width], zero behind a sequence's end
        x = x.reshape(*x.shape[:x.dim() - (2 if heads else 1)], x.shape[-2] if heads else H, -1)
        if packed:
            x = torch.where(inside[..., None, None], x[rows], 0.0)
        elif Tp > T:
            x = torch.cat([x, x.new_zeros(N, Tp - T, *x.shape[2:])], 1)
        if x.shape[2] != H:
            x = x.repeat_interleave(H // x.shape[2], 2)
        return x.reshape(N, nc, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    q, k, v = lay(q, True) * st["scale"], lay(k, True), lay(v, True)
    a, beta = lay(a, False)[..., 0], lay(beta, False)
    b = a.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], 0.0)), 0.0)
    inv = _inverse((k @ k.mT) * decay.tril(-1) * beta + torch.eye(CHUNK, device=q.device))
    grow, rest = torch.exp(b)[..., None], torch.exp(b[..., -1:] - b)[..., None]
    u, w = inv @ (v * beta), inv @ (k * beta * grow)
    scores = (q @ k.mT) * decay
    S = s0 if s0 is not None else q.new_zeros(N, H, dk, dv)
    outs = []
    for c in range(nc):  # a chunk starts from the state that the one before it leaves
        new = u[:, :, c] - w[:, :, c] @ S
        outs.append((q[:, :, c] * grow[:, :, c]) @ S + scores[:, :, c] @ new)
        S = S * grow[:, :, c, -1:] + (k[:, :, c] * rest[:, :, c]).mT @ new
    o = torch.stack(outs, 2).permute(0, 2, 3, 1, 4).reshape(N, Tp, H, dv)
    return (o[inside] if packed else o[:, :T]), S


# ---------------------------------------------------------------- floors
def work(case):
    if case["op"].startswith("norm"):
        n, size = case["M"] * case["G"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        gate = 2 if case["gate"] else 0
        params = 4 * (case["d"] if case["shared"] else case["G"] * case["d"]) * (2 if case["bias"] else 1)
        if case["op"] == "norm_fwd":
            return {"bytes": n * (size + gate + 2) + params, "flops": 12.0 * n}
        return {"bytes": n * (2 * size + 2 * gate + 2) + 2 * params, "flops": 30.0 * n}
    N, T, H, Hk, dk, dv = (case[n] for n in ("N", "T", "H", "Hk", "dk", "dv"))
    tokens = sum(_lengths(case)) if case.get("packed") else N * T
    size = 4 if case.get("dtype") == "f32" else 2
    row = size * (2 * Hk * dk + H * dv) + 8 * H
    states = 4 * N * H * dk * dv
    if case["op"] == "step":
        return {"bytes": tokens * (row + 4 * H * dv) + 2 * states, "flops": 7.0 * tokens * H * dk * dv}
    starts = 1 if case["s0"] else 0
    if case["op"] == "chunk_fwd":
        return {"bytes": tokens * (row + 2 * H * dv) + states * (1 + starts), "flops": 6.0 * tokens * H * dk * dv}
    return {"bytes": tokens * (2 * row + 2 * H * dv) + states * 3 * starts, "flops": 18.0 * tokens * H * dk * dv}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(st)
    if case["op"] == "step":
        return _exact_step(st)
    return _exact_sequence(st)


def _exact_norm(st):
    case = st["case"]
    x, w = st["x"].double(), st["weight"].double()
    mean = x.mean(-1, keepdim=True) if case["center"] else torch.zeros_like(x[..., :1])
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + 1e-5).sqrt()
    xh = (x - mean) * rstd
    n = xh * w + (st["bias"].double() if st["bias"] is not None else 0.0)
    z = st["gate"].double() if st["gate"] is not None else n
    sg = 1 / (1 + torch.exp(-z))
    if case["op"] == "norm_fwd":
        return n * z * sg if st["gate"] is not None else z * sg
    dy = st["dy"].double()
    slope = sg * (1 + z * (1 - sg))
    dn = dy * z * sg if st["gate"] is not None else dy * slope
    dxh = dn * w
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - dxh.mean(-1, keepdim=True)
    over = (0, 1) if case["shared"] else (0,)
    outs = [dx * rstd]
    if st["gate"] is not None:
        outs.append(dy * n * slope)
    outs.append((dn * xh).sum(over))
    if st["bias"] is not None:
        outs.append(dn.sum(over))
    return outs


def _exact_step(st):
    case = st["case"]
    heads = torch.arange(case["H"], device=_device()) // (case["H"] // case["Hk"])
    state = st["state"].double()
    at = st["slot_idx"].long()
    q, k, v = st["q"].double()[:, :, heads], st["k"].double()[:, :, heads], st["v"].double()
    S = state[at]
    o = torch.empty_like(v)
    for t in range(case["T"]):
        S, o[:, t], _, _ = _token(S, q[:, t], k[:, t], v[:, t], st["a"][:, t].double(), st["beta"][:, t].double(),
                                  st["scale"])
    state[at] = S
    return o, state


def _token(S, q, k, v, a, beta, scale):
    """One token of the recurrence: the new state, the output, the decayed state and v minus its prediction."""
    decayed = S * a.exp()[..., None, None]
    z = v - torch.einsum("nhi,nhij->nhj", k, decayed)
    S = decayed + torch.einsum("nhi,nhj->nhij", k, z * beta[..., None])
    return S, scale * torch.einsum("nhi,nhij->nhj", q, S), decayed, z


def _exact_sequence(st):
    case = st["case"]
    N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
    heads = torch.arange(H, device=_device()) // (H // Hk)
    lens = st["lens"] if case["packed"] else [case["T"]] * N
    T, first = max(lens), [sum(lens[:i]) for i in range(N)]
    bwd = case["op"] == "chunk_bwd"

    def spread(x):  # [N, T, ...] in 64 bits; tokens behind the end change nothing (k, v, beta and a of zero)
        if not case["packed"]:
            return x.double()
        y = torch.zeros(N, T, *x.shape[1:], dtype=torch.float64, device=x.device)
        for n in range(N):
            y[n, :lens[n]] = x[first[n]:first[n] + lens[n]].double()
        return y

    def gather(y):
        return torch.cat([y[n, :lens[n]] for n in range(N)]) if case["packed"] else y

    q, k, v, a, beta = (spread(st[n]) for n in ("q", "k", "v", "a", "beta"))
    q, k = q[:, :, heads], k[:, :, heads]
    S = st["s0"].double() if st["s0"] is not None else torch.zeros(N, H, dk, dv, dtype=torch.float64, device=q.device)
    o, scale, every, kept = torch.zeros_like(v), st["scale"], 64, []
    for t in range(T):
        if bwd and t % every == 0:
            kept.append(S)
        S, o[:, t], _, _ = _token(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t], scale)
    if not bwd:
        return gather(o), S
    dO = spread(st["dO"])
    E = st["ds_final"].double() if st["ds_final"] is not None else torch.zeros_like(S)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    da, db = torch.zeros_like(a), torch.zeros_like(beta)
    for c in reversed(range(len(kept))):
        span = range(c * every, min(T, (c + 1) * every))
        S, back = kept[c], []
        for t in span:
            S, _, decayed, z = _token(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t], scale)
            back.append((S, decayed, z))
        for t in reversed(span):
            S, decayed, z = back.pop()
            dq[:, t] = scale * torch.einsum("nhij,nhj->nhi", S, dO[:, t])
            E = E + scale * torch.einsum("nhi,nhj->nhij", q[:, t], dO[:, t])
            du = torch.einsum("nhi,nhij->nhj", k[:, t], E)
            db[:, t] = (du * z).sum(-1)
            dz = du * beta[:, t, :, None]
            dv_[:, t] = dz
            dk_[:, t] = torch.einsum("nhij,nhj->nhi", E, z * beta[:, t, :, None])
            dk_[:, t] -= torch.einsum("nhij,nhj->nhi", decayed, dz)
            E = E - torch.einsum("nhi,nhj->nhij", k[:, t], dz)
            da[:, t] = (E * decayed).sum((-1, -2))
            E = E * a[:, t].exp()[..., None, None]
    dq, dk_ = (x.reshape(N, T, Hk, H // Hk, dk).sum(3) for x in (dq, dk_))
    outs = [gather(x) for x in (dq, dk_, dv_, da, db)]
    return outs + ([E] if st["s0"] is not None else [])
