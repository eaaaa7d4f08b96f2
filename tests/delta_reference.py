"""Plain 64-bit forms of the gated delta rule and of the group norm with an
activation, for the tests: the token recurrence and its gradients by autograd."""
import torch


def recurrence(q, k, v, a, beta, s0, scale):
    """q, k [N,T,Hk,dk], v [N,T,H,dv], a, beta [N,T,H], s0 [N,H,dk,dv] (float64) -> o, S_T."""
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    S, outs = s0, []
    for t in range(v.shape[1]):
        S = S * a[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("nhi,nhij->nhj", k[:, t], S))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        outs.append(scale * torch.einsum("nhi,nhij->nhj", q[:, t], S))
    return (torch.stack(outs, 1) if outs else torch.zeros_like(v)), S


def sequences(d, cu=None):
    """The per-sequence slices of packed inputs d (dict of [T, ...] tensors)."""
    return [{n: x[int(b):int(e)][None] for n, x in d.items()} for b, e in zip(cu[:-1], cu[1:])]


def forward(d, s0, scale, cu=None):
    d = {n: x.double() for n, x in d.items()}
    s0 = s0.double()
    if cu is None:
        return recurrence(d["q"], d["k"], d["v"], d["a"], d["beta"], s0, scale)
    outs = [recurrence(x["q"], x["k"], x["v"], x["a"], x["beta"], s0[i:i + 1], scale)
            for i, x in enumerate(sequences(d, cu))]
    return torch.cat([o[0] for o, _ in outs]), torch.cat([s for _, s in outs])


def backward(d, s0, dO, ds, scale, cu=None):
    """Gradients of <o, dO> + <S_T, ds>: dq, dk, dv, da, dbeta, ds0."""
    leaves = {n: x.double().requires_grad_(True) for n, x in d.items()}
    s0 = s0.double().requires_grad_(True)
    if cu is None:
        o, s = recurrence(*[leaves[n] for n in ("q", "k", "v", "a", "beta")], s0, scale)
        loss = (o * dO.double()).sum() + (s * ds.double()).sum()
    else:
        loss = 0
        for i, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
            x = {n: t[int(b):int(e)][None] for n, t in leaves.items()}
            o, s = recurrence(x["q"], x["k"], x["v"], x["a"], x["beta"], s0[i:i + 1], scale)
            loss = loss + (o[0] * dO[int(b):int(e)].double()).sum() + (s * ds[i:i + 1].double()).sum()
    return torch.autograd.grad(loss, [leaves[n] for n in ("q", "k", "v", "a", "beta")] + [s0], allow_unused=True)


def norm(x, weight, bias, gate, center, act, eps):
    c = x - x.mean(-1, keepdim=True) if center else x
    n = c / (c.square().mean(-1, keepdim=True) + eps).sqrt()
    n = n * (weight if weight is not None else 1.0) + (bias if bias is not None else 0.0)
    f = (lambda z: z / (1 + torch.exp(-z))) if act else (lambda z: z)
    return f(n) if gate is None else n * f(gate)


def rel(x, ref):
    """Relative 2-norm of the difference (0 when both are 0)."""
    x, ref = x.detach().double(), ref.detach().double()
    d, n = float((x - ref).norm()), float(ref.norm())
    return d / n if n else (0.0 if d == 0.0 else float("inf"))
