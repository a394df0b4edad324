"""Linear attention with a decay a head, its gradients, and the norms around a block, in 64 bits and token by token: what the
kernels are compared with.  Plain torch; every function takes tensors of any type and computes in float64 on their device."""
import torch

F64 = torch.float64


def sequences(cu, T):
    if cu is None:
        return [(0, T)]
    c = [int(x) for x in cu]
    return list(zip(c[:-1], c[1:]))


def wide(x, H):
    """[T, heads, d] in 64 bits with its heads repeated to H."""
    return x.to(F64).repeat_interleave(H // x.shape[1], 1)


def prefill(q, k, v, g, cu=None, first=None, scale=1.0):
    """(out [T, H, dv], last states [N, H, dk, dv]); tokens of no sequence are 0."""
    H = v.shape[1]
    q, k, v = wide(q, H), wide(k, H), v.to(F64)
    g = g.to(F64).expand(q.shape[0], H)
    out, last = torch.zeros_like(v), []
    for n, (a, b) in enumerate(sequences(cu, q.shape[0])):
        S = torch.zeros((H, q.shape[2], v.shape[2]), dtype=F64, device=q.device) if first is None else first[n].to(F64)
        for t in range(a, b):
            S = g[t].exp()[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * (q[t][:, :, None] * S).sum(1)
        last.append(S)
    return out, torch.stack(last)


def backward(q, k, v, g, do, cu=None, first=None, dlast=None, scale=1.0):
    """dict of dq, dk [T, Hk, dk], dv, dg (g's shape), dS0; and `each`, the terms of dg's running sum by size, per token and head."""
    H, Hk, fixed = v.shape[1], q.shape[1], g.dim() == 1
    q, k, v, do = wide(q, H), wide(k, H), v.to(F64), do.to(F64)
    T, dk_, dv_ = q.shape[0], q.shape[2], v.shape[2]
    g = g.to(F64).expand(T, H)
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g).clone()
    dS0 = []
    for n, (a, b) in enumerate(sequences(cu, T)):
        S = torch.zeros((H, dk_, dv_), dtype=F64, device=q.device) if first is None else first[n].to(F64)
        before = []
        for t in range(a, b):
            before.append(S)
            S = g[t].exp()[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (S * do[t][:, None, :]).sum(2)
        R = torch.zeros_like(S) if dlast is None else dlast[n].to(F64)
        for t in reversed(range(a, b)):
            R = R + scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = (R * v[t][:, None, :]).sum(2)
            dv[t] = (R * k[t][:, :, None]).sum(1)
            e = g[t].exp()[:, None, None]
            dg[t] = (e * before[t - a] * R).sum((1, 2))
            R = e * R
        dS0.append(R)
    group = H // Hk
    return {"dq": dq.view(T, Hk, group, dk_).sum(2), "dk": dk.view(T, Hk, group, dk_).sum(2), "dv": dv, "dg": dg.sum(0) if fixed else dg,
            "dS0": torch.stack(dS0), "each": (q * dq).sum(-1).abs() + (k * dk).sum(-1).abs(), "dg_token": dg}


def act(kind, z):
    return torch.sigmoid(z) if kind == "sigmoid" else z * torch.sigmoid(z)


def unit(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def block_norm(x, residual=None, gate=None, gate_act="sigmoid", post=None, pre=None, alpha=1.0, eps=1e-6):
    """(s, y or None)"""
    u = x.to(F64)
    if post is not None:
        u = unit(u, eps) * post.to(F64)
    if gate is not None:
        u = u * act(gate_act, gate.to(F64))
    s = alpha * u + (0 if residual is None else residual.to(F64))
    return s, None if pre is None else unit(s, eps) * pre.to(F64)


def block_norm_backward(x, ds, dy=None, sum=None, gate=None, gate_act="sigmoid", post=None, pre=None, alpha=1.0, eps=1e-6):
    """By automatic differentiation in 64 bits: dict of dx, dresidual, dgate, dpost, dpre."""
    d, out = ds.to(F64), {}
    if pre is not None:
        s, w = sum.to(F64).requires_grad_(), pre.to(F64).requires_grad_()
        a, out["dpre"] = torch.autograd.grad(unit(s, eps) * w, (s, w), dy.to(F64))
        d = d + a
    out["dresidual"] = d
    leaves = {"dx": x.to(F64).requires_grad_()}
    if gate is not None:
        leaves["dgate"] = gate.to(F64).requires_grad_()
    if post is not None:
        leaves["dpost"] = post.to(F64).requires_grad_()
    u, _ = block_norm(leaves["dx"], None, leaves.get("dgate"), gate_act, leaves.get("dpost"), None, alpha, eps)
    out.update(zip(leaves, torch.autograd.grad(u, list(leaves.values()), d)))
    return out
