"""A layer of linear attention between its norms, as a training step and a small serving loop would use it.

    python examples/linear_attention_layer.py [--dtype bf16|f32] [--steps 32]

The layer: a norm, projections to queries and keys of 2 heads that 8 heads of values share, a decay and a gate, linear
attention, a norm a head with the gate, the projection back, a norm, the residual and the next layer's norm.  The training part takes
the gradients of packed sequences in FP32 by the library's backward calls and compares all of them with automatic
differentiation in float64.  The serving part runs prompts into a pool of states, then decodes token by token: one CUDA graph
holds the operators of a step and is replayed.  Each operator's result is compared with plain torch on what it was given.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_linear_attention_rule_gb300 as K  # noqa: E402

WIDTH, HK, H, DK, DV, EPS = 256, 2, 8, 64, 64, 1e-6
PARTS = [HK * DK, HK * DK, H * DV, H * DV, H]                                 # queries, keys, values, gate, decay


def weights(dev):
    rnd = lambda *s: torch.randn(s, device=dev)                               # noqa: E731
    return {"first": 1 + 0.1 * rnd(WIDTH), "w_in": rnd(WIDTH, sum(PARTS)) / WIDTH ** 0.5, "head": 1 + 0.1 * rnd(DV),
            "w_out": rnd(H * DV, WIDTH) / (H * DV) ** 0.5, "post": 1 + 0.1 * rnd(WIDTH), "pre": 1 + 0.1 * rnd(WIDTH)}


def split(p):
    """The projection's output in its parts; the decay is the logarithm of a sigmoid, in the projection's type."""
    q, k, v, z, d = p.split(PARTS, -1)
    heads = lambda x, n: x.unflatten(-1, (n, -1)).contiguous()                # noqa: E731
    return heads(q, HK), heads(k, HK), heads(v, H), heads(z, H), torch.nn.functional.logsigmoid(d)


def plain_norm(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def plain_scan(q, k, v, g, cu, first):
    q, k = q.repeat_interleave(H // HK, 1), k.repeat_interleave(H // HK, 1)
    out, last = [], []
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        S = first[n]
        for t in range(a, b):
            S = g[t].exp()[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            out.append(DK ** -0.5 * (q[t][:, :, None] * S).sum(1))
        last.append(S)
    return torch.stack(out), torch.stack(last)


def plain_head_norm(o, z, w):
    return plain_norm(o, w) * torch.sigmoid(z)


def worst(got, want):
    return float((got.double() - want).abs().max() / want.abs().max())


def train(dev):
    """The largest error of each gradient, relative to its largest value."""
    lens = [70, 1, 90]
    T, cu = sum(lens), [0, 70, 71, 161]
    w = weights(dev)
    rnd = lambda *s: torch.randn(s, device=dev)                               # noqa: E731
    x, first = rnd(T, WIDTH), rnd(len(lens), H, DK, DV)
    ds, dy, dlast = rnd(T, WIDTH), rnd(T, WIDTH), rnd(len(lens), H, DK, DV)
    on_dev = torch.tensor(cu, dtype=torch.int32, device=dev)

    a = K.block_norm(x, post_weight=w["first"], eps=EPS)
    p = (a @ w["w_in"]).requires_grad_()
    q, k, v, z, g = parts = split(p)                                          # (the split's own gradient is torch's)
    q, k, v, z, g = (t.detach() for t in parts)
    o, last = K.lin_prefill(q, k, v, g, first, on_dev)
    b = K.block_norm(o, gate=z, post_weight=w["head"], eps=EPS)
    c = b.flatten(1) @ w["w_out"]
    s, y = K.block_norm(c, residual=x, post_weight=w["post"], pre_weight=w["pre"], eps=EPS)

    n3 = K.block_norm_backward(c, ds, dy, s, post_weight=w["post"], pre_weight=w["pre"], eps=EPS)
    n2 = K.block_norm_backward(o, (n3["dx"] @ w["w_out"].T).unflatten(1, (H, DV)), gate=z, post_weight=w["head"], eps=EPS, residual=False)
    lin = K.lin_backward(q, k, v, g, n2["dx"], first, dlast, on_dev)
    dp, = torch.autograd.grad(parts, p, (lin["dq"], lin["dk"], lin["dv"], n2["dgate"], lin["dg"]))
    n1 = K.block_norm_backward(x, dp @ w["w_in"].T, post_weight=w["first"], eps=EPS, residual=False)
    got = {"x": n1["dx"] + n3["dresidual"], "states": lin["dS0"], "first": n1["dpost"], "w_in": a.T @ dp, "head": n2["dpost"],
           "w_out": b.flatten(1).T @ n3["dx"], "post": n3["dpost"], "pre": n3["dpre"]}

    W = {name: t.double().requires_grad_() for name, t in {**w, "x": x, "states": first}.items()}
    Q, Kk, V, Z, G = split(plain_norm(W["x"], W["first"]) @ W["w_in"])
    O, L = plain_scan(Q, Kk, V, G, cu, W["states"])
    Sm = W["x"] + plain_norm(plain_head_norm(O, Z, W["head"]).flatten(1) @ W["w_out"], W["post"])
    Y = plain_norm(Sm, W["pre"])
    want = dict(zip(W, torch.autograd.grad((Sm, Y, L), list(W.values()), (ds.double(), dy.double(), dlast.double()))))
    errors = {"train s": worst(s, Sm.detach()), "train y": worst(y, Y.detach()), "train state": worst(last, L.detach())}
    errors.update({"d " + name: worst(got[name], want[name]) for name in got})
    return errors


def serve(dev, dtype, steps):
    lens = [37, 150, 5]
    N, T = len(lens), sum(lens)
    w = weights(dev)
    w_in, w_out = w["w_in"].to(dtype), w["w_out"].to(dtype)
    pool = torch.zeros(N + 2, H, DK, DV, device=dev)                          # more slots than sequences; new ones start from zero
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=dev)
    cu = torch.tensor([0] + lens, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    workspace = K.lin_prefill_workspace(N, T, HK, H, DK, DV, dtype, dev)
    errors = {}

    def layer(x, scan):
        a = K.block_norm(x, post_weight=w["first"], eps=EPS)
        q, k, v, z, g = split(a @ w_in)
        g = g.float()
        o = scan(q, k, v, g)
        b = K.block_norm(o, gate=z, post_weight=w["head"], eps=EPS)
        c = b.flatten(1) @ w_out
        return (a, q, k, v, z, g, o, b, c) + K.block_norm(c, residual=x, post_weight=w["post"], pre_weight=w["pre"], eps=EPS)

    def check(name, x, got, cu, before):
        a, q, k, v, z, g, o, b, c, s, y = (t.double() for t in got)
        x = x.double()
        want_o, want_pool = plain_scan(q, k, v, g, cu, before[slots.long()].double())
        want_s = x + plain_norm(c, w["post"].double())
        for part, e in (("norm", worst(a, plain_norm(x, w["first"].double()))), ("attention", worst(o, want_o)),
                        ("head norm", worst(b, plain_head_norm(o, z, w["head"].double()))), ("sum", worst(s, want_s)),
                        ("next norm", worst(y, plain_norm(want_s, w["pre"].double()))), ("state", worst(pool[slots.long()], want_pool))):
            errors[f"{name} {part}"] = max(errors.get(f"{name} {part}", 0.0), e)

    x = torch.randn(T, WIDTH, device=dev).to(dtype)
    before = pool.clone()
    got = layer(x, lambda q, k, v, g: K.lin_prefill(q, k, v, g, pool, cu, state_idx=slots, workspace=workspace)[0])
    check("prompts", x, got, cu.tolist(), before)

    x = torch.randn(N, WIDTH, device=dev).to(dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, lambda q, k, v, g: K.lin_decode_step(q, k, v, g, pool, slots))
    for _ in range(steps):
        x.copy_(torch.randn_like(x))
        before = pool.clone()
        graph.replay()
        check("tokens", x, got, list(range(N + 1)), before)
    if K.k3kda_workspace_status(workspace) != 0:
        raise RuntimeError("a wait inside linear attention ran out")
    return errors


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    dev = "cuda:0"
    trained, served = train(dev), serve(dev, torch.bfloat16 if a.dtype == "bf16" else torch.float32, a.steps)
    for name, e in {**trained, **served}.items():
        print(f"{name:18s} largest error / largest value {e:.2e}")
    # A chain of eight operators in FP32, each with sums of at most 512 terms that are off by 2^-23 of a partial sum each, through
    # norms that keep relative errors: 8 * 512 * 2^-23 = 2^-11.  One operator in BF16: half a step of the value, 2^-8, and the same sums
    # of 512 terms, 2^-14, to which operands in two parts add 2^-16 of the absolute sums, here below 2^6 of the largest value.
    bf16 = a.dtype == "bf16"
    bad = [n for n, e in trained.items() if not e <= 2.0 ** -11]
    bad += [n for n, e in served.items() if not e <= (2.0 ** -8 + 2.0 ** -9 if bf16 and not n.endswith("state") else 2.0 ** -11)]
    if bad:
        raise SystemExit(f"too far off: {bad}")
    return {**trained, **served}


if __name__ == "__main__":
    main()
