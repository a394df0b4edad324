"""The attention layers' operators together, as a training step and a small serving loop would use them.

    python examples/attention_layer.py [--fmt i4|bf16] [--steps 32]

A layer of 4 key heads shared by 16 query heads, 128 channels, the last 64 of them turned by position.  The training part
turns queries and keys of packed sequences (the keys' turned part is one head that all heads share) and takes the gradient
back through the rotation.  The serving part appends prompts to a paged cache in 4 bits (or bf16), attends over
them, then decodes token by token: one CUDA graph holds a step's append, attention and length increment and is
replayed.  Every result is compared with plain torch on the values that the cache stands for.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_linear_attention_rule_gb300 as K  # noqa: E402

H, G, D, TURNED, PAGE = 4, 4, 128, 64, 64


def plain_rope(x, pos, sign=1.0):
    """x [T, heads, D] with its last TURNED channels turned in pairs (c, c + TURNED/2), in float64."""
    f = 10000.0 ** (-torch.arange(0, TURNED, 2, device=x.device, dtype=torch.float64) / TURNED)
    a = pos.double()[:, None, None] * f
    u, v = x.double()[..., D - TURNED:].chunk(2, -1)
    turned = torch.cat([u * a.cos() - sign * v * a.sin(), v * a.cos() + sign * u * a.sin()], -1)
    return torch.cat([x.double()[..., :D - TURNED], turned], -1)


def plain_attention(q, k, v, seen, gate):
    """q, gate [c, H*G, D], k, v [L, H, D] -> [c, H*G, D] in float64; token i sees the first seen[i] keys."""
    s = torch.einsum("chgd,lhd->hcgl", q.unflatten(1, (H, G)), k) * D ** -0.5
    hidden = torch.arange(k.shape[0], device=k.device)[None] >= seen[:, None]
    p = torch.softmax(s.masked_fill(hidden[None, :, None], -float("inf")), -1)
    return torch.einsum("hcgl,lhd->chgd", p, v).flatten(1, 2) * torch.sigmoid(gate.double())


def worst(got, want):
    return float((got.double() - want).abs().max() / want.abs().max())


def train(table, dev):
    T = 200
    pos = torch.cat([torch.arange(120), torch.arange(80)]).to(torch.int32).to(dev)
    fused = torch.randn(T, (H * G + 1) * D, device=dev).bfloat16()          # a projection's output: queries, then one key head
    q, k = fused[:, :H * G * D].unflatten(1, (H * G, D)), fused[:, H * G * D:].unflatten(1, (1, D)).expand(T, H, D)
    qr, kr = K.rope(q, pos, table, k)
    dq, dk = torch.randn_like(qr), torch.randn_like(kr)
    gq, gk = K.rope_backward(dq, pos, table, dk_out=dk, k_shared=True)
    return {"rope q": worst(qr, plain_rope(q, pos)), "rope k": worst(kr, plain_rope(k, pos)),
            "rope dq": worst(gq, plain_rope(dq, pos, -1.0)), "rope dk": worst(gk, plain_rope(dk, pos, -1.0).sum(1, keepdim=True))}


def serve(table, dev, fmt, steps):
    prompts = [37, 150, 5]
    N, T, longest = len(prompts), sum(prompts), max(prompts) + steps
    pages = -(-longest // PAGE)
    cache = K.PagedCache(K.paged_pool(N * pages, PAGE, H, D, D, fmt, dev),
                         torch.randperm(N * pages, device=dev).to(torch.int32).view(N, pages),
                         torch.tensor(prompts, dtype=torch.int32, device=dev), PAGE, D, D, fmt)
    workspace = K.paged_attend_workspace(cache, H * G)
    cu = torch.tensor([0] + prompts, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    rnd = lambda *s: torch.randn(s, device=dev).bfloat16()                   # noqa: E731

    def expect(q, gate, starts):
        lens = cache.kv_len.tolist()
        all_cu = torch.tensor([0] + lens, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        k, v = K.paged_read(cache, sum(lens), all_cu, torch.float32)
        out, at, row = [], 0, 0
        for n, L in enumerate(lens):
            c = L - starts[n]
            pos = torch.arange(starts[n], L, device=dev)
            out.append(plain_attention(plain_rope(q[row:row + c], pos), k[at:at + L].double(), v[at:at + L].double(), pos + 1, gate[row:row + c]))
            at, row = at + L, row + c
        return torch.cat(out)

    # the prompts: append, then attend to what was appended
    q, k, v, gate = rnd(T, H * G, D), rnd(T, H, D), rnd(T, H, D), rnd(T, H * G, D)
    K.paged_append(cache, k, v, cu, rope=table)
    got = K.paged_attend(cache, q, cu, max(prompts), rope=table, gate=gate, workspace=workspace)
    errors = {"prompts": worst(got, expect(q, gate, [0] * N))}

    # the tokens: one graph a step
    q, k, v, gate, out = rnd(N, H * G, D), rnd(N, H, D), rnd(N, H, D), rnd(N, H * G, D), rnd(N, H * G, D)

    def step():
        cache.kv_len.add_(1)
        K.paged_append(cache, k, v, rope=table)
        K.paged_attend(cache, q, rope=table, gate=gate, out=out, workspace=workspace)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    errors["tokens"] = 0.0
    for _ in range(steps):
        for t in (q, k, v, gate):
            t.copy_(torch.randn_like(t))
        graph.replay()
        errors["tokens"] = max(errors["tokens"], worst(out, expect(q, gate, [n - 1 for n in cache.kv_len.tolist()])))
    if K.k3kda_workspace_status(workspace) != 0:
        raise RuntimeError("a wait inside the attention ran out")
    return errors


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=("i4", "bf16"), default="i4")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    dev = "cuda:0"
    table = K.rope_table(TURNED, offset=D - TURNED, device=dev)
    errors = {**train(table, dev), **serve(table, dev, a.fmt, a.steps)}
    for name, e in errors.items():
        print(f"{name:8s} largest error / largest value {e:.2e}")
    # bf16 outputs: half a step of the value (2^-8 of it)
    bad = [n for n, e in errors.items() if not e <= 2.0 ** -8]
    if bad:
        raise SystemExit(f"too far off: {bad}")
    return errors


if __name__ == "__main__":
    main()
