"""The operators of linear-attention layers whose decay is one number a head, as cases to be timed.

``prefill``   chunked linear attention over packed sequences, with the state it starts from and the one it leaves
``decode``    one token of it for each sequence, the state updated in place in a pool of slots
``backward``  its gradients, those of the decays and of the first state among them
``norm``      what stands around such a block: the norm of its output, its gate, the residual with its factor and the next norm
``norm_grad`` the gradients of that

Linear attention, per sequence and head, S [dk, dv] from the first state (or zero) on, key heads shared by H / Hk value heads:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

g is one number a token and head, or one a head for all tokens.  The norms, for rows of D channels:

    u = x rsqrt(mean x^2 + eps) post          (u = x without post)
    s = residual + alpha u act(gate)          (no residual: 0; no gate: act = 1; act: sigmoid, or z sigmoid(z))
    y = s rsqrt(mean s^2 + eps) pre

Where ``own`` is false, ``run`` computes them with elementary torch operations; where it is true, through the package.
"""
import math
import random

import torch

own = False
EPS = 1e-6
CHUNK = 64

# ---- the cases -----------------------------------------------------------------------------------------------


def _lin(name, op, n, lo, hi, hk, h, dk, dv, dtype, decay="token", first=True, lens=1):
    """n sequences of lo to hi tokens."""
    return {"name": name, "op": op, "n": n, "lo": lo, "hi": hi, "hk": hk, "h": h, "dk": dk, "dv": dv, "dtype": dtype, "decay": decay,
            "first": first, "lens": lens}


def _norm(name, op, rows, d, dtype, post, gate, residual, pre):
    return {"name": name, "op": op, "rows": rows, "d": d, "dtype": dtype, "post": post, "gate": gate, "residual": residual, "pre": pre}


def listed():
    return [
        # one short question to a small layer: latency
        _lin("prefill short", "prefill", 1, 37, 37, 8, 8, 128, 128, "bf16", first=False),
        # a batch of prompts of many lengths, each continued from its state
        _lin("prefill prompts", "prefill", 16, 256, 3800, 32, 32, 128, 128, "bf16"),
        # one long document
        _lin("prefill long", "prefill", 1, 32768, 32768, 32, 32, 128, 128, "bf16", first=False),
        # shared key heads narrower than the values, fixed decays, in 32 bits
        _lin("prefill grouped f32", "prefill", 3, 301, 1500, 4, 8, 64, 96, "f32", decay="head"),
        # the next token of one conversation
        _lin("decode one", "decode", 1, 1, 1, 4, 16, 128, 128, "bf16"),
        # a decode batch over a pool of states
        _lin("decode batch", "decode", 256, 1, 1, 32, 32, 128, 128, "bf16"),
        # a training batch
        _lin("backward batch", "backward", 4, 2048, 2048, 32, 32, 128, 128, "bf16", first=False),
        # packed sequences with shared key heads, continued from states
        _lin("backward packed", "backward", 5, 77, 1900, 4, 16, 64, 128, "bf16"),
        # the norms between two blocks of a training batch
        _norm("norm train", "norm", 16384, 4096, "bf16", "post", "sigmoid", True, True),
        # a mixer's output, normed and gated head by head
        _norm("norm heads", "norm", 4096 * 32, 128, "bf16", "post", "silu", False, False),
        # their gradients, the weights' among them
        _norm("norm train grad", "norm_grad", 8192, 4096, "bf16", "post", "sigmoid", True, True),
        # rows of an odd width, in 32 bits
        _norm("norm grad f32", "norm_grad", 2777, 1111, "f32", "post", "silu", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    op = rng.choice(["prefill", "prefill", "decode", "backward", "backward", "norm", "norm_grad"])
    if op in ("norm", "norm_grad"):
        d = rng.choice([64, 128, _log(rng, 32, 8192), 8 * _log(rng, 8, 1000), 2048, 4096])
        rows = _log(rng, 1, max(2, (20 << 20) // d))
        post, gate = rng.choice(["none", "post", "post"]), rng.choice(["none", "sigmoid", "silu"])
        residual = rng.random() < 0.7
        c = _norm("", op, rows, d, dtype, post, gate, residual, rng.random() < 0.6 or (post == gate == "none" and not residual))
    else:
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 128), (64, 64), (128, 64), (48, 112), (32, 96), (16, 16)])
        hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        h = hk * rng.choice([1, 1, 2, 4])
        most = (100 << 20) // (h * 128)                          # tokens
        if op == "backward":
            most //= 4
        if dtype == "f32":
            most //= 6
        if op == "decode":
            n, lo, hi = _log(rng, 1, max(2, min(512, 8192 // h))), 1, 1
        else:
            hi = _log(rng, 1, min(most, 30000))
            n = max(1, min(_log(rng, 1, 64), most // hi))
            lo = max(1, hi // rng.choice([1, 2, 10]))
        c = _lin("", op, n, lo, hi, hk, h, dk, dv, dtype, rng.choice(["token", "token", "head"]), rng.random() < 0.5, rng.randrange(1 << 20))
    del c["name"]
    return c


def _lengths(case):
    r = random.Random(case["lens"] * 7919 + case["n"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if "rows" in case:
        n = case["rows"] * case["d"]
        post, gate, res, pre = case["post"] == "post", case["gate"] != "none", case["residual"], case["pre"]
        if case["op"] == "norm":
            arrays = 1 + gate + res + 1 + pre                     # x, gate, residual; s, y
        else:
            arrays = (post or gate) + gate + pre + 1 + pre + 1 + gate + res     # x, gate, s, ds, dy; dx, dgate, dresidual
        return {"bytes": n * arrays * size + 8 * case["d"], "flops": 6 * n}
    T, N, hk, h, dk, dv = sum(_lengths(case)), case["n"], case["hk"], case["h"], case["dk"], case["dv"]
    state, decays = N * h * dk * dv * 4, (h if case["decay"] == "head" else T * h) * 4
    if case["op"] == "decode":
        return {"bytes": 2 * state + decays + T * (2 * hk * dk + 2 * h * dv) * size, "flops": 4 * N * h * dk * dv}
    if case["op"] == "prefill":
        return {"bytes": T * (2 * hk * dk + 2 * h * dv) * size + decays + state * (2 if case["first"] else 1), "flops": 4 * T * h * dk * dv}
    return {"bytes": T * (4 * hk * dk + 3 * h * dv) * size + 2 * decays + state * (3 if case["first"] else 1), "flops": 10 * T * h * dk * dv}


# ---- inputs --------------------------------------------------------------------------------------------------


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed * 1000003 + 29)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    if own:
        import hybrid_linear_attention_rule_gb300 as K
        s["K"] = K
    if "rows" in case:
        R, D = case["rows"], case["d"]
        s["x"] = normal(R, D)
        s["gate"] = normal(R, D) if case["gate"] != "none" else None
        s["post"] = 1 + normal(D, std=0.2, dtype=torch.float32) if case["post"] == "post" else None
        s["pre"] = 1 + normal(D, std=0.2, dtype=torch.float32) if case["pre"] else None
        s["alpha"] = 0.5 if case["residual"] else 1.0
        if case["op"] == "norm":
            s["residual"] = normal(R, D) if case["residual"] else None
        else:
            s["sum"] = normal(R, D, std=1.1) if case["pre"] else None        # what the forward pass left
            s["ds"] = normal(R, D, std=0.1)
            s["dy"] = normal(R, D, std=0.1) if case["pre"] else None
            if own:
                s["workspace"] = K.block_norm_workspace(R, D, device=dev)
        return s
    lens, N, hk, h, dk, dv = _lengths(case), case["n"], case["hk"], case["h"], case["dk"], case["dv"]
    T = sum(lens)
    s["q"], s["k"], s["v"] = normal(T, hk, dk), normal(T, hk, dk, std=dk ** -0.25), normal(T, h, dv)
    # memories of about 1 to 500 tokens, a head each
    slope = torch.exp2(-8.0 * (torch.arange(h, device=dev) + 0.5) / h)
    s["g"] = -slope if case["decay"] == "head" else -slope * torch.nn.functional.softplus(normal(T, h, dtype=torch.float32) + 0.5)
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    s["cu"] = cu.to(dev) if N > 1 else None
    s["starts"] = cu.to(dev).long()
    s["longest"] = max(lens)
    if case["op"] == "decode":
        slots = N + 3
        s["state"] = normal(slots, h, dk, dv, std=0.5, dtype=torch.float32)
        s["idx"] = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
        return s
    s["first"] = normal(N, h, dk, dv, std=0.5, dtype=torch.float32) if case["first"] else None
    if case["op"] == "backward":
        s["do"] = normal(T, h, dv)
        s["dlast"] = normal(N, h, dk, dv, std=0.5, dtype=torch.float32) if case["first"] else None
    if own:
        s["workspace"] = (K.lin_backward_workspace if case["op"] == "backward" else K.lin_prefill_workspace)(N, T, hk, h, dk, dv, dt, device=dev)
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------


def _padded(s, x, group=1):
    """x [T, heads, ...] in 32 bits as [N, heads * group, chunks, CHUNK, ...], zeros behind each sequence."""
    case, at = s["case"], s["starts"]
    nc = -(-s["longest"] // CHUNK)
    t = at[:-1, None] + torch.arange(nc * CHUNK, device=at.device)
    inside = t < at[1:, None]
    y = x.float()[torch.where(inside, t, 0)]
    y = torch.where(inside.view(inside.shape + (1,) * (x.dim() - 1)), y, 0.0)
    y = y.transpose(1, 2).unflatten(2, (nc, CHUNK))
    return y.repeat_interleave(group, 1) if group > 1 else y


def _packed(s, y):
    """The inverse: [N, heads, chunks, CHUNK, ...] -> [T, heads, ...]."""
    at = s["starts"]
    t = torch.arange(int(s["q"].shape[0]), device=at.device)
    n = torch.searchsorted(at, t, right=True) - 1
    return y.flatten(2, 3)[n, :, t - at[n]]


def _decays(s):
    """Sums of g in 64 bits: within each chunk [N, H, nc, C], and up to each chunk's end [N, H, nc]."""
    case, T = s["case"], s["q"].shape[0]
    g = s["g"].expand(T, case["h"]) if s["g"].dim() == 1 else s["g"]
    G = _padded(s, g).double().cumsum(-1)
    return G, G[..., -1].cumsum(-1)


def _between(E):
    """exp of the decay from behind chunk c' to before chunk c, [N, H, nc + 1, nc] for c' < c, and from the start to before each c."""
    before = torch.cat([torch.zeros_like(E[..., :1]), E], -1)
    c = torch.arange(before.shape[-1], device=E.device)
    W = torch.where(c[:, None] > c[None, :-1], before[..., :, None] - E[..., None, :], -math.inf).exp().float()
    return W, before.exp().float()


def _states(G, E, k, v, first):
    """The state before each chunk, and behind the last: [N, H, nc + 1, dk, dv]."""
    local = (k * (G[..., -1:] - G).exp().float()[..., None]).transpose(-1, -2) @ v
    W, begin = _between(E)
    S = (W @ local.flatten(-2)).unflatten(-1, local.shape[-2:])
    return S if first is None else S + begin[..., None, None] * first[:, :, None]


def _inside(G):
    """exp(G_i - G_j) for j <= i, else 0."""
    c = torch.arange(CHUNK, device=G.device)
    return torch.where(c[:, None] >= c, G[..., :, None] - G[..., None, :], -math.inf).exp().float()


def _prefill(s):
    case = s["case"]
    group = case["h"] // case["hk"]
    q, k, v = _padded(s, s["q"], group), _padded(s, s["k"], group), _padded(s, s["v"])
    G, E = _decays(s)
    S = _states(G, E, k, v, s["first"])
    o = (q @ k.transpose(-1, -2) * _inside(G)) @ v + G.exp().float()[..., None] * (q @ S[:, :, :-1])
    return _packed(s, o * case["dk"] ** -0.5).to(s["q"].dtype), S[:, :, -1].contiguous()


def _backward(s):
    case = s["case"]
    group, scale = case["h"] // case["hk"], case["dk"] ** -0.5
    q, k, v, do = _padded(s, s["q"], group), _padded(s, s["k"], group), _padded(s, s["v"]), _padded(s, s["do"])
    G, E = _decays(s)
    D = _inside(G)
    S = _states(G, E, k, v, s["first"])
    up, down = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    # what reaches each chunk's end from behind it: R [N, H, nc + 1, dk, dv], the first entry for the first state
    local = (q * up * scale).transpose(-1, -2) @ do
    before = torch.cat([torch.zeros_like(E[..., :1]), E], -1)          # decay up to before chunk c, and up to the end
    c = torch.arange(before.shape[-1], device=E.device)
    U = torch.where(c[:, None] <= c[None, :-1], before[..., None, :-1] - before[..., :, None], -math.inf).exp().float()
    R = (U @ local.flatten(-2)).unflatten(-1, local.shape[-2:])
    if s["dlast"] is not None:
        R = R + (E[..., -1:] - before).exp().float()[..., None, None] * s["dlast"][:, :, None]
    Sc, Rc = S[:, :, :-1], R[:, :, 1:]
    A, B = D * (q @ k.transpose(-1, -2)), D * (do @ v.transpose(-1, -2))
    dq_far, dk_far = scale * up * (do @ Sc.transpose(-1, -2)), down * (v @ Rc.transpose(-1, -2))
    dq = scale * (B @ k) + dq_far
    dk = scale * (B.transpose(-1, -2) @ q) + dk_far
    dv = scale * (A.transpose(-1, -2) @ do) + down * (k @ Rc)
    # g_t decays what tokens before t give to t and those behind it: pairs within the chunk, and over its borders
    pairs = (scale * A * (do @ v.transpose(-1, -2))).tril(-1)
    x = (pairs.sum(-1) + (q * dq_far).sum(-1)).double() - (pairs.sum(-2) + (k * dk_far).sum(-1)).double()
    over = (S[:, :, 1:] * Rc).sum((-1, -2)).double()[..., None]
    dg = x.flip(-1).cumsum(-1).flip(-1) + over
    dg = _packed(s, dg)
    dg = dg.sum(0) if s["g"].dim() == 1 else dg
    dt = s["q"].dtype
    dq, dk = (y.unflatten(1, (-1, group)).sum(2) if group > 1 else y for y in (dq, dk))
    out = {"dq": _packed(s, dq).to(dt), "dk": _packed(s, dk).to(dt), "dv": _packed(s, dv).to(dt), "dg": dg.float()}
    if s["first"] is not None:
        out["dfirst"] = R[:, :, 0].contiguous()
    return out


def _decode(s):
    case = s["case"]
    group, at = case["h"] // case["hk"], s["idx"].long()
    q, k = (x.float().repeat_interleave(group, 1) for x in (s["q"], s["k"]))
    a = s["g"].exp().expand(case["n"], case["h"])[..., None, None]
    S = a * s["state"][at] + k[..., :, None] * s["v"].float()[..., None, :]
    s["state"][at] = S
    o = (q[..., None, :] @ S).squeeze(-2) * case["dk"] ** -0.5
    return o.to(s["q"].dtype), s["state"]


def _act(kind, z):
    """act(z) and its derivative."""
    sig = 1 / (1 + (-z).exp())
    return (sig, sig * (1 - sig)) if kind == "sigmoid" else (z * sig, sig * (1 + z * (1 - sig)))


def _normed(x, w):
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w


def _norm_forward(s):
    case, dt = s["case"], s["x"].dtype
    z = s["x"].float()
    if s["post"] is not None:
        z = _normed(z, s["post"])
    if s["gate"] is not None:
        z = z * _act(case["gate"], s["gate"].float())[0]
    z = s["alpha"] * z
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return (z.to(dt), _normed(z, s["pre"]).to(dt)) if s["pre"] is not None else z.to(dt)


def _norm_back(dy, x, w):
    """Gradients of _normed's x and w, in 32 bits; sums over rows in 64."""
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    h = x * r
    d = dy * w
    return r * (d - h * (d * h).mean(-1, keepdim=True)), (dy * h).sum(0, dtype=torch.float64).float()


def _norm_gradient(s):
    case, dt, out = s["case"], s["x"].dtype, {}
    d = s["ds"].float()
    if s["pre"] is not None:
        more, out["dpre"] = _norm_back(s["dy"].float(), s["sum"].float(), s["pre"])
        d = d + more
    if case["residual"]:
        out["dresidual"] = d.to(dt)
    d = s["alpha"] * d
    x = s["x"].float()
    if s["gate"] is not None:
        a, da = _act(case["gate"], s["gate"].float())
        u = x if s["post"] is None else _normed(x, s["post"])
        out["dgate"] = (d * u * da).to(dt)
        d = d * a
    if s["post"] is not None:
        d, out["dpost"] = _norm_back(d, x, s["post"])
    out["dx"] = d.to(dt)
    return out


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        K = s["K"]
        if op == "prefill":
            return K.lin_prefill(s["q"], s["k"], s["v"], s["g"], initial_state=s["first"], cu_seqlens=s["cu"], workspace=s["workspace"])
        if op == "decode":
            return K.lin_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], state_idx=s["idx"]), s["state"]
        if op == "backward":
            d = K.lin_backward(s["q"], s["k"], s["v"], s["g"], s["do"], initial_state=s["first"], dS_final=s["dlast"], cu_seqlens=s["cu"],
                               workspace=s["workspace"])
            out = {"dq": d["dq"], "dk": d["dk"], "dv": d["dv"], "dg": d["dg"]}
            if s["first"] is not None:
                out["dfirst"] = d["dS0"]
            return out
        act = case["gate"] if case["gate"] != "none" else "sigmoid"
        if op == "norm":
            return K.block_norm(s["x"], residual=s["residual"], gate=s["gate"], gate_act=act, post_weight=s["post"], pre_weight=s["pre"],
                                alpha=s["alpha"], eps=EPS)
        d = K.block_norm_backward(s["x"], s["ds"], dy=s["dy"], sum=s["sum"], gate=s["gate"], gate_act=act, post_weight=s["post"],
                                  pre_weight=s["pre"], alpha=s["alpha"], eps=EPS, residual=case["residual"], workspace=s["workspace"])
        return {k: v for k, v in d.items() if v is not None}
    return {"prefill": _prefill, "decode": _decode, "backward": _backward, "norm": _norm_forward, "norm_grad": _norm_gradient}[op](s)


# ---- the definition in 64 bits, token by token ------------------------------------------------------------------


def _rows(x, starts, longest, group=1):
    """x [T, heads, ...] in 64 bits as a list over positions of [N, heads * group, ...], zeros behind each sequence."""
    N = starts.numel() - 1
    y = torch.zeros((longest, N) + x.shape[1:], dtype=torch.float64, device=x.device)
    for n in range(N):
        a, b = int(starts[n]), int(starts[n + 1])
        y[:b - a, n] = x[a:b].double()
    return torch.repeat_interleave(y, group, dim=2)


def _unrows(y, starts):
    return torch.cat([y[:int(starts[n + 1] - starts[n]), n] for n in range(starts.numel() - 1)])


def exact(case, seed):
    s = prepare(case, seed)
    if "rows" in case:
        return _exact_norm(s)
    starts, L, group, scale = s["starts"], s["longest"], case["h"] // case["hk"], 1.0 / math.sqrt(case["dk"])
    T = s["q"].shape[0]
    g = s["g"].double()
    fixed = g.dim() == 1
    if fixed:
        g = g.unsqueeze(0).repeat(T, 1)
    q, k, v = _rows(s["q"], starts, L, group), _rows(s["k"], starts, L, group), _rows(s["v"], starts, L)
    alpha = torch.exp(_rows(g, starts, L)).unsqueeze(-1).unsqueeze(-1)
    N, H, dk, dv = case["n"], case["h"], case["dk"], case["dv"]
    S = torch.zeros((N, H, dk, dv), dtype=torch.float64, device=q.device)
    if case["op"] == "decode":
        S = s["state"].double()[s["idx"].long()]
    elif s["first"] is not None:
        S = s["first"].double()
    do = _rows(s["do"], starts, L) if case["op"] == "backward" else None
    rows = torch.empty((L, N, H, dk if do is not None else dv), dtype=torch.float64, device=q.device)
    for t in range(L):
        S = torch.addcmul(alpha[t] * S, k[t].unsqueeze(-1), v[t].unsqueeze(-2))
        rows[t] = (torch.matmul(S, do[t].unsqueeze(-1)).squeeze(-1) if do is not None else torch.matmul(q[t].unsqueeze(-2), S).squeeze(-2))
    rows *= scale
    if case["op"] == "decode":
        pool = s["state"].double()
        pool[s["idx"].long()] = S
        return _unrows(rows, starts), pool
    if case["op"] == "prefill":
        return _unrows(rows, starts), S
    R = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    over = (S * R).sum((-1, -2))
    dk_, dv_ = torch.empty((L, N, H, dk), dtype=torch.float64, device=q.device), torch.empty((L, N, H, dv), dtype=torch.float64, device=q.device)
    for t in reversed(range(L)):
        R = torch.addcmul(R, scale * q[t].unsqueeze(-1), do[t].unsqueeze(-2))
        dk_[t] = torch.matmul(R, v[t].unsqueeze(-1)).squeeze(-1)
        dv_[t] = torch.matmul(k[t].unsqueeze(-2), R).squeeze(-2)
        R = alpha[t] * R
    # every decay of a sequence scales what is behind it: d/dg_t = sum over u >= t of (q . dq - k . dk)_u, and the last state's share
    x = (q * rows).sum(-1) - (k * dk_).sum(-1)
    dg = _unrows(torch.flip(torch.cumsum(torch.flip(x, [0]), 0), [0]) + over, starts)
    shared = lambda y: _unrows(y, starts).reshape(T, case["hk"], group, dk).sum(2)  # noqa: E731
    out = {"dq": shared(rows), "dk": shared(dk_), "dv": _unrows(dv_, starts), "dg": dg.sum(0) if fixed else dg}
    if s["first"] is not None:
        out["dfirst"] = R
    return out


def _exact_norm(s):
    case = s["case"]

    def unit(x):
        return x / torch.sqrt(torch.mean(x * x, dim=1, keepdim=True) + EPS)

    def act(z):
        return torch.sigmoid(z) if case["gate"] == "sigmoid" else z * torch.sigmoid(z)

    def block(x, gate, post):
        u = x if post is None else unit(x) * post
        return u if gate is None else u * act(gate)

    wide = {name: None if s.get(name) is None else s[name].double() for name in ("x", "gate", "post", "pre", "residual", "sum", "ds", "dy")}
    if case["op"] == "norm":
        z = s["alpha"] * block(wide["x"], wide["gate"], wide["post"])
        if wide["residual"] is not None:
            z = z + wide["residual"]
        return z if wide["pre"] is None else (z, unit(z) * wide["pre"])
    # the gradients by automatic differentiation
    leaf = {name: wide[name].requires_grad_() for name in ("x", "gate", "post", "pre", "sum") if wide[name] is not None}
    out, ds = {}, wide["ds"]
    if "pre" in leaf:
        got = torch.autograd.grad(unit(leaf["sum"]) * leaf["pre"], (leaf["sum"], leaf["pre"]), wide["dy"])
        ds, out["dpre"] = ds + got[0], got[1]
    if case["residual"]:
        out["dresidual"] = ds
    names = [name for name in ("x", "gate", "post") if name in leaf]
    got = torch.autograd.grad(s["alpha"] * block(leaf["x"], leaf.get("gate"), leaf.get("post")), [leaf[name] for name in names], ds)
    for name, d in zip(names, got):
        out["d" + name] = d
    return out
