"""The attention layers' serving and training operators, as cases to be timed.

Three operators of the hybrid's gated attention layers: the rotary position rotation with its gradient
(``rope``, ``rope_grad``), the append of new key and value rows to a paged cache with the rotation applied on
the way (``append``; the pass reads the rows back as the values the cache stands for), and the attention of
new tokens over that cache (``attend``).  Where ``own`` is false, ``run`` computes them with elementary torch
operations; where it is true, through the package.

The paged cache.  A pool is uint8 [pages, heads, block bytes]; a (page, head) block holds page/16 strips of 16
tokens, and a strip one plane for every 64 channels of the key, then one for every 64 channels of the value.

  "i4"    plane = 576 bytes: 16 rows of 32 bytes (channel c in the low half of byte c/2 when c is even, else in
          the high half), then 16 pairs (scale, minimum) in fp16.  A group of 64 channels x of one token is held as
          m = fp16(min x), s = fp16(max(max x - m, 0) / 15) (both kept within +-65504), codes
          min(max(rint((x - m) / s), 0), 15) (0 where s = 0), and stands for s * code + m.  A group with an
          infinity or a NaN has s = m = NaN.
  "bf16"  plane = 2048 bytes: 16 rows of 64 bf16 values; the 16-byte piece c of row r is at piece c ^ (r & 7).
"""
import math
import random

import torch

own = False

# ---- the cases -----------------------------------------------------------------------------------------------


def _rope_case(name, op, tokens, hq, hk, d, dim, off, layout, scaling, dtype, shared, seqlen):
    return {"name": name, "op": op, "tokens": tokens, "hq": hq, "hk": hk, "d": d, "dim": dim, "off": off, "layout": layout,
            "scaling": scaling, "dtype": dtype, "shared": shared, "seqlen": seqlen}


def _paged_case(name, op, n, heads, group, dqk, dv, page, fmt, past, new, dim, off, layout, dtype, gate, lens=1):
    return {"name": name, "op": op, "n": n, "heads": heads, "group": group, "dqk": dqk, "dv": dv, "page": page, "fmt": fmt,
            "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1], "dim": dim, "off": off,
            "layout": layout, "scaling": "none", "dtype": dtype, "gate": gate, "lens": lens}


def listed():
    return [
        # the queries and keys of one decode batch, whole heads turned
        _rope_case("rope decode", "rope", 64, 32, 8, 128, 128, 0, "half", "none", "bf16", False, 131072),
        # a training batch of packed sequences; 64 of 192 channels turned, in pairs, stretched to a longer context
        _rope_case("rope train", "rope", 16384, 32, 32, 192, 64, 128, "interleaved", "by_parts", "bf16", False, 16384),
        # its backward with whole heads turned, one key head shared by all query heads
        _rope_case("rope train grad", "rope_grad", 16384, 32, 32, 128, 128, 0, "half", "linear", "bf16", True, 8192),
        # gradients in 32 bits, as accumulated over an odd number of tokens
        _rope_case("rope grad f32", "rope_grad", 3001, 16, 4, 128, 64, 0, "half", "ntk", "f32", False, 3001),
        # one token for each sequence of a decode batch
        _paged_case("append decode i4", "append", 256, 32, 1, 128, 128, 64, "i4", (0, 4095), (1, 1), 64, 64, "half", "bf16", False),
        # prompts of many lengths, a few of them continued
        _paged_case("append prompts i4", "append", 16, 32, 1, 128, 128, 64, "i4", (0, 700), (256, 3800), 128, 0, "half", "bf16", False),
        # prompts in 32 bits, keys wider than values, small pages held in bf16
        _paged_case("append prompts bf16", "append", 7, 8, 1, 192, 128, 16, "bf16", (0, 300), (37, 2500), 64, 128, "interleaved", "f32", False),
        # the smallest call: one sequence's next token
        _paged_case("attend one i4", "attend", 1, 8, 4, 128, 128, 64, "i4", (511, 511), (1, 1), 128, 0, "half", "bf16", False),
        # a decode batch of a layer whose heads each have their own keys, with the output gate
        _paged_case("attend batch i4", "attend", 64, 32, 1, 128, 128, 64, "i4", (0, 8191), (1, 1), 0, 0, "half", "bf16", True),
        # one very long context, query heads sharing keys
        _paged_case("attend long i4", "attend", 1, 8, 4, 128, 128, 32, "i4", (250007, 250007), (1, 1), 128, 0, "half", "bf16", False),
        # prompts cut into chunks, each attending to what is cached and to itself
        _paged_case("attend chunks i4", "attend", 4, 8, 4, 128, 128, 64, "i4", (2000, 6000), (65, 160), 64, 0, "half", "bf16", False),
        # a few tokens checked at once for each sequence, keys wider than values, pages in bf16
        _paged_case("attend few bf16", "attend", 48, 4, 8, 192, 128, 16, "bf16", (100, 4000), (1, 5), 64, 128, "interleaved", "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    layout = rng.choice(["half", "interleaved"])
    op = rng.choice(["rope", "rope_grad", "append", "append", "attend", "attend", "attend"])
    if op in ("rope", "rope_grad"):
        d = rng.choice([64, 128, 192, 256])
        dim = rng.choice([d, d // 2, 64, 32, 48])
        hq = rng.choice([1, 4, 8, 16, 32, 40])
        shared = op == "rope_grad" and rng.random() < 0.5
        hk = hq if shared else max(1, hq // rng.choice([1, 2, 4, 8]))
        top = (180 << 20) // ((hq + hk) * d * (4 if dtype == "f32" else 2))
        tokens = _log(rng, 1, max(2, top))
        c = _rope_case("", op, tokens, hq, hk, d, dim, rng.choice([0, d - dim]), layout,
                       rng.choice(["none", "linear", "ntk", "by_parts"]), dtype, shared, _log(rng, 16, 200000))
        del c["name"]
        return c
    dqk, dv = rng.choice([(128, 128), (128, 128), (192, 128), (64, 64), (256, 256), (256, 128), (64, 128)])
    fmt = rng.choice(["i4", "i4", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([0, 32, 64, dqk])
    off = rng.choice([0, dqk - dim])
    heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
    if op == "append":
        new = _log(rng, 1, 3000)
        n = max(1, min(256, _log(rng, 1, 256), 24000 * 32 // (new * heads)))
        c = _paged_case("", op, n, heads, 1, dqk, dv, page, fmt, (0, _log(rng, 1, 2000)), (max(1, new // 3), new), dim, off, layout, dtype, False,
                        rng.randrange(1 << 20))
    else:
        group = rng.choice([1, 1, 2, 4, 5, 8, 16])
        new = rng.choice([1, 1, 1, 2, 4, 7, _log(rng, 8, 200)])
        past = _log(rng, 1, 100000)
        most = 30000000 if fmt == "i4" else 8000000                  # cached (token, head) rows of 128 + 128 channels
        n = max(1, min(128, _log(rng, 1, 128), most * 256 // (past * heads * (dqk + dv)), 40000000 // (past * heads * group * new)))
        past = max(1, min(past, 40000000 // (heads * group * new)))
        c = _paged_case("", op, n, heads, group, dqk, dv, page, fmt, (past // rng.choice([1, 2, 30]), past), (max(1, new // 2), new), dim, off, layout,
                        "bf16", rng.random() < 0.5, rng.randrange(1 << 20))
    del c["name"]
    return c


def _lengths(case):
    """(tokens already cached, new tokens) of each sequence."""
    r = random.Random(case["lens"] * 7919 + case["n"])
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["n"])]
    return past, [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]


#: Bytes of one token and head in the cache.
def _row_bytes(case):
    return (case["dqk"] + case["dv"]) // 64 * (36 if case["fmt"] == "i4" else 128)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("rope", "rope_grad"):
        wide, narrow = case["hq"] + case["hk"], case["hq"] + (1 if case["shared"] else case["hk"])
        rows = case["tokens"] * (wide + narrow)
        return {"bytes": rows * case["d"] * size + case["tokens"] * 4, "flops": 3 * case["tokens"] * wide * case["dim"]}
    past, new = _lengths(case)
    d, H, T = case["dqk"] + case["dv"], case["heads"], sum(new)
    if case["op"] == "append":
        return {"bytes": T * H * (d * size + _row_bytes(case) + d * 2), "flops": T * H * (6 * d + 3 * case["dim"])}
    rows = sum((a * b + b * (b + 1) // 2) for a, b in zip(past, new)) * H * case["group"]
    kept = sum(a + b for a, b in zip(past, new)) * H * _row_bytes(case)
    return {"bytes": kept + T * H * case["group"] * (d + (case["dv"] if case["gate"] else 0)) * size, "flops": 2 * rows * d}


# ---- inputs --------------------------------------------------------------------------------------------------

SCALING = {  # factor, original length, beta_fast, beta_slow
    "none": (1.0, 0, 32.0, 1.0), "linear": (4.0, 8192, 32.0, 1.0), "ntk": (8.0, 8192, 32.0, 1.0), "by_parts": (16.0, 4096, 32.0, 1.0)}
THETA = 10000.0


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed * 1000003 + 17)
    dt = _type(case["dtype"])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = {"case": case, "table": None}
    factor, length, fast, slow = SCALING[case["scaling"]]
    if own:
        import hybrid_linear_attention_rule_gb300 as K
        s["K"] = K
        if case["dim"]:
            s["table"] = K.rope_table(case["dim"], THETA, offset=case["off"], layout=case["layout"], scaling=case["scaling"],
                                      factor=factor, original_length=length, beta_fast=fast, beta_slow=slow, device=dev)
    if case["dim"]:
        s["freq"], s["mscale"] = _frequencies(case["dim"], case["scaling"])
        s["freq"] = s["freq"].to(dev)
    if case["op"] in ("rope", "rope_grad"):
        T, d = case["tokens"], case["d"]
        start = torch.randint(0, case["seqlen"], (1,), generator=gen, device=dev)
        # tokens of packed sequences one after the other, or of a decode batch anywhere
        s["pos"] = ((torch.arange(T, device=dev) + start) % case["seqlen"] if T > 256 else
                    torch.randint(0, case["seqlen"], (T,), generator=gen, device=dev)).to(torch.int32)
        s["q"], s["k"] = normal(T, case["hq"], d), normal(T, case["hk"], d)
        return s
    past, new = _lengths(case)
    N, H, P, T = case["n"], case["heads"], case["page"], sum(new)
    total = [a + b for a, b in zip(past, new)]
    widest = max(-(-t // P) for t in total)
    pages = sum(-(-t // P) for t in total)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((N, widest), dtype=torch.int32)
    at = 0
    rows = []
    for n, t in enumerate(total):
        rows.append((n, at, -(-t // P)))
        at += -(-t // P)
    order = order.cpu()
    for n, a, c in rows:
        table[n, :c] = order[a:a + c]
    s["table_of_pages"] = table.to(dev)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new, dtype=torch.int32).cumsum(0)
    s["cu"] = cu.to(dev)
    s["max_new"] = max(new)
    s["single"] = case["new_hi"] == 1
    strips, planes = P // 16, (case["dqk"] + case["dv"]) // 64
    if case["op"] == "append":
        s["pool"] = torch.zeros((pages, H, strips * planes * (576 if case["fmt"] == "i4" else 2048)), dtype=torch.uint8, device=dev)
        s["k"], s["v"] = normal(T, H, case["dqk"]), normal(T, H, case["dv"])
    else:
        s["pool"] = _filled_pool(case, pages, gen)
        s["q"] = normal(T, H * case["group"], case["dqk"])
        s["gate"] = normal(T, H * case["group"], case["dv"]) if case["gate"] else None
    if own:
        s["cache"] = K.PagedCache(s["pool"], s["table_of_pages"], s["kv_len"], page_size=P, dqk=case["dqk"], dv=case["dv"], fmt=case["fmt"])
        if case["op"] == "attend":
            s["workspace"] = K.paged_attend_workspace(s["cache"], H * case["group"])
    return s


def _filled_pool(case, pages, gen):
    """A pool whose every strip is one of 4096 strips of quantised rows: keys with an offset of their own in each
    channel, values around zero."""
    dev, bank, d = "cuda", 4096, case["dqk"] + case["dv"]
    x = torch.randn((bank, 16, d), generator=gen, device=dev, dtype=torch.float64)
    x[..., :case["dqk"]] += 0.5 * torch.randn((1, 1, case["dqk"]), generator=gen, device=dev, dtype=torch.float64)
    x = x.view(bank, 16, d // 64, 64)
    if case["fmt"] == "i4":
        codes, pair = _quantise(x)
        rows = torch.cat([codes.transpose(1, 2).reshape(bank, d // 64, 512),
                          pair.transpose(1, 2).contiguous().view(torch.uint8).reshape(bank, d // 64, 64)], -1).reshape(bank, -1)
    else:
        y = x.to(torch.bfloat16).view(bank, 16, d // 64, 8, 8)
        r = torch.arange(16, device=dev)
        piece = (torch.arange(8, device=dev)[None, :] ^ (r[:, None] & 7))[None, :, None, :, None].expand(y.shape)
        rows = y.gather(3, piece).transpose(1, 2).contiguous().view(torch.uint8).reshape(bank, -1)
    n = pages * case["heads"] * (case["page"] // 16)
    # whole strips moved as 64-bit words
    words = rows.contiguous().view(torch.int64).index_select(0, torch.randint(0, bank, (n,), generator=gen, device=dev))
    return words.view(torch.uint8).view(pages, case["heads"], -1)


# ---- the plain forms -----------------------------------------------------------------------------------------


def _frequencies(dim, scaling):
    """Angle of a pair for each position, in 64 bits, and the factor on what is turned."""
    factor, length, fast, slow = SCALING[scaling]
    i = torch.arange(dim // 2, dtype=torch.float64)
    theta = THETA * factor ** (dim / (dim - 2.0)) if scaling == "ntk" else THETA
    f = theta ** (-2.0 * i / dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        turns = length * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0)


def _turned(x, pos, s, back=False, wide=torch.float32):
    """x [T, heads, d] with its pairs turned by their positions [T], in `wide`."""
    case = s["case"]
    x = x.to(wide)
    if not case["dim"]:
        return x
    half, off = case["dim"] // 2, case["off"]
    ang = pos.to(torch.float64)[:, None] * s["freq"]
    c, n = (ang.cos() * s["mscale"]).to(wide)[:, None], (ang.sin() * s["mscale"]).to(wide)[:, None]
    n = -n if back else n
    part = x[..., off:off + case["dim"]]
    if case["layout"] == "half":
        a, b = part[..., :half], part[..., half:]
        new = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([x[..., :off], new, x[..., off + case["dim"]:]], -1)


def _fp16(x):
    """fp16 values nearest to x (float64), rounded once, within +-65504."""
    e = torch.frexp(x).exponent.to(torch.int64)
    ulp = (((e - 11).clamp(min=-24) + 1023) << 52).view(torch.float64)      # the power of two, by its bits
    return ((x / ulp).round() * ulp).clamp(-65504.0, 65504.0)


def _quantise(x):
    """Codes (two a byte) [..., 32] and (scale, minimum) [..., 2] of groups x [..., 64] in 64 bits."""
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(bad, 0.0, x)
    m = _fp16(x.amin(-1, keepdim=True))
    sc = _fp16((x.amax(-1, keepdim=True) - m).clamp(min=0) / 15)
    code = torch.where(sc > 0, ((x - m) / torch.where(sc > 0, sc, 1.0)).round(), 0.0).clamp(0, 15).to(torch.uint8)
    pair = torch.where(bad, float("nan"), torch.cat([sc, m], -1)).to(torch.float16)
    return code[..., 0::2] | (code[..., 1::2] << 4), pair


def _planes(pool, case):
    """Views of a pool: i4 (codes [..., 16, 32], pairs [..., 16, 2]), bf16 [..., 16, 8, 8]."""
    planes, strips = (case["dqk"] + case["dv"]) // 64, case["page"] // 16
    p = pool.view(pool.shape[:-1] + (strips, planes, -1))
    if case["fmt"] == "bf16":
        return p.view(torch.bfloat16).unflatten(-1, (16, 8, 8))
    return p[..., :512].unflatten(-1, (16, 32)), p[..., 512:].view(torch.float16).unflatten(-1, (16, 2))


def _places(s):
    """(sequence, position, page, strip, row) of each new token."""
    cu, P = s["cu"].long(), s["case"]["page"]
    t = torch.arange(int(s["q" if "q" in s else "k"].shape[0]), device=cu.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    pos = s["kv_len"].long()[n] - cu[n + 1] + t
    return n, pos, s["table_of_pages"][n, pos // P].long(), pos % P // 16, pos % 16


def _values(codes, pair):
    """fp32 values of codes [..., 32] with pairs [..., 2]."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.float32)
    pair = pair.to(torch.float32)
    return both * pair[..., :1] + pair[..., 1:]


def _append(s):
    case = s["case"]
    n, pos, page, strip, row = _places(s)
    x = torch.cat([_turned(s["k"], pos, s, wide=torch.float64), s["v"].to(torch.float64)], -1).unflatten(-1, (-1, 64))
    if case["fmt"] == "i4":
        codes, pairs = _planes(s["pool"], case)
        codes[page, :, strip, :, row], pairs[page, :, strip, :, row] = _quantise(x)
        y = _values(codes[page, :, strip, :, row], pairs[page, :, strip, :, row]).flatten(-2)
    else:
        rows = _planes(s["pool"], case)
        piece = (torch.arange(8, device=row.device) ^ (row[:, None] & 7))[:, None, None, :, None]
        x = x.to(torch.bfloat16).unflatten(-1, (8, 8))
        rows[page, :, strip, :, row] = x.gather(3, piece.expand(x.shape))
        y = rows[page, :, strip, :, row].gather(3, piece.expand(x.shape)).flatten(2)
    return y[..., :case["dqk"]].to(torch.bfloat16), y[..., case["dqk"]:].to(torch.bfloat16)


def _attend(s):
    case = s["case"]
    N, H, G, dqk, dv = case["n"], case["heads"], case["group"], case["dqk"], case["dv"]
    n, pos, _, _, _ = _places(s)
    if case["fmt"] == "i4":
        codes, pairs = _planes(s["pool"], case)
        y = _values(codes[s["table_of_pages"].long()], pairs[s["table_of_pages"].long()])
    else:
        y = _planes(s["pool"], case)[s["table_of_pages"].long()]
        r = torch.arange(16, device=y.device)
        piece = (torch.arange(8, device=y.device) ^ (r[:, None] & 7))[:, :, None]
        y = y.gather(-2, piece.expand(y.shape)).flatten(-2).to(torch.float32)
    # [N, pages, H, strips, planes, 16, 64] -> [N, H, tokens, channels]
    y = y.permute(0, 2, 1, 3, 5, 4, 6).reshape(N, H, -1, dqk + dv)
    i = torch.arange(n.numel(), device=n.device) - s["cu"].long()[n]
    q = torch.zeros((N, s["max_new"], H * G, dqk), device=n.device)
    q[n, i] = _turned(s["q"], pos, s)
    q = q.view(N, s["max_new"], H, G, dqk).permute(0, 2, 1, 3, 4).reshape(N, H, -1, dqk)
    score = q @ y[..., :dqk].transpose(-1, -2) * dqk ** -0.5
    count = s["cu"][1:] - s["cu"][:-1]
    last = (s["kv_len"] - count)[:, None] + torch.arange(s["max_new"], device=n.device)       # [N, new]
    seen = torch.arange(score.shape[-1], device=n.device) <= last[:, None, :, None, None]      # [N, 1, new, 1, keys]
    score = score.view(N, H, s["max_new"], G, -1).masked_fill(~seen, -float("inf")).view(score.shape)
    p = (score - score.amax(-1, keepdim=True)).exp()
    out = p @ y[..., dqk:] / p.sum(-1, keepdim=True)
    out = out.view(N, H, s["max_new"], G, dv).permute(0, 2, 1, 3, 4).reshape(N, s["max_new"], H * G, dv)[n, i]
    if s["gate"] is not None:
        out = out * (1 / (1 + (-s["gate"].to(torch.float32)).exp()))
    return out.to(_type(case["dtype"]))


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        K = s["K"]
        if op == "rope":
            return K.rope(s["q"], s["pos"], s["table"], k=s["k"])
        if op == "rope_grad":
            return K.rope_backward(s["q"], s["pos"], s["table"], dk_out=s["k"], k_shared=case["shared"])
        cu = None if s["single"] else s["cu"]
        if op == "append":
            K.paged_append(s["cache"], s["k"], s["v"], cu_seqlens=cu, rope=s["table"])
            return K.paged_read(s["cache"], s["k"].shape[0], cu_seqlens=cu, out_dtype=torch.bfloat16)
        return K.paged_attend(s["cache"], s["q"], cu_seqlens=cu, max_new=s["max_new"], rope=s["table"], gate=s["gate"], workspace=s["workspace"])
    if op == "rope":
        return tuple(_turned(x, s["pos"], s).to(x.dtype) for x in (s["q"], s["k"]))
    if op == "rope_grad":
        dq, dk = (_turned(x, s["pos"], s, back=True) for x in (s["q"], s["k"]))
        return dq.to(s["q"].dtype), (dk.sum(1, keepdim=True) if case["shared"] else dk).to(s["k"].dtype)
    return _append(s) if op == "append" else _attend(s)


# ---- the definition in 64 bits -------------------------------------------------------------------------------


def _exact_turn(x, pos, case, sign):
    """x [T, heads, d] in 64 bits: each pair as a complex number times mscale * exp(sign * i * pos * freq)."""
    dim, off = case["dim"], case["off"]
    if not dim:
        return x
    factor, length, fast, slow = SCALING[case["scaling"]]
    freq, grow = [], 1.0
    for j in range(dim // 2):
        f = math.pow(THETA, -2.0 * j / dim)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "ntk":
            f = math.pow(THETA * math.pow(factor, dim / (dim - 2.0)), -2.0 * j / dim)
        elif case["scaling"] == "by_parts":
            share = (length * f / (2 * math.pi) - slow) / (fast - slow)
            share = min(1.0, max(0.0, share))
            f = share * f + (1 - share) * f / factor
            grow = 0.1 * math.log(factor) + 1.0
        freq.append(f)
    ang = sign * pos.double().unsqueeze(1) * torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(ang, grow), ang).unsqueeze(1)
    first = range(off, off + dim // 2) if case["layout"] == "half" else range(off, off + dim, 2)
    first = torch.tensor(list(first), device=x.device)
    second = first + (dim // 2 if case["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_group(x):
    """What a group [..., 64] in 64 bits stands for once it is held in 4 bits."""
    def half(v):  # numpy rounds 64 bits to fp16 in one step
        return torch.from_numpy(v.cpu().numpy().astype("float16").astype("float64")).to(v.device)
    low = half(x.min(-1).values)
    step = half(torch.relu(x.max(-1).values - low) / 15.0)
    place = torch.nan_to_num((x - low.unsqueeze(-1)) / step.unsqueeze(-1), nan=0.0, posinf=0.0, neginf=0.0)
    return torch.round(place).clamp(0.0, 15.0) * step.unsqueeze(-1) + low.unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_grad"):
        sign = 1.0 if case["op"] == "rope" else -1.0
        q = _exact_turn(s["q"].double(), s["pos"], case, sign)
        k = _exact_turn(s["k"].double(), s["pos"], case, sign)
        return q, (k.sum(1, keepdim=True) if case["shared"] else k)
    past, new = _lengths(case)
    dqk, P = case["dqk"], case["page"]
    start = [0]
    for b in new:
        start.append(start[-1] + b)
    if case["op"] == "append":
        ks, vs = [], []
        for n, (a, b) in enumerate(zip(past, new)):
            at = slice(start[n], start[n + 1])
            k = _exact_turn(s["k"][at].double(), torch.arange(a, a + b, device="cuda"), case, 1.0)
            v = s["v"][at].double()
            if case["fmt"] == "i4":
                k, v = (_exact_group(t.reshape(t.shape[0], t.shape[1], -1, 64)).reshape(t.shape) for t in (k, v))
            ks.append(k)
            vs.append(v)
        return torch.cat(ks), torch.cat(vs)
    outs = []
    for n, (a, b) in enumerate(zip(past, new)):
        L, H, G = a + b, case["heads"], case["group"]
        blocks = s["pool"][s["table_of_pages"][n, :-(-L // P)].long()]                    # [pages, H, bytes]
        blocks = blocks.reshape(blocks.shape[0], H, P // 16, (dqk + case["dv"]) // 64, -1)
        if case["fmt"] == "i4":
            byte = blocks[..., :512].reshape(blocks.shape[:-1] + (16, 32))
            y = torch.empty(byte.shape[:-1] + (64,), dtype=torch.float64, device="cuda")
            y[..., 0::2], y[..., 1::2] = (byte % 16).double(), (byte // 16).double()
            par = blocks[..., 512:].contiguous().view(torch.float16).reshape(blocks.shape[:-1] + (16, 2)).double()
            y = y * par[..., 0:1] + par[..., 1:2]
        else:
            y = blocks.contiguous().view(torch.bfloat16).reshape(blocks.shape[:-1] + (16, 64)).double()
            z = torch.empty_like(y)
            for r in range(16):
                for c in range(8):
                    at = c ^ (r % 8)
                    z[..., r, 8 * c:8 * c + 8] = y[..., r, 8 * at:8 * at + 8]
            y = z
        y = y.permute(1, 0, 2, 4, 3, 5).reshape(H, -1, dqk + case["dv"])[:, :L]
        q = _exact_turn(s["q"][start[n]:start[n + 1]].double(), torch.arange(a, a + b, device="cuda"), case, 1.0)
        q = q.reshape(b, H, G, dqk).transpose(0, 1).reshape(H, b * G, dqk)
        w = torch.bmm(q, y[..., :dqk].transpose(1, 2)) / math.sqrt(dqk)
        hidden = torch.arange(L, device="cuda")[None, :] > (a + torch.arange(b, device="cuda"))[:, None]
        w = w.reshape(H, b, G, L).masked_fill(hidden[None, :, None, :], -math.inf).reshape(H, b * G, L)
        o = torch.bmm(torch.softmax(w, -1), y[..., dqk:])
        outs.append(o.reshape(H, b, G, -1).transpose(0, 1).reshape(b, H * G, -1))
    o = torch.cat(outs)
    return o * torch.sigmoid(s["gate"].double()) if s["gate"] is not None else o
