"""Plain 64-bit forms (numpy) of the rotary positions, the paged cache's formats and the attention over it, for the
tests; independent of the library and of torch's arithmetic."""
import math

import numpy as np


def frequencies(dim, theta=10000.0, scaling="none", factor=1.0, original_length=0.0, beta_fast=32.0, beta_slow=1.0):
    base = theta * factor ** (dim / (dim - 2.0)) if scaling == "ntk" else theta
    f = np.array([math.pow(base, -2.0 * i / dim) for i in range(dim // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        g = np.clip((original_length * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        f = g * f + (1 - g) * f / factor
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0)


def pairs(dim, offset, layout):
    i = np.arange(dim // 2)
    return (offset + i, offset + i + dim // 2) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)


def rotate(x, pos, dim, offset=0, layout="half", sign=1.0, **scaling):
    """x [T, H, d] float64, pos [T]."""
    x = np.array(x, dtype=np.float64)
    if dim == 0:
        return x
    f, m = frequencies(dim, **scaling)
    a, b = pairs(dim, offset, layout)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * f
    c, s = m * np.cos(ang), m * sign * np.sin(ang)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotate_slack(x, dim, offset, layout, mscale=1.0):
    """Bound on the FP32 rotation's error, channel by channel: 4.8e-7 (|x| + |y|) of the pair (three roundings of 2^-24, and
    2^-22.5 for the cosine and sine), 0 for channels that pass through."""
    e = np.zeros(x.shape)
    if dim:
        a, b = pairs(dim, offset, layout)
        e[..., a] = e[..., b] = 4.8e-7 * mscale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return e


def fp16(x):
    with np.errstate(over="ignore"):
        return np.clip(np.asarray(x, np.float64), -65504.0, 65504.0).astype(np.float16).astype(np.float64)


def quantise(x):
    """Groups [..., 64] -> (codes uint8 [..., 64], scale, minimum)."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    m = fp16(x.min(-1))
    s = fp16(np.maximum(x.max(-1) - m, 0.0) / 15.0)
    safe = np.where(s > 0, s, 1.0)
    code = np.clip(np.rint((x - m[..., None]) / safe[..., None]), 0, 15)
    code = np.where((s > 0)[..., None], code, 0).astype(np.uint8)
    return code, np.where(bad, np.nan, s), np.where(bad, np.nan, m)


def strips_i4(rows):
    """Rows [heads, page, d] of one page -> its blocks' bytes [heads, block]."""
    H, P, d = rows.shape
    code, s, m = quantise(rows.reshape(H, P, d // 64, 64))
    byte = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(H, P // 16, 16, d // 64, 32)
    par = np.stack([s, m], -1).astype(np.float16).reshape(H, P // 16, 16, d // 64, 2)
    byte = byte.transpose(0, 1, 3, 2, 4).reshape(H, P // 16, d // 64, 512)
    par = np.ascontiguousarray(par.transpose(0, 1, 3, 2, 4)).view(np.uint8).reshape(H, P // 16, d // 64, 64)
    return np.concatenate([byte, par], -1).reshape(H, -1)


def unpack_i4(block, P, d):
    """Blocks' bytes [..., block] -> values [..., P, d]."""
    lead = block.shape[:-1]
    b = block.reshape(lead + (P // 16, d // 64, 576))
    byte = b[..., :512].reshape(lead + (P // 16, d // 64, 16, 32))
    par = np.ascontiguousarray(b[..., 512:]).view(np.float16).reshape(lead + (P // 16, d // 64, 16, 2)).astype(np.float64)
    v = np.empty(byte.shape[:-1] + (64,))
    v[..., 0::2], v[..., 1::2] = byte & 15, byte >> 4
    v = v * par[..., :1] + par[..., 1:]
    return np.moveaxis(v, -3, -2).reshape(lead + (P, d))


def unpack_bf16(block, P, d):
    lead = block.shape[:-1]
    w = np.ascontiguousarray(block).view(np.uint16).reshape(lead + (P // 16, d // 64, 16, 8, 8)).astype(np.uint32)
    v = (w << 16).view(np.float32).astype(np.float64)
    out = np.empty_like(v)
    for r in range(16):
        for c in range(8):
            out[..., r, c, :] = v[..., r, c ^ (r & 7), :]
    out = out.reshape(lead + (P // 16, d // 64, 16, 64))
    return np.moveaxis(out, -3, -2).reshape(lead + (P, d))


def unpack(block, P, d, fmt):
    return unpack_i4(block, P, d) if fmt == "i4" else unpack_bf16(block, P, d)


def attend(q, k, v, seen, scale, gate=None):
    """q [c, Hq, dqk], k [L, H, dqk], v [L, H, dv], seen [c] (keys each token sees) -> [c, Hq, dv]; a token that sees
    none gets zeros."""
    c, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((c, Hq, v.shape[2]))
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(c):
            n = int(seen[i])
            if n <= 0:
                continue
            for h in range(Hq):
                s = scale * (k[:n, h // G] @ q[i, h])
                p = np.exp(s - s.max())
                out[i, h] = (p @ v[:n, h // G]) / p.sum()
        return out if gate is None else out / (1.0 + np.exp(-gate))


def strips_bf16(rows):
    """Rows [heads, page, d] that bf16 holds -> blocks' bytes [heads, block]."""
    H, P, d = rows.shape
    w = (np.ascontiguousarray(rows, np.float32).view(np.uint32) >> 16).astype(np.uint16).reshape(H, P // 16, 16, d // 64, 8, 8)
    out = np.empty_like(w)
    for r in range(16):
        for c in range(8):
            out[:, :, r, :, c ^ (r & 7)] = w[:, :, r, :, c]
    return np.ascontiguousarray(out.transpose(0, 1, 3, 2, 4, 5)).view(np.uint8).reshape(H, -1)
