"""Rotary positions on the GPU against the 64-bit form: forward and gradient, both layouts, part of the head,
scaled frequencies, both types, odd sizes, strided and shared heads, in place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import paged_plain as PP  # noqa: E402

BF_HALF = 2.0 ** -8                                          # half a bf16 step, relative to the value
DEV = "cuda:0"


def _rand(shape, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).to(dtype).to(DEV)


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(got, want, slack, dtype, what):
    tol = slack * (1 + BF_HALF) + (BF_HALF if dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(want)
    err = np.abs(_np(got) - want)
    assert got.dtype == dtype
    assert (err <= tol).all(), f"{what}: {err.max():.3e}, {(err - tol).max():.3e} over"


SHAPES = [  # T, Hq, Hk, d, dim, offset
    (1, 1, 0, 64, 64, 0), (1, 32, 8, 128, 128, 0), (3, 4, 4, 192, 64, 128), (37, 5, 1, 128, 64, 32), (7, 3, 2, 70, 34, 5),
    (300, 2, 1, 64, 32, 0), (129, 1, 1, 16, 16, 0), (5, 2, 0, 9, 2, 3), (2, 40, 8, 256, 48, 208), (4, 2, 2, 1024, 512, 256)]
SCALINGS = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=16.0, original_length=4096.0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_forward_and_gradient(shape, layout, dtype):
    T, Hq, Hk, d, dim, off = shape
    q, k = _rand((T, Hq, d), dtype, 1), _rand((T, Hk, d), dtype, 2) if Hk else None
    pos = torch.from_numpy(np.random.default_rng(3).integers(0, 5000, T).astype(np.int32)).to(DEV)
    table = K.rope_table(dim, offset=off, layout=layout, device=DEV)
    for sign, fn in ((1.0, K.rope), (-1.0, K.rope_backward)):
        got = fn(q, pos, table, k) if sign > 0 else fn(q, pos, table, dk_out=k)
        got = got if Hk else (got,)
        for x, y in zip((q, k), got):
            xn = _np(x)
            want = PP.rotate(xn, _np(pos), dim, off, layout, sign)
            _check(y, want, PP.rotate_slack(xn, dim, off, layout), dtype, f"sign {sign}")
            keep = np.ones(d, bool)
            keep[off:off + dim] = False
            assert np.array_equal(_np(y)[..., keep], xn[..., keep])


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k["scaling"])
@pytest.mark.parametrize("top", [100, 1 << 17, 2 ** 31 - 1])
def test_scaled_frequencies_and_far_positions(kw, top):
    """The angle keeps its accuracy at any int32 position: beyond the rotation's own error only the table's (a
    frequency's 2^-52, on both sides) times the position."""
    T, d = 64, 128
    q = _rand((T, 2, d), torch.float32, 4)
    p = np.random.default_rng(5).integers(-top, top, T).astype(np.int32)
    p[:3] = 0, top, -top
    table = K.rope_table(d, device=DEV, **kw)
    got = K.rope(q, torch.from_numpy(p).to(DEV), table)
    want = PP.rotate(_np(q), p, d, **kw)
    m = table.mscale
    angle = 4 * 2.0 ** -52 * top * m * 2 * np.abs(_np(q)).max()
    _check(got, want, PP.rotate_slack(_np(q), d, 0, "half", m) + angle, torch.float32, kw["scaling"])


def test_position_zero_is_the_identity_and_gradient_is_the_transpose():
    q = _rand((8, 3, 64), torch.float32, 6)
    table = K.rope_table(64, device=DEV)
    assert torch.equal(K.rope(q, torch.zeros(8, dtype=torch.int32, device=DEV), table), q)
    pos = torch.arange(8, dtype=torch.int32, device=DEV) * 1001
    g = _rand((8, 3, 64), torch.float32, 7)
    # <g, R x> = <R^T g, x>: sums of 64 products, each with the rotation's slack
    a, b = (_np(g) * _np(K.rope(q, pos, table))).sum(-1), (_np(K.rope_backward(g, pos, table)) * _np(q)).sum(-1)
    assert np.abs(a - b).max() <= 2 * 64 * 4.8e-7 * 2 * np.abs(_np(q)).max() * np.abs(_np(g)).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """A central difference of L(x) = <w, rope(x)>, which is linear: only FP32's rounding remains."""
    x, w = _rand((3, 2, 64), torch.float32, 8), _rand((3, 2, 64), torch.float32, 9)
    pos = torch.tensor([1, 77, 40000], dtype=torch.int32, device=DEV)
    table = K.rope_table(32, offset=16, layout=layout, scaling="by_parts", factor=4.0, original_length=1000.0, device=DEV)
    g = _np(K.rope_backward(w, pos, table))
    for at in ((0, 0, 3), (0, 1, 16), (1, 0, 31), (1, 1, 32), (2, 0, 47), (2, 1, 63)):
        e = torch.zeros_like(x)
        e[at] = 1.0
        up, down = (_np(K.rope(x + s * e, pos, table)) * _np(w) for s in (1.0, -1.0))
        assert abs((up.sum() - down.sum()) / 2 - g[at]) <= 8 * 4.8e-7 * (np.abs(_np(x)).max() + 1) * np.abs(_np(w)).max() * 2


@pytest.mark.parametrize("shape", [(1, 32, 32, 128, 128, 0), (33, 8, 8, 192, 64, 128), (5, 3, 40, 70, 34, 5), (64, 1, 7, 64, 32, 32)], ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_shared_key_head_gets_the_sum(shape, layout, dtype):
    T, Hq, Hk, d, dim, off = shape
    one = _rand((T, 1, d), dtype, 10)
    q, dq, dk = _rand((T, Hq, d), dtype, 11), _rand((T, Hq, d), dtype, 12), _rand((T, Hk, d), dtype, 13)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 97
    table = K.rope_table(dim, offset=off, layout=layout, device=DEV)
    # forward: one head, stride 0, written out to every head
    _, ko = K.rope(q, pos, table, one.expand(T, Hk, d))
    want = PP.rotate(_np(one), _np(pos), dim, off, layout)
    _check(ko, np.broadcast_to(want, (T, Hk, d)), np.broadcast_to(PP.rotate_slack(_np(one), dim, off, layout), (T, Hk, d)), dtype, "forward")
    gq, gk = K.rope_backward(dq, pos, table, dk_out=dk, k_shared=True)
    _check(gq, PP.rotate(_np(dq), _np(pos), dim, off, layout, -1.0), PP.rotate_slack(_np(dq), dim, off, layout), dtype, "dq")
    total, size = _np(dk).sum(1, keepdims=True), np.abs(_np(dk)).sum(1, keepdims=True)
    # the sum's rounding (Hk terms, each at most the sum of magnitudes), then the rotation
    slack = PP.rotate_slack(size, dim, off, layout) + 2 * Hk * 2.0 ** -24 * PP.rotate_slack(size, dim, off, layout) / 4.8e-7 + Hk * 2.0 ** -24 * size
    assert gk.shape == (T, 1, d)
    _check(gk, PP.rotate(total, _np(pos), dim, off, layout, -1.0), slack, dtype, "dk")
    again = K.rope_backward(dq, pos, table, dk_out=dk, k_shared=True)[1]
    assert torch.equal(gk, again)


@pytest.mark.parametrize("shift", [0, 1])
def test_strided_views_and_in_place(shift):
    """Slices of a fused projection, aligned and not, and rotation in place, which leaves the rest untouched."""
    T, H, d, dim, off = 19, 3, 128, 64, 64
    fused = _rand((T, 3 * H * d + 2 * shift), torch.bfloat16, 14)
    q = fused[:, shift:shift + H * d].unflatten(1, (H, d))
    k = fused[:, shift + H * d:shift + 2 * H * d].unflatten(1, (H, d))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = K.rope_table(dim, offset=off, device=DEV)
    before = fused.clone()
    qo, ko = K.rope(q, pos, table, k)
    assert torch.equal(before, fused)
    for x, y in ((q, qo), (k, ko)):
        _check(y, PP.rotate(_np(x), _np(pos), dim, off), PP.rotate_slack(_np(x), dim, off, "half"), torch.bfloat16, "view")
    K.rope(q, pos, table, k, out=(q, k))
    assert torch.equal(q, qo) and torch.equal(k, ko)
    rest = torch.ones(fused.shape[1], dtype=torch.bool, device=DEV)
    rest[shift:shift + 2 * H * d] = False
    assert torch.equal(fused[:, rest], before[:, rest])


def test_no_tokens_other_stream_and_graph():
    table = K.rope_table(64, device=DEV)
    assert K.rope(torch.empty(0, 2, 64, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), table).shape == (0, 2, 64)
    q = _rand((50, 4, 64), torch.float32, 15)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    want = K.rope(q, pos, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = K.rope(q, pos, table, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        K.rope(q, pos, table, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A view whose rows lie more than 2^32 bytes apart."""
    big = torch.zeros(3, (1 << 31) + 64, dtype=torch.bfloat16, device=DEV)
    x = big[:, -64:].unflatten(1, (1, 64))
    x.copy_(_rand((3, 1, 64), torch.bfloat16, 16))
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    table = K.rope_table(64, device=DEV)
    got = K.rope(x, pos, table)
    _check(got, PP.rotate(_np(x), _np(pos), 64), PP.rotate_slack(_np(x), 64, 0, "half"), torch.bfloat16, "far")
