"""The paged cache's operators at values, arrays and streams where they could go wrong: against the 64-bit forms, or against what the header
says of such data."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import paged_plain as PP  # noqa: E402
from test_gpu_paged_append import Case as Append  # noqa: E402
from test_gpu_paged_attend import Case as Attend, _check, _long  # noqa: E402

DEV = "cuda:0"


def _np(t):
    return t.detach().cpu().double().numpy()


def _stored(c, k):
    """What the definition stores for keys k (float64, turned) and the case's values."""
    want = np.concatenate([k, _np(c.v)], -1)
    code, s, m = PP.quantise(want.reshape(len(want), c.heads, -1, 64))
    return (code * s[..., None] + m[..., None]).reshape(want.shape)


@pytest.mark.parametrize("base,step", [(20000.0, 2.0 ** -9), (-60000.0, 2.0 ** -8), (2048.0, 2.0 ** -12), (512.0, 2.0 ** -14), (-1040.0, 2.0 ** -13)])
@pytest.mark.parametrize("most", [8, 40, 300])
def test_groups_far_from_zero_and_narrow(base, step, most):
    """FP32 channels of one large value plus 0..most units of its last place: the minimum over the scale has more bits than FP32."""
    rng = np.random.default_rng(most)
    c = Append([0, 9], [64, 30], 4, 128, 64, 32, "i4", torch.float32, make=lambda *s: base + step * rng.integers(0, most + 1, s))
    K.paged_append(c.cache, c.k, c.v, c.cu)
    assert np.array_equal(c.rows(), _stored(c, _np(c.k)))


def _wide(s, rng):
    """Finite channels up to FP32's largest: groups of both signs, of one sign, and of a few such channels among ordinary ones."""
    x = rng.standard_normal(s)
    kind = rng.integers(0, 4, s[:2] + (1,))
    big = rng.uniform(1.8e38, 3.3e38, s) * np.where(rng.random(s) < 0.5, -1.0, 1.0)
    some = rng.random(s) < 0.05
    return np.where(kind == 0, big, np.where(kind == 1, np.abs(big), np.where((kind == 2) & some, big, x)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rope", [None, dict(dim=128), dict(dim=64, offset=64, layout="interleaved"),
                                  dict(dim=34, offset=5, scaling="by_parts", factor=16.0, original_length=4096.0)], ids=str)
def test_finite_groups_wider_than_fp32(rope, dtype):
    """Groups whose range, or whose rotation, exceeds FP32's largest value hold no infinity: their scale and minimum saturate."""
    rng = np.random.default_rng(3)
    c = Append([0, 40], [64, 50], 4, 128, 64, 32, "i4", dtype, make=lambda *s: _wide(s, rng))
    K.paged_append(c.cache, c.k, c.v, c.cu, rope=K.rope_table(device=DEV, **rope) if rope else None)
    k = PP.rotate(_np(c.k), c.pos, **rope) if rope else _np(c.k)
    got = c.rows()
    assert np.isfinite(got).all()
    assert np.array_equal(got, _stored(c, k))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_turned_channel_that_is_not_finite_beside_wide_ones(value):
    """Of the two groups of each turned head, those that a channel which is not finite reaches are NaN, the others are not."""
    rng = np.random.default_rng(4)
    c = Append([3], [20], 2, 128, 64, 16, "i4", torch.float32, make=lambda *s: _wide(s, rng))
    c.k[4, 1, 70], c.k[7, 0, 3] = value, value                # half layout over 64 channels: 70 does not turn, 3 turns with 35
    K.paged_append(c.cache, c.k, c.v, c.cu, rope=K.rope_table(64, device=DEV))
    gone = np.isnan(c.rows()).reshape(20, 2, 3, 64)
    assert gone[4, 1, 1].all() and gone[7, 0, 0].all() and gone.sum() == 128


@pytest.mark.parametrize("total,new,heads,group", [([37, 2], [37, 1], 2, 1), ([40, 3], [4, 3], 2, 1), ([30], [12], 2, 4), ([5000], [12], 1, 1), ([5000], [3], 1, 2)], ids=str)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_row_whose_keys_all_score_minus_infinity(total, new, heads, group, out):
    """As in a plain softmax: NaN while no key scores more, ordinary once one does."""
    spoiled = [t - c + min(3, c - 1) if c > 1 else t for t, c in zip(total, new)]      # keys 0 .. of each sequence

    def spoil(n, rows):
        rows[:spoiled[n], 0, 3] = float("inf")
    c = Attend(total, new, heads, group, 128, 128, 16, "bf16", seed=12, edit=spoil)
    c.q[:, :, 3] = -0.75
    want, tol = c.want()
    got = c.run(out)
    assert np.isnan(want).any() and np.isfinite(want).any()
    _check(got, want, tol, out)


def _bounds(c):
    """The attention cases' bounds for all rows."""
    return np.concatenate([c._bound(n, PP.rotate(_np(c.q[int(c.cu[n]):int(c.cu[n + 1])]), np.arange(t - m, t), *c.rope), m)
                           for n, (t, m) in enumerate(zip(c.total, c.new))])


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("total,new,heads,group,width", [([3001], [3001], 2, 4, 1 << 20), ([2048, 1500], [2048, 1400], 8, 8, 1 << 18),
                                                         ([1030, 7, 4000], [1030, 7, 3333], 3, 1, 1 << 22)], ids=str)
def test_long_prompts_under_wide_tables(fmt, total, new, heads, group, width):
    """Prompts of thousands of tokens, from position 0 and behind cached ones, with a block table made for long contexts: against the
    64-bit form, and the bits of a narrow table."""
    c = Attend(total, new, heads, group, 128, 128, 64, fmt, (128, 0, "half"), seed=41)
    narrow = c.run()
    _check(narrow, _long(c), _bounds(c))
    tab = np.full((len(total), width // 64), -3, np.int32)
    tab[:, :c.tab.shape[1]] = c.tab
    c.cache = K.PagedCache(c.pool, torch.from_numpy(tab).to(DEV), c.cache.kv_len, 64, 128, 128, fmt)
    assert torch.equal(c.run(), narrow)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("max_new", [1, 6, 60])
@pytest.mark.parametrize("cu", [[0, 60, 0, 60, 0, 60], [0, 20, 10, 30, 40, 60], [0, 60, 60, 60, 60, 59], [7, 5, 60, 60, 60, 60]], ids=str)
def test_a_packing_that_decreases(cu, max_new, fmt):
    """Sequences that overlap count more rows than the call has: nothing is attended to, every output is NaN."""
    c = Attend([100] * 5, [12] * 5, 2, 4, 128, 128, 16, fmt, seed=2)
    right = c.run()
    ws = K.paged_attend_workspace(c.cache, 8)
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    for out in (torch.float32, torch.bfloat16):
        assert torch.isnan(K.paged_attend(c.cache, c.q, bad, max_new, scale=c.scale, out_dtype=out, workspace=ws)).all()
    assert torch.equal(c.run(ws=ws), right) and K.k3kda_workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("max_new", [None, 1, 3, 9, 400])
@pytest.mark.parametrize("new,group", [([1, 0, 40, 2, 0, 0, 0, 7], 2), ([1, 0, 3, 2, 0, 0, 0, 1], 4), ([0, 8, 0, 0, 0, 0, 0, 0], 1)], ids=str)
def test_max_new_chooses_a_kernel_and_changes_no_result(new, group, max_new, fmt):
    """Too small or too large: whichever kernel takes the call reads the counts that there are."""
    c = Attend([60 + 30 * i for i in range(8)], new, 2, group, 128, 128, 32, fmt, (64, 0, "interleaved"), gate=True, seed=15)
    want, tol = [], []
    for n, (t, m) in enumerate(zip(c.total, new)):
        if m:
            at = slice(int(c.cu[n]), int(c.cu[n + 1]))
            q = PP.rotate(_np(c.q[at]), np.arange(t - m, t), *c.rope)
            want.append(PP.attend(q, c.k[n], c.v[n], t - m + 1 + np.arange(m), c.scale, _np(c.gate[at])))
            tol.append(c._bound(n, q, m))
    want, tol = np.concatenate(want), np.concatenate(tol)
    table = K.rope_table(64, layout="interleaved", device=DEV)
    _check(K.paged_attend(c.cache, c.q, c.cu, max_new, table, gate=c.gate, out_dtype=torch.float32), want, tol)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("dqk,rows", [(64, 4), (64, 5), (64, 8), (64, 9), (64, 44), (64, 45), (128, 36), (128, 37), (192, 28), (192, 29), (256, 60)])
def test_both_sides_of_the_borders_between_the_kernels(dqk, rows, fmt):
    """4-bit pages: four rows, eight, then blocks of 128 from 45, 37 and 29 rows on; bf16 pages from 9; keys of 256 channels never.  Short
    sequences and ones that many CTAs share."""
    for total, new, heads, group in (([300, rows, 77], [rows] * 3, 2, 1), ([15000], [1], 2, rows)):
        c = Attend(total, new, heads, group, dqk, 128, 64, fmt, (64, 0, "half"), seed=rows)
        _check(c.run(), _long(c), _bounds(c))


@pytest.mark.parametrize("fmt,group", [("i4", 4), ("i4", 8), ("i4", 64), ("bf16", 4), ("bf16", 8), ("bf16", 64)])
@pytest.mark.parametrize("what", ["queries", "weights"])
def test_both_parts_of_queries_and_weights_count(what, fmt, group):
    """Two keys a sequence: the first scores 0, the second what the difference of two large products leaves ("queries", so that an error of
    2^-16 of either shows) or one small product ("weights").  Values of 0 and of 0..15.

    Bounds: parts of 16 bits leave 2^-16 of a query's channel or of a weight, parts of 22 bits 2^-22, FP32's sums and exponentials 2^-20;
    a score's error d moves p = 1 / (1 + e^-s) by at most d / 4.  One part alone is off by 2^-9 or 2^-12: a hundred times the bound."""
    large = 4096.0 if fmt == "bf16" else 7680.0                            # 15 * 512: its group's scale is exact
    key = large if what == "queries" else 1.0 if fmt == "bf16" else 15.0

    def edit(n, rows):
        rows[...] = 0
        rows[1, :, :2] = key
        rows[1, :, 128:] = np.arange(128) % 16
    c = Attend([2] * 8, [1] * 8, 16, group, 128, 128, 16, fmt, dtype=torch.float32, seed=1, edit=edit)
    rng = np.random.default_rng(group)
    q = np.zeros(tuple(c.q.shape))
    if what == "queries":
        q[..., 1] = rng.uniform(0.5, 2.0, q.shape[:2])
        q[..., 0] = rng.uniform(-2.0, 2.0, q.shape[:2]) / (key * c.scale) - q[..., 1]
    else:
        q[..., 0] = rng.uniform(-3.0, 3.0, q.shape[:2]) / (key * c.scale)
    c.q.copy_(torch.from_numpy(q.astype(np.float32)))
    want, _ = c.want()
    part = (2.0 ** -16 if fmt == "bf16" else 2.0 ** -22) + 2.0 ** -20
    score = key * c.scale * np.abs(_np(c.q)[..., :2]).sum(-1, keepdims=True) * part
    p = want[..., 15:16] / 15
    err = np.abs(_np(c.run()) - want)
    assert (err <= (np.arange(128) % 16) * (score / 4 + p * part)).all(), f"{(err.max(-1) / (15 * (score[..., 0] / 4 + p[..., 0] * part))).max():.2f}"
