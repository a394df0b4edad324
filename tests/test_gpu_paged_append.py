"""The paged cache on the GPU against the 64-bit definition of its formats: what append stores (4-bit blocks byte
for byte), what read gives back, and what neither may touch."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import paged_plain as PP  # noqa: E402

DEV = "cuda:0"
BF_HALF = 2.0 ** -8


def _np(t):
    return t.detach().cpu().double().numpy()


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """N sequences with `past` tokens cached and `new` ones to come, pages in a shuffled order, spare pages around."""

    def __init__(self, past, new, heads, dqk, dv, page, fmt, dtype=torch.bfloat16, seed=0, fill=0xA5, make=None):
        rng = np.random.default_rng(seed)
        self.past, self.new, self.total = past, new, [a + b for a, b in zip(past, new)]
        N, T = len(past), sum(new)
        need = [-(-t // page) for t in self.total]
        width, spare = max(need + [1]) + 1, 3
        order = rng.permutation(sum(need) + spare)
        self.spare = order[sum(need):]
        self.tab = np.full((N, width), -7, np.int32)         # entries past a length are never looked at
        at = 0
        for n, c in enumerate(need):
            self.tab[n, :c] = order[at:at + c]
            at += c
        self.page, self.fmt, self.heads, self.dqk, self.dv = page, fmt, heads, dqk, dv
        self.pool = K.paged_pool(len(order), page, heads, dqk, dv, fmt, DEV)
        self.pool.fill_(fill)
        self.cache = K.PagedCache(self.pool, _i(self.tab), _i(self.total), page, dqk, dv, fmt)
        make = make or (lambda *s: rng.standard_normal(s))
        self.k = torch.from_numpy(make(T, heads, dqk).astype(np.float32)).to(dtype).to(DEV)
        self.v = torch.from_numpy(make(T, heads, dv).astype(np.float32)).to(dtype).to(DEV)
        self.cu = _i(np.concatenate([[0], np.cumsum(new)]))
        self.pos = np.concatenate([np.arange(a, a + b) for a, b in zip(past, new)]) if T else np.zeros(0, int)
        self.seq = np.repeat(np.arange(N), new)

    def rows(self):
        """What the pool stands for at the new tokens: [T, heads, dqk + dv]."""
        block = self.pool.cpu().numpy()
        vals = PP.unpack(block, self.page, self.dqk + self.dv, self.fmt)
        return vals[self.tab[self.seq, self.pos // self.page], :, self.pos % self.page]


CASES = [  # past, new, heads, dqk, dv, page, rope (dim, offset, layout)
    ([0], [1], 1, 64, 64, 16, (64, 0, "half")),
    ([511, 0, 3], [1, 1, 1], 8, 128, 128, 64, (128, 0, "half")),
    ([0, 5, 16, 70], [16, 11, 0, 33], 2, 192, 128, 16, (64, 128, "interleaved")),
    ([100, 0, 31], [3, 200, 66], 3, 128, 128, 32, (32, 16, "half")),
    ([7, 9], [0, 130], 1, 256, 256, 128, (0, 0, "half")),
    ([63, 64], [65, 1], 4, 64, 128, 48, (34, 5, "interleaved")),
    ([2], [75], 5, 256, 64, 256, (48, 208, "half"))]


def _table(r):
    return K.rope_table(r[0], offset=r[1], layout=r[2], device=DEV) if r[0] else None


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_append_stores_the_definition(case, dtype, fmt):
    past, new, heads, dqk, dv, page, rope = case
    c = Case(past, new, heads, dqk, dv, page, fmt, dtype, seed=sum(new))
    before = c.pool.clone()
    K.paged_append(c.cache, c.k, c.v, None if max(new) == min(new) == 1 else c.cu, rope=_table(rope))
    want = np.concatenate([PP.rotate(_np(c.k), c.pos, rope[0], rope[1], rope[2]), _np(c.v)], -1)
    got = c.rows()
    if fmt == "i4":
        code, s, m = PP.quantise(want.reshape(len(want), heads, -1, 64))
        assert np.array_equal(got, (code * s[..., None] + m[..., None]).reshape(want.shape))
    else:
        slack = np.concatenate([PP.rotate_slack(_np(c.k), *rope), np.zeros_like(_np(c.v))], -1)
        assert (np.abs(got - want) <= BF_HALF * np.abs(want) + slack * (1 + BF_HALF)).all()
        exact = slack == 0
        assert np.array_equal(got[exact], torch.from_numpy(want[exact].astype(np.float32)).bfloat16().double().numpy())
    # nothing else changed: restore the new tokens' rows and compare all bytes
    after, old = c.pool.cpu().numpy().copy(), before.cpu().numpy()
    planes, size = (dqk + dv) // 64, 576 if fmt == "i4" else 2048
    a, o = (x.reshape(len(x), heads, page // 16, planes, size) for x in (after, old))
    for n, p in zip(c.seq, c.pos):
        pg, st, r = c.tab[n, p // page], p % page // 16, p % 16
        for lo, w in ((r * 32, 32), (512 + r * 4, 4)) if fmt == "i4" else ((r * 128, 128),):
            a[pg, :, st, :, lo:lo + w] = o[pg, :, st, :, lo:lo + w]
    assert np.array_equal(after, old)
    # and read gives the values, rounded once
    for out in (torch.float32, torch.bfloat16):
        kr, vr = K.paged_read(c.cache, len(want), None if max(new) == min(new) == 1 else c.cu, out)
        both = np.concatenate([_np(kr), _np(vr)], -1)
        assert (np.abs(both - got) <= (BF_HALF * (1 + 2.0 ** -16) if out == torch.bfloat16 else 2.0 ** -24) * np.abs(got)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["integers", "constant", "zeros", "huge", "tiny", "spread", "near ties"])
def test_codes_where_rounding_is_close(kind, dtype):
    """Groups made of ties, of one value, past fp16's range, in its denormals: the bytes are still the definition's."""
    rng = np.random.default_rng(7)
    make = {"integers": lambda *s: rng.integers(-15, 16, s).astype(float),
            "constant": lambda *s: np.broadcast_to(rng.standard_normal(s[:2] + (1,)), s).copy(),
            "zeros": lambda *s: np.zeros(s),
            "huge": lambda *s: rng.standard_normal(s) * 10.0 ** rng.integers(3, 9, s[:2] + (1,)),
            "tiny": lambda *s: rng.standard_normal(s) * 10.0 ** -rng.integers(3, 12, s[:2] + (1,)).astype(float),
            "spread": lambda *s: rng.standard_normal(s) * 10.0 ** rng.integers(-6, 4, s).astype(float),
            "near ties": lambda *s: rng.integers(0, 31, s) / 2.0 + rng.integers(-2, 3, s) * 2.0 ** -20}[kind]
    c = Case([0, 40], [64, 200], 4, 128, 128, 32, "i4", dtype, make=make)
    K.paged_append(c.cache, c.k, c.v, c.cu)
    want = np.concatenate([_np(c.k), _np(c.v)], -1)
    code, s, m = PP.quantise(want.reshape(len(want), 4, -1, 64))
    assert np.array_equal(c.rows(), (code * s[..., None] + m[..., None]).reshape(want.shape))


def test_many_rotated_groups_match_the_definition_byte_for_byte():
    """Half a million rotated groups: hundreds lie closer to a border than FP32 can tell."""
    c = Case([0, 3000], [4000, 300], 60, 128, 64, 64, "i4", torch.bfloat16, seed=11)
    K.paged_append(c.cache, c.k, c.v, c.cu, rope=K.rope_table(128, device=DEV))
    want = PP.rotate(_np(c.k), c.pos, 128)
    code, s, m = PP.quantise(want.reshape(len(want), 60, 2, 64))
    got = c.rows()[..., :128]
    assert np.array_equal(got, (code * s[..., None] + m[..., None]).reshape(want.shape))


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite_stays_in_its_group(fmt, value):
    c = Case([3], [20], 2, 128, 128, 16, fmt)
    c.k[4, 1, 70], c.v[9, 0, 3] = value, value
    K.paged_append(c.cache, c.k, c.v, c.cu)
    got, want = c.rows(), np.concatenate([_np(c.k), _np(c.v)], -1)
    if fmt == "bf16":
        assert np.array_equal(got, want, equal_nan=True)
        return
    gone = np.isnan(got).reshape(20, 2, 4, 64)
    assert gone[4, 1, 1].all() and gone[9, 0, 2].all() and gone.sum() == 128


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_bad_pages_and_lengths_are_left_out(fmt):
    """A page outside the pool, a length past the table or below the new tokens: nothing is written there, read gives
    NaN; the other tokens are stored as ever."""
    past, new = [20, 5, 0, 9], [30, 12, 6, 4]
    c = Case(past, new, 2, 128, 64, 16, fmt)
    tab = c.tab.copy()
    tab[0, 2] = len(c.pool)                                  # tokens 32..47 of sequence 0
    lens = list(c.total)
    lens[1], lens[2] = tab.shape[1] * 16 + 1, 4              # too long; 2 of its 6 tokens before position 0
    c.cache.block_table.copy_(_i(tab))
    c.cache.kv_len.copy_(_i(lens))
    before = c.pool.clone()
    K.paged_append(c.cache, c.k, c.v, c.cu)
    kr, vr = K.paged_read(c.cache, sum(new), c.cu, torch.float32)
    bad = np.zeros(sum(new), bool)
    pos = c.pos.copy()
    pos[42:48] = np.arange(-2, 4)
    bad[:30] = (pos[:30] >= 32) & (pos[:30] < 48)
    bad[30:42] = True
    bad[42:44] = True
    got = np.concatenate([_np(kr), _np(vr)], -1)
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    want = np.concatenate([_np(c.k), _np(c.v)], -1)
    if fmt == "i4":
        code, s, m = PP.quantise(want.reshape(len(want), 2, -1, 64))
        want = (code * s[..., None] + m[..., None]).reshape(want.shape)
    assert (np.abs(got[~bad] - want[~bad]) <= 2.0 ** -24 * np.abs(want[~bad])).all()
    for p in range(len(c.pool)):                             # pages of no stored token are as they were
        used = {int(tab[n, q // 16]) for n, q, b in zip(c.seq, pos, bad) if not b}
        if p not in used:
            assert torch.equal(c.pool[p], before[p])


def test_strided_rows_and_no_tokens():
    c = Case([4, 0], [9, 28], 3, 128, 128, 32, "i4")
    for pad in (0, 3):                                       # 16-byte aligned rows, and not
        wide = torch.zeros(37, 3, 256 + 8 * (pad == 0) + pad, dtype=torch.bfloat16, device=DEV)
        wide[..., pad:pad + 128], wide[..., 128 + pad:256 + pad] = c.k, c.v
        K.paged_append(c.cache, wide[..., pad:pad + 128], wide[..., 128 + pad:256 + pad], c.cu, rope=K.rope_table(64, device=DEV))
        one = c.pool.clone()
        K.paged_append(c.cache, c.k, c.v, c.cu, rope=K.rope_table(64, device=DEV))
        assert torch.equal(one, c.pool)
    K.paged_append(c.cache, c.k[:0], c.v[:0], _i([0, 0, 0]))
    assert torch.equal(one, c.pool)
    shared = c.k[:, :1].expand(37, 3, 128)                   # one head for all
    K.paged_append(c.cache, shared, c.v, c.cu)
    one = c.pool.clone()
    K.paged_append(c.cache, shared.contiguous(), c.v, c.cu)
    assert torch.equal(one, c.pool)


def test_offsets_past_32_bits():
    """The last page of a pool of more than 2^32 bytes."""
    page, heads = 64, 32
    block = K.k3mla_paged_block_bytes("i4", page, 128, 128)
    pages = (1 << 32) // (block * heads) + 10
    pool = torch.empty((pages, heads, block), dtype=torch.uint8, device=DEV)
    pool[:4].zero_()
    cache = K.PagedCache(pool, _i([[pages - 1]]), _i([33]), page, 128, 128)
    k = torch.randn(5, heads, 128, device=DEV)
    v = torch.randn(5, heads, 128, device=DEV)
    K.paged_append(cache, k, v, _i([0, 5]))
    kr, vr = K.paged_read(cache, 5, _i([0, 5]), torch.float32)
    for x, y in ((k, kr), (v, vr)):
        code, s, m = PP.quantise(_np(x).reshape(5, heads, 2, 64))
        want = (code * s[..., None] + m[..., None]).reshape(5, heads, 128)
        assert (np.abs(_np(y) - want) <= 2.0 ** -24 * np.abs(want)).all()
    assert not pool[:4].any()


def test_append_in_a_graph_follows_the_lengths():
    c = Case([10, 70], [1, 1], 2, 128, 128, 16, "i4")
    table = K.rope_table(128, device=DEV)
    K.paged_append(c.cache, c.k, c.v, rope=table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.paged_append(c.cache, c.k, c.v, rope=table)
    want = [c.rows()]
    c.cache.kv_len.sub_(1)                                   # the same rows one token earlier
    g.replay()
    c.pos = c.pos - 1
    got = c.rows()
    code, s, m = PP.quantise(PP.rotate(_np(c.k), c.pos, 128).reshape(2, 2, 2, 64))
    assert np.array_equal(got[..., :128], (code * s[..., None] + m[..., None]).reshape(2, 2, 128))
    assert np.array_equal(got[..., 128:], want[0][..., 128:])
