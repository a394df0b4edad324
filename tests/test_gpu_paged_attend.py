"""Attention over the paged cache on the GPU against the 64-bit form, with every row that no token sees holding NaN."""
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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Case:
    """N sequences of `total` cached tokens, the last `new` of them new; pages in a shuffled order; whatever no
    token holds is 0xFF bytes: NaN in both formats."""

    def __init__(self, total, new, heads, group, dqk, dv, page, fmt, rope=(0, 0, "half"), dtype=torch.bfloat16, gate=False, seed=0,
                 edit=None):
        rng = np.random.default_rng(seed)
        self.total, self.new, self.heads, self.group, self.fmt, self.page = list(total), list(new), heads, group, fmt, page
        self.dqk, self.dv, self.rope = dqk, dv, rope
        need = [-(-t // page) for t in total]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.tab = np.full((len(total), max(need + [1])), -3, np.int32)
        pool = np.full((pages, heads, K.k3mla_paged_block_bytes(fmt, page, dqk, dv)), 0xFF, np.uint8)
        self.k, self.v, self.kabs, self.vabs, at = [], [], 0.0, 0.0, 0
        for n, t in enumerate(total):
            rows = rng.standard_normal((t, heads, dqk + dv)).astype(np.float32)
            rows[..., :dqk] += rng.standard_normal((1, heads, dqk)).astype(np.float32)
            rows = torch.from_numpy(rows).bfloat16().float().numpy()
            if edit:
                edit(n, rows)
            held = np.full((heads, need[n] * page, dqk + dv), np.nan)
            held[:, :t] = rows.transpose(1, 0, 2)
            self.tab[n, :need[n]] = order[at:at + need[n]]
            vals = np.zeros((t, heads, dqk + dv))
            for j in range(need[n]):
                block = (PP.strips_i4 if fmt == "i4" else PP.strips_bf16)(held[:, j * page:(j + 1) * page])
                pool[order[at + j]] = block
                live = min(page, t - j * page)
                vals[j * page:j * page + live] = PP.unpack(block, page, dqk + dv, fmt)[:, :live].transpose(1, 0, 2)
            at += need[n]
            self.k.append(vals[..., :dqk])
            self.v.append(vals[..., dqk:])
        T, Hq = sum(new), heads * group
        self.pool = torch.from_numpy(pool).to(DEV)
        self.cache = K.PagedCache(self.pool, _i(self.tab), _i(self.total), page, dqk, dv, fmt)
        self.q = torch.from_numpy(rng.standard_normal((T, Hq, dqk)).astype(np.float32)).to(dtype).to(DEV)
        self.gate = torch.from_numpy(rng.standard_normal((T, Hq, dv)).astype(np.float32)).to(dtype).to(DEV) if gate else None
        self.cu = _i(np.concatenate([[0], np.cumsum(new)]))
        self.single = all(c == 1 for c in new)
        self.scale = dqk ** -0.5

    def run(self, out_dtype=torch.float32, ws=None, **kw):
        table = K.rope_table(self.rope[0], offset=self.rope[1], layout=self.rope[2], device=DEV) if self.rope[0] else None
        return K.paged_attend(self.cache, self.q, None if self.single else self.cu, max([1] + self.new), table, self.scale, self.gate,
                              out_dtype=out_dtype, workspace=ws, **kw)

    def want(self, rows=None):
        """(values, bound on the error): see _bound."""
        out, tol, at = [], [], 0
        for n, (t, c) in enumerate(zip(self.total, self.new)):
            q = PP.rotate(_np(self.q[at:at + c]), np.arange(t - c, t), *self.rope)
            g = None if self.gate is None else _np(self.gate[at:at + c])
            seen = t - c + 1 + np.arange(c)
            out.append(PP.attend(q, self.k[n], self.v[n], seen, self.scale, g))
            tol.append(self._bound(n, q, c))
            at += c
        return np.concatenate(out), np.concatenate(tol)

    def _bound(self, n, q, c):
        """A score is a sum of products |q| |x| whose terms (4-bit: 15 scale + |minimum| for |x|) carry an
        error of 2^-20 of themselves (two 11-bit parts of q, the sums; bf16 pages: 2^-16, two 8-bit parts) and the
        rotation's 2 * 4.8e-7; an error d of the scores moves a weighted mean of v by at most 2 d max|v|; the weights' own
        split, exponentials and sums cost 2^-19 (2^-15) of max|v|."""
        def size(x):
            x = np.where(np.isfinite(x), x, 0.0)
            if self.fmt == "bf16" or not x.size:
                return np.abs(x)
            grp = x.reshape(x.shape[:2] + (-1, 64))
            return np.repeat(2 * np.abs(grp).max(-1) + (grp.max(-1) - grp.min(-1)), 64, -1).reshape(x.shape)
        ka, va = size(self.k[n]), size(self.v[n])
        if not ka.size:
            return np.zeros((c, self.heads * self.group, self.dv))
        # rotated rows of at most |x| + |y|: twice the largest entry covers it
        a = (np.abs(q).max(-1).reshape(c, self.heads, self.group) * (2 if self.rope[0] else 1)) * ka.max(0).sum(-1)[None, :, None]
        e = (2.0 ** -20 if self.fmt == "i4" else 2.0 ** -16) + (1e-6 if self.rope[0] else 0)
        b = (2 * self.scale * a * e + (2.0 ** -19 if self.fmt == "i4" else 2.0 ** -15)) * va.max((0, 2))[None, :, None]
        return np.repeat(b.reshape(c, -1, 1), self.dv, -1)


def _check(got, want, tol, out_dtype=torch.float32):
    tol = tol + (BF_HALF if out_dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(want)
    err = np.abs(_np(got) - want)
    assert got.dtype == out_dtype
    assert np.array_equal(np.isnan(_np(got)), np.isnan(want))
    assert (np.nan_to_num(err) <= np.nan_to_num(tol)).all(), f"{np.nanmax(err):.3e}, {np.nanmax(err - tol):.3e} over"


CASES = [  # total, new, heads, group, dqk, dv, page, rope, gate
    ([1], [1], 1, 1, 64, 64, 16, (0, 0, "half"), False),
    ([2], [1], 2, 1, 128, 128, 64, (128, 0, "half"), True),
    ([512], [1], 8, 4, 128, 128, 64, (128, 0, "half"), False),
    ([33, 1, 500, 64, 17], [1] * 5, 3, 1, 128, 128, 32, (0, 0, "half"), True),
    ([40, 7, 300], [3, 7, 2], 2, 2, 192, 128, 16, (64, 128, "interleaved"), True),
    ([0, 5, 0, 90], [0, 5, 0, 4], 2, 5, 64, 128, 48, (34, 5, "interleaved"), False),
    ([130, 31], [1, 1], 1, 16, 256, 256, 128, (48, 208, "half"), False),
    ([77, 200], [33, 1], 1, 3, 256, 64, 256, (0, 0, "half"), True),
    ([16, 15, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], [1] * 12, 1, 2, 64, 256, 16, (64, 0, "half"), False),
    ([90, 64], [90, 64], 2, 8, 128, 64, 64, (32, 16, "half"), True),
    ([1500], [1], 1, 40, 192, 256, 32, (0, 0, "half"), False)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_against_the_64_bit_form(case, fmt, dtype):
    total, new, heads, group, dqk, dv, page, rope, gate = case
    c = Case(total, new, heads, group, dqk, dv, page, fmt, rope, dtype, gate, seed=len(total) + page)
    want, tol = c.want()
    for out in (torch.float32, torch.bfloat16):
        _check(c.run(out), want, tol, out)


def _long(c):
    """The 64-bit form on the GPU, for lengths that numpy takes too long over."""
    outs, at = [], 0
    for n, (t, m) in enumerate(zip(c.total, c.new)):
        q = torch.from_numpy(PP.rotate(_np(c.q[at:at + m]), np.arange(t - m, t), *c.rope)).to(DEV)
        k, v = torch.from_numpy(c.k[n]).to(DEV), torch.from_numpy(c.v[n]).to(DEV)
        s = torch.einsum("chgd,lhd->hcgl", q.unflatten(1, (c.heads, c.group)), k) * c.scale
        hide = torch.arange(t, device=DEV)[None] > (t - m + torch.arange(m, device=DEV))[:, None]
        s = s.masked_fill(hide[None, :, None], -float("inf"))
        outs.append(torch.einsum("hcgl,lhd->chgd", torch.softmax(s, -1), v).flatten(1, 2))
        at += m
    return torch.cat(outs).cpu().numpy()


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("total,new,heads,group", [([70001], [1], 2, 4), ([9000, 3, 20000, 700, 1], [1] * 5, 3, 1),
                                                   ([5000, 4000], [70, 200], 2, 4), ([300 + 7 * i for i in range(90)], [1] * 90, 8, 1)], ids=str)
def test_long_and_ragged(fmt, total, new, heads, group):
    """Rows that many CTAs share, many sequences, prompts' chunks; twice with one workspace: the same bits."""
    c = Case(total, new, heads, group, 128, 128, 64, fmt, (128, 0, "half"), seed=3)
    tol = np.concatenate([c._bound(n, PP.rotate(_np(c.q[int(c.cu[n]):int(c.cu[n + 1])]), np.arange(t - m, t), *c.rope), m)
                          for n, (t, m) in enumerate(zip(total, new))])
    ws = K.paged_attend_workspace(c.cache, heads * group)
    got = c.run(ws=ws)
    _check(got, _long(c), tol)
    assert torch.equal(got, c.run(ws=ws))
    assert K.k3kda_workspace_status(ws) == 0
    assert not ws[256:4352].any()                            # the counters are as the next call needs them


def test_one_workspace_serves_calls_of_other_shapes():
    ws = None
    for i, (total, heads, group, dqk, dv, fmt) in enumerate([([30000], 1, 1, 128, 128, "i4"), ([2000, 9], 4, 8, 256, 256, "bf16"),
                                                             ([5, 4000, 77], 2, 2, 64, 64, "i4"), ([30000], 1, 1, 128, 128, "i4")]):
        c = Case(total, [1] * len(total), heads, group, dqk, dv, 32, fmt, seed=i)
        ws = torch.zeros(K.k3mla_paged_attend_workspace_size(8, 1, 256, 256), dtype=torch.uint8, device=DEV) if ws is None else ws
        tol = np.concatenate([c._bound(n, _np(c.q[n:n + 1]), 1) for n in range(len(total))])
        _check(c.run(ws=ws), _long(c), tol)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_rows_that_see_nothing_and_lengths_outside(fmt):
    """A row before position 0 and an empty sequence give 0; a length outside the table and a page outside the pool NaN for
    the rows that see them."""
    total, new = [3, 0, 40, 100, 50], [3, 0, 2, 5, 1]
    c = Case(total, new, 2, 2, 128, 128, 16, fmt, gate=True, seed=5)
    want, tol = c.want()
    c.cache.kv_len.copy_(_i([1, 0, -1, 100, 1000]))
    tab = c.tab.copy()
    tab[3, 6] = len(c.pool)                                  # tokens 96..111: seen by the last four of 95..99
    c.cache.block_table.copy_(_i(tab))
    got = _np(c.run())
    # sequence 0 now has 1 token for 3 new ones: two rows at positions -2 and -1, one that sees token 0
    assert (got[:2] == 0).all()
    g = 1 / (1 + np.exp(-_np(c.gate)))
    assert np.abs(got[2] - np.repeat(c.v[0][0], 2, 0) * g[2]).max() <= tol[2].max() + 2.0 ** -23 * np.abs(got[2]).max()
    assert np.isnan(got[3:5]).all() and np.isnan(got[10]).all()
    assert np.isnan(got[6:10]).all()
    assert (np.abs(got[5] - want[5]) <= tol[5] + 2.0 ** -23 * np.abs(want[5])).all()
    # an empty sequence with a row
    e = Case([0, 20], [0, 1], 1, 1, 64, 64, 16, fmt)
    one = K.paged_attend(K.PagedCache(e.pool, _i(e.tab), _i([0, 20]), 16, 64, 64, fmt), torch.cat([e.q, e.q]))
    assert (one[0] == 0).all() and torch.isfinite(one[1].float()).all()


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_cannot_reach_it(fmt, value):
    """Values and keys that are not finite in the last of five new tokens: the four rows before it are as without."""
    def spoil(n, rows):
        if n == 1:
            rows[-1, :, 128 + 70] = value
            rows[-1, 0, 3] = value
    args = ([200, 37], [1, 5], 2, 3, 128, 128, 16, fmt)
    clean, dirty = Case(*args, seed=8), Case(*args, seed=8, edit=spoil)
    a, b = clean.run(), dirty.run()
    assert torch.equal(a[:5], b[:5])
    # the last row is finite where the 64-bit form is (a key that scores -inf weighs nothing)
    assert np.array_equal(np.isfinite(_np(b[5])), np.isfinite(dirty.want()[0][5]))


def test_values_of_every_size():
    """Scales from fp16's denormals to its limit side by side, and scores far apart: the weights keep their accuracy."""
    def edit(n, rows):
        r = np.random.default_rng(9)
        rows[..., 128:] *= 10.0 ** r.integers(-5, 4, rows.shape[:2] + (1,))
        rows[..., :128] *= 6
    c = Case([3000, 50], [1, 1], 2, 2, 128, 128, 64, "i4", seed=10, edit=edit)
    tol = np.concatenate([c._bound(n, _np(c.q[n:n + 1]), 1) for n in range(2)])
    _check(c.run(), _long(c), tol)
    # all values tiny: errors stay relative to them
    c = Case([700], [1], 1, 1, 128, 128, 64, "i4", seed=11, edit=lambda n, rows: rows[..., 128:].__imul__(1e-4))
    _check(c.run(), _long(c), c._bound(0, _np(c.q), 1))
    # constant groups (scale 0) and a query of zeros
    c = Case([100], [1], 1, 2, 64, 64, 16, "i4", seed=12, edit=lambda n, rows: rows.__setitem__(Ellipsis, rows[..., :1]))
    c.q[0, 1] = 0
    _check(c.run(), _long(c), c._bound(0, _np(c.q), 1))


def test_strided_queries_other_stream_graph_and_no_tokens():
    c = Case([300, 20], [1, 1], 2, 2, 128, 128, 32, "i4", (64, 64, "half"), gate=True, seed=13)
    want = c.run()
    wide = torch.zeros(2, 4, 300, dtype=torch.bfloat16, device=DEV)
    wide[..., 3:131], wide[..., 140:268] = c.q, c.gate
    table = K.rope_table(64, offset=64, device=DEV)
    got = K.paged_attend(c.cache, wide[..., 3:131], rope=table, gate=wide[..., 140:268], out_dtype=torch.float32)
    assert torch.equal(got, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    assert K.paged_attend(c.cache, c.q[:0], _i([0, 0, 0])).shape == (0, 4, 128)
    ws, out = K.paged_attend_workspace(c.cache, 4), torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.paged_attend(c.cache, c.q, rope=table, gate=c.gate, out=out, workspace=ws)
    g.replay()
    assert torch.equal(out, want)
    c.cache.kv_len.copy_(_i([250, 3]))                       # the graph follows the lengths
    g.replay()
    c.total = [250, 3]
    c.k, c.v = [x[:t] for x, t in zip(c.k, c.total)], [x[:t] for x, t in zip(c.v, c.total)]
    _check(out, *c.want())


def test_append_then_attend_over_steps():
    """A prompt, then ten tokens one at a time, pages growing as they go: each step equals attention over the values read back."""
    torch.manual_seed(0)
    N, H, G, page, L = 3, 2, 2, 16, 60
    table = K.rope_table(64, offset=64, layout="interleaved", device=DEV)
    tab = torch.randperm(N * 4, device=DEV).to(torch.int32).view(N, 4)
    for fmt in ("i4", "bf16"):
        kv_len = _i([17, 30, 5])
        cache = K.PagedCache(K.paged_pool(N * 4, page, H, 128, 128, fmt, DEV), tab, kv_len, page, 128, 128, fmt)
        T = 52
        cu = _i([0, 17, 47, 52])
        rnd = lambda *s: torch.randn(s, device=DEV).bfloat16()
        K.paged_append(cache, rnd(T, H, 128), rnd(T, H, 128), cu, rope=table)
        ws = K.paged_attend_workspace(cache, H * G)
        for step in range(10):
            kv_len.add_(1)
            k, v, q = rnd(N, H, 128), rnd(N, H, 128), rnd(N, H * G, 128)
            K.paged_append(cache, k, v, rope=table)
            got = K.paged_attend(cache, q, rope=table, out_dtype=torch.float32, workspace=ws)
            lens = kv_len.tolist()
            kr, vr = K.paged_read(cache, sum(lens), _i(np.concatenate([[0], np.cumsum(lens)])), torch.float32)
            at = 0
            for n, t in enumerate(lens):
                qr = PP.rotate(_np(q[n:n + 1]), [t - 1], 64, 64, "interleaved")
                want = PP.attend(qr, _np(kr[at:at + t]), _np(vr[at:at + t]), [t], 128 ** -0.5)
                assert np.abs(_np(got[n]) - want[0]).max() <= (1e-4 if fmt == "i4" else 2e-3)
                at += t


# ---- blocks of 128 rows (more than 16 query rows of a key head) ------------------------------------------------

ROWS = [  # total, new, heads, group, dqk, dv, page, rope, gate
    ([64], [17], 1, 1, 64, 64, 16, (0, 0, "half"), False),
    ([200], [128], 1, 1, 128, 128, 64, (128, 0, "half"), True),
    ([129, 0, 300, 31], [129, 0, 40, 31], 2, 1, 192, 128, 32, (64, 128, "interleaved"), True),
    ([1, 65, 63, 64, 500], [1, 1, 1, 1, 1], 2, 20, 128, 64, 48, (32, 3, "half"), False),
    ([300, 5], [6, 5], 3, 8, 64, 128, 16, (34, 5, "interleaved"), True),
    ([77, 256, 257], [77, 3, 140], 1, 3, 192, 64, 256, (0, 0, "half"), False)]


@pytest.mark.parametrize("case", ROWS, ids=str)
@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_blocks_of_rows_against_the_64_bit_form(case, fmt, dtype):
    total, new, heads, group, dqk, dv, page, rope, gate = case
    c = Case(total, new, heads, group, dqk, dv, page, fmt, rope, dtype, gate, seed=sum(total))
    want, tol = c.want()
    for out in (torch.float32, torch.bfloat16):
        _check(c.run(out), want, tol, out)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_blocks_of_rows_that_many_ctas_share(fmt):
    """Few (sequence, head)s and long contexts: a block's tiles over many CTAs; the same bits each time; no counter left."""
    for total, new, heads, group in (([40000], [3], 1, 8), ([3000, 17, 9000], [40, 17, 1], 2, 17), ([900] * 30, [9] * 30, 4, 4)):
        c = Case(total, new, heads, group, 128, 128, 64, fmt, (64, 0, "interleaved"), seed=21)
        tol = np.concatenate([c._bound(n, PP.rotate(_np(c.q[int(c.cu[n]):int(c.cu[n + 1])]), np.arange(t - m, t), *c.rope), m)
                              for n, (t, m) in enumerate(zip(total, new))])
        ws = K.paged_attend_workspace(c.cache, heads * group)
        got = c.run(ws=ws)
        _check(got, _long(c), tol)
        for _ in range(3):
            assert torch.equal(got, c.run(ws=ws))
        assert K.k3kda_workspace_status(ws) == 0 and not ws[256:4352].any()


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_blocks_of_rows_what_a_row_does_not_see_cannot_reach_it(fmt, value):
    """A value that is not finite in the 11th of 20 new tokens: the tokens before it are as without, the others have it in
    the channels that hold it (4-bit: its group), and nowhere else."""
    def spoil(n, rows):
        if n == 1:
            rows[-10, 1, 128 + 70] = value
    args = ([200, 37], [1, 20], 2, 3, 128, 128, 16, fmt)
    clean, dirty = Case(*args, seed=8), Case(*args, seed=8, edit=spoil)
    a, b = clean.run(), dirty.run()
    assert torch.equal(a[:11], b[:11])
    gone = ~torch.isfinite(b[11:])
    assert not gone[:, :3].any()
    seen = torch.zeros(128, dtype=torch.bool, device=DEV)
    seen[64:128] = True
    if fmt == "bf16":
        seen[:] = False
        seen[70] = True
    assert torch.equal(gone[:, 3:], seen.expand(10, 3, 128))


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_blocks_of_rows_bad_pages_and_lengths(fmt):
    total, new = [30, 0, 40, 100, 50], [30, 0, 20, 25, 20]
    c = Case(total, new, 2, 2, 128, 128, 16, fmt, gate=True, seed=5)
    want, tol = c.want()
    c.cache.kv_len.copy_(_i([28, 0, -1, 100, 1000]))
    tab = c.tab.copy()
    tab[3, 5] = -1                                           # tokens 80..95: seen by tokens 80.. of 75..99
    c.cache.block_table.copy_(_i(tab))
    got = _np(c.run())
    assert (got[:2] == 0).all() and np.isfinite(got[2:30]).all()       # two rows before position 0
    assert np.isnan(got[30:50]).all() and np.isnan(got[75:]).all()
    assert (np.abs(got[50:55] - want[50:55]) <= tol[50:55] + 2.0 ** -23 * np.abs(want[50:55])).all()
    assert np.isnan(got[55:75]).all()


def test_blocks_of_rows_values_of_every_size():
    def edit(n, rows):
        r = np.random.default_rng(9)
        rows[..., 128:] *= 10.0 ** r.integers(-5, 4, rows.shape[:2] + (1,))
        rows[..., :128] *= 6
    c = Case([3000, 50], [9, 20], 2, 2, 128, 128, 64, "i4", seed=10, edit=edit)
    tol = np.concatenate([c._bound(n, _np(c.q[int(c.cu[n]):int(c.cu[n + 1])]), m) for n, m in enumerate(c.new)])
    _check(c.run(), _long(c), tol)
    c = Case([700], [40], 1, 1, 128, 128, 64, "i4", seed=11, edit=lambda n, rows: rows[..., 128:].__imul__(1e-4))
    _check(c.run(), _long(c), c._bound(0, _np(c.q), 40))


MORE_ROWS = [  # blocks of 128 rows for 4-bit pages too: more than 56 rows (32 beyond 128 key channels)
    ([64], [57], 1, 1, 64, 64, 16, (0, 0, "half"), False),
    ([63, 1, 200], [1, 1, 1], 2, 60, 128, 128, 48, (128, 0, "half"), True),
    ([300, 130], [16, 5], 2, 8, 64, 128, 16, (34, 5, "interleaved"), True),
    ([40, 257], [9, 3], 3, 13, 192, 64, 32, (64, 128, "half"), False),
    ([128, 129, 127], [128, 64, 127], 1, 1, 128, 64, 128, (32, 16, "interleaved"), False)]


@pytest.mark.parametrize("case", MORE_ROWS, ids=str)
@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_more_blocks_of_rows_against_the_64_bit_form(case, fmt):
    total, new, heads, group, dqk, dv, page, rope, gate = case
    c = Case(total, new, heads, group, dqk, dv, page, fmt, rope, torch.bfloat16, gate, seed=sum(new))
    want, tol = c.want()
    for out in (torch.float32, torch.bfloat16):
        _check(c.run(out), want, tol, out)


def test_more_blocks_of_rows_long_shared_and_of_every_size():
    def edit(n, rows):
        r = np.random.default_rng(9)
        rows[..., 128:] *= 10.0 ** r.integers(-5, 4, rows.shape[:2] + (1,))
        rows[..., :128] *= 6
    for total, new, heads, group, kw in (([30000], [8], 1, 8, {}), ([900] * 20, [10] * 20, 4, 6, {}), ([3000, 90], [9, 20], 2, 8, dict(edit=edit)),
                                         ([700], [80], 1, 1, dict(edit=lambda n, rows: rows[..., 128:].__imul__(1e-4)))):
        c = Case(total, new, heads, group, 128, 128, 64, "i4", seed=23, **kw)
        tol = np.concatenate([c._bound(n, _np(c.q[int(c.cu[n]):int(c.cu[n + 1])]), m) for n, m in enumerate(new)])
        ws = K.paged_attend_workspace(c.cache, heads * group)
        got = c.run(ws=ws)
        _check(got, _long(c), tol)
        assert torch.equal(got, c.run(ws=ws)) and not ws[256:4352].any()


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_32_bits(fmt, new):
    """The same pages at the end of a pool of more than 2^32 bytes: the same bits."""
    c = Case([300, 90], [new, new], 2, 2, 128, 128, 64, fmt, (128, 0, "half"), seed=31)
    small, own = c.run(), c.pool.shape[0]
    pages = (1 << 32) // c.pool[0].numel() + own + 1
    pool = torch.empty((pages,) + tuple(c.pool.shape[1:]), dtype=torch.uint8, device=DEV)
    pool[-own:] = c.pool
    c.cache = K.PagedCache(pool, _i(np.where(c.tab >= 0, c.tab + pages - own, c.tab)), _i(c.total), 64, 128, 128, fmt)
    assert torch.equal(c.run(), small)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new", [4, 20])
def test_a_key_that_is_not_finite_scores_as_its_product_does(fmt, value, new):
    """A bf16 key with an infinity scores plus or minus infinity by the sign of the query's channel, whatever parts the query
    is held in (some channels need only one): a row that it scores minus infinity is as without it."""
    def spoil(n, rows):
        if n == 1:
            rows[-2, 1, 3] = value
    c = Case([200, 37], [1, new], 2, 4, 128, 128, 16, fmt, seed=12, edit=spoil)
    c.q[:, :, 3] = torch.where(torch.arange(8, device=DEV) % 2 == 0, 0.5, -0.75).bfloat16()
    want, tol = c.want()
    got = _np(c.run())
    finite = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), finite)
    assert (np.abs(got - want)[finite] <= (tol + 2.0 ** -23 * np.abs(want))[finite]).all()
