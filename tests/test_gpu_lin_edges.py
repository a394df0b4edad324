"""Linear attention with a decay a head where its calls meet their limits: inputs that share memory, scales far from one, sums of
decays beyond 64 bits, values that are not finite and the decays' gradient, the bits that are promised.  Bounds are those of test_gpu_lin.py."""
import functools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import lin_plain as P  # noqa: E402
import test_gpu_lin as L  # noqa: E402

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("hk", [2, 4])
def test_inputs_of_other_widths_in_one_place(hk):
    """q, k and v may lie in one another: views of the same memory with other widths and heads."""
    T, h = 200, 4
    gen = torch.Generator(DEV).manual_seed(61)
    buf, do = (torch.randn(T * h * 128, generator=gen, device=DEV).bfloat16() for _ in range(2))
    g = -torch.rand((T, h), generator=gen, device=DEV)
    small, wide = buf[:T * hk * 64].view(T, hk, 64), buf.view(T, h, 128)
    first = torch.randn((1, h, 64, 128), generator=gen, device=DEV)
    for views, grad in (((small, small, wide), do.view(T, h, 128)), ((small, small, wide), wide)):
        apart = [x.clone() for x in views]
        a, b = K.lin_prefill(*views, g, first), K.lin_prefill(*apart, g, first)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        for need in (True, False):
            a, b = K.lin_backward(*views, g, grad, first, need_dg=need), K.lin_backward(*apart, g, grad.clone(), first, need_dg=need)
            assert all(torch.equal(a[x], b[x]) for x in b if b[x] is not None)


@pytest.mark.parametrize("scale", [2.0 ** 40, -2.0 ** 33, 2.0 ** -40])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scales_far_from_one(scale, dtype):
    """Decays of up to 2^-99 a chunk times a scale leave FP32's range in a factor, not in any result."""
    c = L._case([200], 2, 2, 64, 64, dtype, seed=62)
    c["g"].fill_(-1.07)
    c["scale"] = scale
    a = [c[x] for x in "qkvg"]
    out, last = K.lin_prefill(*a, c["first"], scale=scale, out_dtype=F32)
    want, wlast = P.prefill(*a, None, c["first"], scale)
    M, Ml = P.prefill(*(c[x].abs() for x in "qkv"), c["g"], None, c["first"].abs(), abs(scale))
    L._near(out, want, M, L._arith(dtype, 200, True), "out")
    L._near(last, wlast, Ml, L._arith(dtype, 200, True), "state")
    for need in (True, False):
        d = K.lin_backward(*a, c["do"], c["first"], c["dlast"], scale=scale, need_dg=need)
        w = P.backward(*a, c["do"], None, c["first"], c["dlast"], scale)
        M = P.backward(*(c[x].abs() for x in "qkv"), c["g"], c["do"].abs(), None, c["first"].abs(), c["dlast"].abs(), abs(scale))
        for x in ("dq", "dk", "dv"):
            L._near(d[x], w[x], M[x], L._arith(dtype, 200), x)
        L._near(d["dS0"], w["dS0"], M["dS0"], L._arith(dtype, 200, True), "dS0")
        if need:
            L._near(d["dg"], w["dg"], M["each"].flip(0).cumsum(0).flip(0) + M["dg_token"], L._arith(dtype, 200, True), "dg")


def _after_resets(T, N, dtype):
    """One sequence of T tokens, each a reset, among N - 1 empty ones: out_t = scale (q_t . k_t) v_t, whatever came before."""
    gen = torch.Generator(DEV).manual_seed(60)
    block = 1 << 16
    rows = [torch.randn((block, 1, 16), generator=gen, device=DEV).to(dtype) for _ in range(3)]
    q, k, v = (x.repeat((T + block - 1) // block, 1, 1)[:T] for x in rows)
    cu = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    cu[N // 2 + 1:] = T
    out, last = K.lin_prefill(q, k, v, torch.full((T, 1), -float("inf"), device=DEV), None, cu)
    p = 0.25 * (rows[0].double() * rows[1].double())
    want, M = p.sum(-1, keepdim=True) * rows[2].double(), p.abs().sum(-1, keepdim=True) * rows[2].double().abs()
    for t in range(0, T, block):
        n = min(block, T - t)
        L._near(out[t:t + n], want[:n], M[:n], L._arith(dtype, 1), f"from token {t}")
    t = (T - 1) % block
    L._near(last[N // 2, 0], rows[1][t, 0].double()[:, None] * rows[2][t, 0].double(), torch.ones(16, 16, device=DEV, dtype=torch.float64),
            L._arith(dtype, 1, True) * 32, "state")


def test_pieces_of_so_many_resets_that_64_bits_would_not_hold_their_sum():
    """A reset counts as 4,096 powers of two in units of 2^-32 of one: 2^19 of them are 2^63.  Three pieces of one sequence in FP32; 152 of one in
    BF16."""
    _after_resets(3 * (2 ** 19 + 64), 100, F32)
    _after_resets(152 * (2 ** 19 + 128), 1, BF)


def _backward_raw(c, dS0):
    """k3lin_backward, with or without room for the first state's gradient: dg."""
    q, k, v, g = (c[x] for x in "qkvg")
    T, hk, dk = q.shape
    N = 1 if c["cu"] is None else c["cu"].numel() - 1
    dg = torch.empty_like(g)
    K.k3lin_backward(q, k, v, g, c["do"], c["first"], c["dlast"], c["cu"], c["scale"], torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), dg,
                     torch.empty((N, v.shape[1], dk, v.shape[2]), device=DEV) if dS0 else None,
                     K.lin_backward_workspace(N, T, hk, v.shape[1], dk, v.shape[2], q.dtype))
    return dg


@functools.lru_cache(None)
def _poison_case(dtype, states):
    """A case, its dg and the bound on it; sums over a stretch of 512 tokens, from its end or from its beginning."""
    lens, h = [130, 1300, 70], 3
    c = L._case(lens, h, h, 48, 32, dtype, first=True, seed=63, decay=0.2)
    if states != "both":
        c["dlast"] = None
    if states == "none":
        c["first"] = None
    size = lambda x: None if x is None else x.abs()  # noqa: E731
    want = P.backward(*(c[x] for x in ("q", "k", "v", "g", "do")), c["cu"], c["first"], c["dlast"], c["scale"])["dg"]
    M = P.backward(*(c[x].abs() for x in "qkv"), c["g"], c["do"].abs(), c["cu"], size(c["first"]), size(c["dlast"]), c["scale"])
    reach = M["dg_token"].clone()
    for a, b in P.sequences(c["cu"], sum(lens)):
        for s in range(a, b, 512):
            e = min(s + 512, b)
            reach[s:e] += M["each"][s:e].sum(0) + M["dg_token"][[s, e - 1]].sum(0)
    return c, want, 2.0 ** -24 * want.abs() + L._arith(dtype, 1300, True) * reach + 2.0 ** -96


@pytest.mark.parametrize("at", [0, 300, 511, 512, 1299])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("dtype,states", [(BF, "both"), (F32, "both"), (BF, "first"), (F32, "none"), (BF, "none")],
                         ids=lambda x: x if isinstance(x, str) else str(x)[6:])
def test_the_decays_gradient_is_finite_where_what_is_not_does_not_reach(dtype, states, which, at):
    """dg_t is of the pairs of a token (or the first state) before t with a token (or the last state's gradient) from t on: a key or value
    at s is in none of those with t <= s, a query or an output's gradient at u in none with t > u."""
    c, want, bound = _poison_case(dtype, states)
    a, b, _ = (int(x) for x in c["cu"][1:])
    token, head = a + at, 1
    clean = torch.ones_like(c["g"], dtype=torch.bool)
    if which in "kv":
        clean[token + 1:b, head] = False
        none = slice(token + 1, b)
    else:
        clean[a:token + 1, head] = False
        none = slice(a + (states == "none"), token + 1)             # (nothing comes before the first token: 0, or not a number)
    for value in (float("nan"), float("inf")):
        e = dict(c)
        e[which] = c[which].clone()
        e[which][token, head, 5] = value
        for dS0 in (True, False):
            dg = _backward_raw(e, dS0)
            off = (dg.double() - want).abs()
            assert torch.isfinite(dg[clean]).all()
            assert (off <= bound)[clean].all(), (off / bound)[clean].max().item()
            assert not torch.isfinite(dg[none, head]).any()


def _ints(most, *shape, seed=0):
    return torch.randint(-most, most + 1, shape, generator=torch.Generator().manual_seed(seed)).float().to(DEV)


def _one_hot(T, h, d, seed):
    """Rows with one channel of 1 or -1."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.zeros((T, h, d))
    return x.scatter_(2, torch.randint(0, d, (T, h, 1), generator=gen), torch.randint(0, 2, (T, h, 1), generator=gen) * 2.0 - 1).to(DEV)


def _two_parts(x):
    """What two BF16 numbers hold of x."""
    high = x.bfloat16().double()
    return high + (x - high).bfloat16().double()


def _only(x, tokens):
    y = torch.zeros_like(x)
    y[tokens] = x[tokens]
    return y


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_outputs_in_fp32_hold_24_bits(dtype):
    """Whole numbers whose sums stay below 2^22 by size are exact in FP32 in any order, so nothing but an operand in fewer bits can change a
    result.  States of up to 22 bits under queries that pick one entry; scores of up to 20 bits on values that pick one."""
    T, h, d = 700, 2, 16
    g = torch.zeros((T, h), device=DEV)
    some = torch.arange(0, T, 28, device=DEV)                        # 25 tokens of 255 * 127 and a state of 2^21: below 2^22 in all
    k, v = _only(_ints(255, T, h, d, seed=1), some), _only(_ints(127, T, h, d, seed=2), some)
    first = _ints(2 ** 21 - 1, 1, h, d, d, seed=3)
    for q, k, v, first in ((_one_hot(T, h, d, 4), k, v, first),
                           (_ints(255, T, h, d, seed=5).abs(), _ints(255, T, h, d, seed=6).abs(), _only(_one_hot(T, h, d, 7), [3, 70, 500]), None)):
        q, k, v = (x.to(dtype) for x in (q, k, v))
        want, wlast = P.prefill(q, k, v, g, None, first, 1.0)
        M, Ml = P.prefill(q.abs(), k.abs(), v.abs(), g, None, None if first is None else first.abs(), 1.0)
        assert max(M.max(), Ml.max()) < 2 ** 22 and (_two_parts(want) != want).any()
        out, last = K.lin_prefill(q, k, v, g, first, scale=1.0, out_dtype=F32)
        assert torch.equal(out.double(), want) and torch.equal(last.double(), wlast)


@pytest.mark.parametrize("T", [2, 64, 65, 500])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_states_hold_24_bits(dtype, T):
    """One token's key under a decay that comes after it: the exponential is off by less than 2^-20, its product with the key and the sum of its three
    parts by 2^-22.  (Two parts leave up to 2^-17.)"""
    h, d = 4, 128
    q, k, v = (_only(x, [0]).to(dtype) for x in (_ints(255, T, h, d, seed=8), _ints(255, T, h, d, seed=9), torch.ones((T, h, d), device=DEV)))
    g = torch.zeros((T, h), device=DEV)
    g[T - 1] = torch.tensor([-0.3, -1.1, -0.71, -2.9], device=DEV)
    out, last = K.lin_prefill(q, k, v, g, scale=1.0)
    _, want = P.prefill(q, k, v, g, None, None, 1.0)
    assert ((last.double() - want).abs() <= (2.0 ** -20 + 2.0 ** -22) * want.abs()).all()
    d = K.lin_backward(k, q, v, g, v, scale=1 / 3, need_dg=False)    # R = scale k v^T, exact but for the product with the scale
    want = P.backward(k, q, v, g, v, None, None, None, torch.tensor(1 / 3).double())["dS0"]
    assert ((d["dS0"].double() - want).abs() <= (2.0 ** -20 + 2.0 ** -22) * want.abs()).all() and want.abs().max() > 10


@pytest.mark.parametrize("case", ["scores of dq", "scores of dv", "first state", "last state's gradient"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_the_decays_gradient_holds_24_bits(dtype, case):
    """Whole numbers as above: two queries after two keys, four pairs of 2^20, or seven that pick a state's entries of 2^19."""
    T, h, d = 700, 2, 16
    early, late = ([3, 66], [70, 90]) if "scores" in case else (list(range(0, 60, 9)), list(range(80, 600, 80)))
    wide, pick = lambda s: _ints(255, T, h, d, seed=s).abs(), torch.zeros((T, h, d), device=DEV)  # noqa: E731
    pick[:, :, 0] = 1
    c = {x: pick if "scores" in case else _one_hot(T, h, d, 16 + i) for i, x in enumerate(("q", "k", "v", "do"))}
    if case == "scores of dq":
        c.update(v=wide(10), do=wide(11))
    if case == "scores of dv":
        c.update(q=wide(12), k=wide(13))
    c = {x: _only(y, early if x in "kv" else late).to(dtype) for x, y in c.items()}
    first = _ints(2 ** 19 - 1, 1, h, d, d, seed=14) if case == "first state" else None
    last = _ints(2 ** 19 - 1, 1, h, d, d, seed=15) if case == "last state's gradient" else None
    g = torch.zeros((T, h), device=DEV)
    want = P.backward(c["q"], c["k"], c["v"], g, c["do"], None, first, last, 1.0)["dg"]
    assert want.abs().max() < 2 ** 22 and (_two_parts(want) != want).any()
    dg = K.lin_backward(c["q"], c["k"], c["v"], g, c["do"], first, last, scale=1.0)["dg"]
    assert torch.equal(dg.double(), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("which", ["q", "k", "v", "first", "g 8", "g 30", "g 40"])
def test_differences_along_the_gradient(which, dtype):
    """The loss moves by the sum of the gradient's sizes along its signs: many times what the arithmetic may be off by, so that a gradient that
    is 0, of the other sign or partly lost shows.  For g one token of each sequence moves and all inputs are positive, so that sums are not
    small beside their terms; the definition's own difference takes the step's square out.  Inputs are multiples of 1/16 below 4 and steps of
    1/2, which BF16 holds."""
    which, _, token = which.partition(" ")
    c = L._case([90, 41], 2, 4, 64, 48, dtype, seed=64)
    for x in ("q", "k", "v", "do"):
        c[x] = (c[x].float().clamp(-3, 3) * 16).round().div(16).to(dtype)
    if which == "g":
        c.update({x: y.abs() for x, y in c.items() if x in ("q", "k", "v", "do", "first", "dlast")})
    names = {"q": "dq", "k": "dk", "v": "dv", "first": "dS0", "g": "dg"}
    args = lambda c: (c["q"], c["k"], c["v"], c["g"])  # noqa: E731
    size = {x: y if x == "g" else y.abs() for x, y in c.items() if isinstance(y, torch.Tensor) and x != "cu"}
    d = K.lin_backward(*args(c), c["do"], c["first"], c["dlast"], c["cu"])[names[which]].double()
    formula = P.backward(*args(c), c["do"], c["cu"], c["first"], c["dlast"], c["scale"])[names[which]]
    G = P.backward(*args(size), size["do"], c["cu"], size["first"], size["dlast"], c["scale"])
    if which == "g":
        G["dg"] = G["each"].flip(0).cumsum(0).flip(0) + G["dg_token"]
    step = torch.sign(formula) / 2
    if which == "g":
        at = [int(token), 90 + int(token)]
        step = _only(step, at)
    w, dl = c["do"].double(), c["dlast"].double()

    def losses(sign):
        """(of the kernels, of the definition, by size) with the input moved"""
        e = {**c, which: (c[which].double() + sign * step).to(c[which].dtype)}
        o, s = K.lin_prefill(*args(e), e["first"], e["cu"], out_dtype=F32)
        po, ps = P.prefill(*args(e), e["cu"], e["first"], e["scale"])
        m = {x: y if x == "g" else y.abs() for x, y in e.items() if isinstance(y, torch.Tensor) and x != "cu"}
        mo, ms = P.prefill(*args(m), e["cu"], m["first"], e["scale"])
        return torch.stack([(a.double() * ww).sum() + (b.double() * wl).sum() for a, b, ww, wl in ((o, s, w, dl), (po, ps, w, dl),
                                                                                                 (mo, ms, w.abs(), dl.abs()))])
    up, down = losses(1), losses(-1)
    got, plain = ((up - down) / 2)[:2]
    want, exact = (d * step).sum(), (formula * step).sum()
    arith = L._arith(dtype, 90, which in ("g", "first"))
    grad = (step.abs() * ((0 if which in ("g", "first") else L._half(dtype)) * formula.abs() + arith * G[names[which]])).sum()
    bound = (L._arith(F32, 90) + 2.0 ** -24) * (up + down)[2] / 2 + grad
    assert bound < exact / 20, (bound / exact).item()
    assert abs((got - plain) - (want - exact)) <= bound
    assert abs(want - exact) <= grad


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("hk", [2, 4])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_of_a_padded_batch(dtype, hk, fixed):
    """Rows behind the last sequence: what they hold reaches nothing, and what is there of the outputs stays."""
    lens, T, h, dk, dv = [600, 0, 31], 700, 4, 64, 48
    c = L._case([T], hk, h, dk, dv, dtype, first=False, fixed=fixed, seed=65)
    N, n = len(lens), sum(lens)
    gen = torch.Generator(DEV).manual_seed(66)
    first, dlast = (torch.randn((N, h, dk, dv), generator=gen, device=DEV) for _ in range(2))
    cu = L._cu(lens).to(DEV)
    rows = [c[x] if x == "g" and fixed else c[x][:n] for x in ("q", "k", "v", "g", "do")]
    want = K.lin_backward(*rows, first, dlast, cu)
    for x in ("q", "k", "v", "do") + (() if fixed else ("g",)):
        c[x][n:] = float("nan")
    out = {x: torch.full_like(c[y], 7) for x, y in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    dS0 = torch.empty_like(first)
    K.k3lin_backward(c["q"], c["k"], c["v"], c["g"], c["do"], first, dlast, cu, dk ** -0.5, out["dq"], out["dk"], out["dv"], out["dg"], dS0,
                     K.lin_backward_workspace(N, T, hk, h, dk, dv, dtype))
    # (as pieces go by T, sums may be cut otherwise than without the rows)
    M = P.backward(*(x if x is rows[3] else x.abs() for x in rows), cu, first.abs(), dlast.abs(), dk ** -0.5)
    for x in ("dq", "dk", "dv"):
        assert (out[x][n:] == 7).all()
        L._near(out[x][:n], want[x].double(), M[x], L._half(dtype) + 2 * L._arith(dtype, 600), x)
    L._near(dS0, want["dS0"].double(), M["dS0"], 2 * L._arith(dtype, 600, True), "dS0")
    reach = (M["each"].flip(0).cumsum(0).flip(0) + (M["dg_token"] if not fixed else M["each"].sum(0) + M["dg_token"]))
    if fixed:
        L._near(out["dg"], want["dg"].double(), reach.sum(0), 2 * L._arith(dtype, 600, True), "dg")
    else:
        assert (out["dg"][n:] == 7).all()
        L._near(out["dg"][:n], want["dg"].double(), reach, 2 * L._arith(dtype, 600, True), "dg")


@pytest.mark.parametrize("lens,h", [([37], 2), ([500, 0, 1, 900], 4), ([64] * 40, 4), ([3000], 2)], ids=["short", "mixed", "many", "long"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_workspace_holds_nothing_that_matters(lens, h, dtype):
    """All of it but the status word may hold anything, such as what calls of other shapes left."""
    c = L._case(lens, h // 2, h, 64, 48, dtype, seed=67)
    a = [c[x] for x in "qkvg"]
    size = (len(lens), sum(lens), h // 2, h, 64, 48, dtype)

    def filled(make, byte):
        w = make(*size)
        w[256:] = byte
        return w
    want = [*K.lin_prefill(*a, c["first"], c["cu"])]
    for need in (True, False):
        want += [x for x in K.lin_backward(*a, c["do"], c["first"], c["dlast"], c["cu"], need_dg=need).values() if x is not None]
    for byte in (255, 127):
        got = [*K.lin_prefill(*a, c["first"], c["cu"], workspace=filled(K.lin_prefill_workspace, byte))]
        for need in (True, False):
            got += [x for x in K.lin_backward(*a, c["do"], c["first"], c["dlast"], c["cu"], need_dg=need,
                                              workspace=filled(K.lin_backward_workspace, byte)).values() if x is not None]
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_calls_on_two_streams_at_once():
    cases = [L._case([700, 300], 2, 4, 128, 128, BF, seed=68), L._case([1200], 4, 4, 64, 96, BF, seed=69)]

    def run(c, **kw):
        a = [c[x] for x in "qkvg"]
        return [*K.lin_prefill(*a, c["first"], c["cu"], **kw), *K.lin_backward(*a, c["do"], c["first"], c["dlast"], c["cu"], **kw).values()]
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(run(cases[i], stream=s))
    torch.cuda.synchronize()
    for w, rounds in zip(want, got):
        assert all(torch.equal(x, y) for r in rounds for x, y in zip(w, r))
