"""The norms around a block on the GPU against the definition in 64 bits.

Tolerances: an output's own rounding (half a step of its type), and the FP32 arithmetic.  A norm's factor is a sum of D squares, all
of one sign: at most (log2 of the threads + 16) additions in a row, a square root and a division: 64 roundings of 2^-24 are more than that,
2^-18.  Act adds a few (BF16: the fast exponential, 2^-21 times the exponent's size of at most 8 here, and division), 2^-17 in all.  Gradients
subtract a mean of products from a product, so their bound is on the terms by size: |d| + |h| mean |d h|.  A weight's gradient is a
sum over rows: another rounding a row, over the terms by size."""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import lin_plain as P  # noqa: E402

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
A = 2.0 ** -17


def _half(t):
    return torch.finfo(t.dtype).eps / 2


def _near(got, want, M, arith, what):
    bound = _half(got) * want.abs() + arith * M
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= bound).all(), f"{what}: {(off / bound.clamp_min(1e-300)).max().item():.3g} times the bound"


def _case(rows, D, dtype, post=True, gate="sigmoid", residual=True, pre=True, seed=0, alpha=0.5):
    g = torch.Generator(DEV).manual_seed(seed + D)
    rand = lambda *s, dt=dtype: torch.randn(s, generator=g, device=DEV).to(dt)  # noqa: E731
    return dict(x=rand(rows, D), residual=rand(rows, D) if residual else None, gate=rand(rows, D) if gate else None, gate_act=gate or "sigmoid",
                post=1 + rand(D, dt=F32) / 4 if post else None, pre=1 + rand(D, dt=F32) / 4 if pre else None, alpha=alpha,
                ds=rand(rows, D), dy=rand(rows, D) if pre else None, sum=rand(rows, D) if pre else None)


def _forward(c, **kw):
    return K.block_norm(c["x"], c["residual"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"], **kw)


def _backward(c, **kw):
    return K.block_norm_backward(c["x"], c["ds"], c["dy"], c["sum"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"],
                                 residual=c["residual"] is not None, **kw)


def _check_forward(c, got):
    want, wy = P.block_norm(c["x"], c["residual"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"])
    s, y = got if isinstance(got, tuple) else (got, None)
    branch = want - (0 if c["residual"] is None else c["residual"].double())
    M = branch.abs() + (0 if c["residual"] is None else c["residual"].double().abs())
    _near(s, want, M, A, "s")
    assert (y is None) == (wy is None)
    if y is not None:
        scale = 1 / torch.sqrt((want * want).mean(-1, keepdim=True) + 1e-6)
        _near(y, wy, (M * scale + wy.abs()) * (c["pre"].double().abs() + 1), 2 * A, "y")


def _check_backward(c, d):
    want = P.block_norm_backward(c["x"], c["ds"], c["dy"], c["sum"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"])
    eps = 1e-6

    def terms(d, x, w):
        """The terms of a norm's gradient by size, and those of its weight's."""
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        h = (x * r).abs()
        return r * (d * w.abs() + h * (d * w.abs() * h).mean(-1, keepdim=True)), (d * h).sum(0)
    rows = c["x"].shape[0]
    M = c["ds"].double().abs()
    if c["pre"] is not None:
        more, mw = terms(c["dy"].double().abs(), c["sum"].double(), c["pre"].double())
        M = M + more
        _near(d["dpre"], want["dpre"], mw, A + (rows + 16) * 2.0 ** -24, "dpre")
    if c["residual"] is not None:
        _near(d["dresidual"], want["dresidual"], M, A, "dresidual")
    else:
        assert d["dresidual"] is None
    M, x = M * abs(c["alpha"]), c["x"].double()
    if c["gate"] is not None:
        z = c["gate"].double()
        u = x if c["post"] is None else P.unit(x, eps) * c["post"].double()
        # act' is a sum of terms no larger than 1 + |z| / 4
        _near(d["dgate"], want["dgate"], M * u.abs() * (1 + z.abs() / 4), 2 * A, "dgate")
        M = M * P.act(c["gate_act"], z).abs()
    if c["post"] is not None:
        M, mw = terms(M, x, c["post"].double())
        _near(d["dpost"], want["dpost"], mw, 2 * A + (rows + 16) * 2.0 ** -24, "dpost")
    _near(d["dx"], want["dx"], M, 3 * A, "dx")


#: both sides of every width at which another number of threads takes a row, odd ones, and the largest
WIDTHS = [1, 7, 8, 64, 127, 128, 129, 512, 513, 1111, 2048, 2049, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_widths(D, dtype):
    for rows in (1, 2, 37):
        c = _case(rows, D, dtype)
        _check_forward(c, _forward(c))
        _check_backward(c, _backward(c))


@pytest.mark.parametrize("D", [63, 65, 96, 97, 255, 257, 383, 385, 1025, 1535, 1537])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_widths_at_which_a_thread_holds_more(D, dtype):
    for rows in (1, 70):
        c = _case(rows, D, dtype, gate="silu", seed=8)
        _check_forward(c, _forward(c))
        _check_backward(c, _backward(c))


@pytest.mark.parametrize("post,gate,residual,pre", list(itertools.product([False, True], [None, "sigmoid", "silu"], [False, True], [False, True])))
@pytest.mark.parametrize("dtype,D", [(BF, 256), (F32, 130)], ids=["bf16", "f32"])
def test_parts(post, gate, residual, pre, dtype, D):
    c = _case(19, D, dtype, post, gate, residual, pre, seed=3, alpha=1.25)
    _check_forward(c, _forward(c))
    _check_backward(c, _backward(c))


@pytest.mark.parametrize("rows,D", [(5000, 128), (3001, 512), (700, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_rows(rows, D, dtype):
    c = _case(rows, D, dtype, gate="silu", seed=4)
    _check_forward(c, _forward(c))
    _check_backward(c, _backward(c))


def test_leading_dimensions_are_rows():
    c = _case(24, 64, BF, seed=5)
    flat = _forward(c)
    e = {k: v.view(4, 6, 64) if isinstance(v, torch.Tensor) and v.dim() == 2 else v for k, v in c.items()}
    assert all(torch.equal(a.view(24, 64), b) for a, b in zip(_forward(e), flat))


def test_arrays_off_sixteen_bytes():
    D, rows = 256, 9
    big = torch.randn(rows * D + 1, device=DEV).bfloat16()
    c = _case(rows, D, BF, seed=6)
    for name in ("x", "gate", "residual"):
        e = dict(c)
        e[name] = big[1:].view(rows, D)
        _check_forward(e, _forward(e))
        _check_backward(e, _backward(e))


def test_outputs_in_place():
    c = _case(50, 512, BF, seed=7)
    s, y = _forward(c)
    e = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    K.k3blk_norm(e["x"], e["residual"], e["gate"], "sigmoid", e["post"], e["pre"], 0.5, 1e-6, e["residual"], e["x"])
    assert torch.equal(e["residual"], s) and torch.equal(e["x"], y)
    d = _backward(c)
    e = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    dpost, dpre = torch.empty(512, device=DEV), torch.empty(512, device=DEV)
    K.k3blk_norm_backward(e["x"], e["ds"], e["dy"], e["sum"], e["gate"], "sigmoid", e["post"], e["pre"], 0.5, 1e-6, e["x"], e["ds"], e["gate"], dpost,
                          dpre, K.block_norm_workspace(50, 512))
    for a, b in ((e["x"], d["dx"]), (e["ds"], d["dresidual"]), (e["gate"], d["dgate"]), (dpost, d["dpost"]), (dpre, d["dpre"])):
        assert torch.equal(a, b)


def test_rows_of_zeros_and_rows_that_are_not_finite():
    c = _case(40, 1024, BF, seed=8)
    for name in ("x", "residual", "sum"):
        c[name][3] = 0
    _check_forward(c, _forward(c))
    _check_backward(c, _backward(c))
    ref, rd = _forward(c), _backward(c)
    c["x"][7, 11], c["gate"][8, 0] = float("nan"), float("nan")
    got, d = _forward(c), _backward(c)
    keep = torch.tensor([i for i in range(40) if i not in (7, 8)], device=DEV)
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, ref))
    assert all(torch.equal(d[x][keep], rd[x][keep]) for x in ("dx", "dgate", "dresidual"))
    assert torch.isnan(got[0][7]).all() and torch.isnan(got[1][8]).all() and torch.isnan(d["dgate"][8, 0])


def test_gates_far_from_zero():
    for dtype in (BF, F32):
        c = _case(8, 256, dtype, seed=9)
        c["gate"] = (torch.linspace(-200, 200, 2048, device=DEV).view(8, 256)).to(dtype)
        for kind in ("sigmoid", "silu"):
            c["gate_act"] = kind
            s, y = _forward(c)
            want, _ = P.block_norm(c["x"], c["residual"], c["gate"], kind, c["post"], None, 0.5)
            # the exponential of z is off by 2^-21 |z| where it counts, and gone where it does not
            _near(s, want, (want - c["residual"].double()).abs() + c["residual"].double().abs(), A + 200 * 2.0 ** -21, kind)
            assert all(torch.isfinite(x).all() for x in _backward(c).values())


def test_no_rows():
    c = _case(0, 64, BF)
    s, y = _forward(c)
    assert s.shape == y.shape == (0, 64)
    d = _backward(c)
    assert (d["dpost"] == 0).all() and (d["dpre"] == 0).all()


def test_results_do_not_change_and_can_be_captured():
    c = _case(2000, 512, BF, seed=10)
    ws = K.block_norm_workspace(2000, 512)
    want = [*_forward(c), *_backward(c).values()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = [*_forward(c), *_backward(c, workspace=ws).values()]
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_another_stream():
    c = _case(300, 2048, BF, seed=11)
    want = [*_forward(c), *_backward(c).values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20_000_000)
        got = [*_forward(c, stream=s), *_backward(c, stream=s).values()]
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_against_differences():
    """s is linear in the residual, alpha u in post: any step gives the derivative.  For x and the gate the step's square remains: for a
    step of size h in every element, h^2 / 6 times a third derivative that is below 60 times the sum of the loss's terms by size for values of
    size 1 (checked with x and gate of at least 1/4 root mean square)."""
    c = _case(5, 96, F32, seed=12, pre=False)
    w = c["ds"].double()
    d = _backward(c)
    loss = lambda **kw: (_forward({**c, **kw}).double() * w).sum().item()  # noqa: E731
    want, _ = P.block_norm(c["x"], None, c["gate"], "sigmoid", c["post"], None, 0.5)
    size = ((want.abs() + c["residual"].double().abs() + 4) * w.abs()).sum().item()
    gen = torch.Generator(DEV).manual_seed(1)
    for name, grad in (("residual", "dresidual"), ("post", "dpost")):
        step = torch.randn(c[name].shape, generator=gen, device=DEV).clamp(-4, 4)
        got = (loss(**{name: c[name] + step}) - loss(**{name: c[name] - step})) / 2
        assert abs(got - (d[grad].double() * step).sum().item()) <= 4 * A * size, name
    h = 2.0 ** -5
    for name, grad in (("x", "dx"), ("gate", "dgate")):
        step = torch.rand(c[name].shape, generator=gen, device=DEV) * 2 - 1
        got = (loss(**{name: c[name] + h * step}) - loss(**{name: c[name] - h * step})) / (2 * h)
        assert abs(got - (d[grad].double() * step).sum().item()) <= (2 * A / h + 10 * h * h) * size, name


def _check_with_eps(c, eps):
    """Forward and gradients for another eps: the bounds above, with it in the norms' factors."""
    half = _half(c["x"])
    x, res, post, pre = (c[n].double() for n in ("x", "residual", "post", "pre"))
    args = (c["x"], c["residual"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"])
    s, y = K.block_norm(*args, eps=eps)
    want, wy = P.block_norm(*args, eps)
    M = (want - res).abs() + res.abs()
    _near(s, want, M, A, "s")
    _near(y, wy, (M / torch.sqrt((want * want).mean(-1, keepdim=True) + eps) + wy.abs()) * (pre.abs() + 1), 2 * A, "y")
    d = K.block_norm_backward(c["x"], c["ds"], c["dy"], c["sum"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"], eps)
    w = P.block_norm_backward(c["x"], c["ds"], c["dy"], c["sum"], c["gate"], c["gate_act"], c["post"], c["pre"], c["alpha"], eps)
    rows = x.shape[0]

    def terms(d, x, weight):
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        h = (x * r).abs()
        return r * (d * weight.abs() + h * (d * weight.abs() * h).mean(-1, keepdim=True)), (d * h).sum(0)
    more, mw = terms(c["dy"].double().abs(), c["sum"].double(), pre)
    M = c["ds"].double().abs() + more
    _near(d["dpre"], w["dpre"], mw, A + (rows + 16) * 2.0 ** -24, "dpre")
    _near(d["dresidual"], w["dresidual"], M, A, "dresidual")
    M, z = M * abs(c["alpha"]), c["gate"].double()
    _near(d["dgate"], w["dgate"], M * (P.unit(x, eps) * post).abs() * (1 + z.abs() / 4), 2 * A, "dgate")
    M, mw = terms(M * P.act(c["gate_act"], z).abs(), x, post)
    _near(d["dpost"], w["dpost"], mw, 2 * A + (rows + 16) * 2.0 ** -24, "dpost")
    _near(d["dx"], w["dx"], M, 3 * A, "dx")


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -10, 4.0])
@pytest.mark.parametrize("D", [8, 64, 512, 768, 1024, 1111, 2048, 2560, 16384])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_other_eps(D, eps, dtype):
    """With an eps of 0 as well, rows that a CTA's last round does not have add nothing to the weights' gradients."""
    for rows in (1, 3, 37, 70):
        _check_with_eps(_case(rows, D, dtype, seed=13), eps)


@pytest.mark.parametrize("which", ["x", "gate", "residual", "post", "pre"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_differences_along_the_gradient(which, act):
    """The loss moves by the sum of the gradient's sizes along its signs, many times what the arithmetic may be off by.  The definition's own
    difference at the same step takes out what the step's square adds."""
    c = _case(5, 96, F32, gate=act, seed=14)
    c["sum"], _ = _forward(c)
    names = {"x": "dx", "gate": "dgate", "residual": "dresidual", "post": "dpost", "pre": "dpre"}
    d = _backward(c)[names[which]].double()
    plain_of = lambda c: P.block_norm(c["x"], c["residual"], c["gate"], act, c["post"], c["pre"], 0.5)  # noqa: E731
    s64, _ = plain_of(c)
    formula = P.block_norm_backward(c["x"], c["ds"], c["dy"], s64, c["gate"], act, c["post"], c["pre"], 0.5)[names[which]]
    h = 2.0 ** -3
    step = (h * torch.sign(formula)).float()
    ds, dy = c["ds"].double(), c["dy"].double()

    def losses(sign):
        """(of the kernels, of the definition, by size) with the input moved"""
        e = {**c, which: c[which] + sign * step}
        s, y = _forward(e)
        ps, py = plain_of(e)
        M = (ps - e["residual"].double()).abs() + e["residual"].double().abs()
        My = (M / torch.sqrt((ps * ps).mean(-1, keepdim=True) + 1e-6) + py.abs()) * (e["pre"].double().abs() + 1)
        return torch.stack([(s.double() * ds).sum() + (y.double() * dy).sum(), (ps * ds).sum() + (py * dy).sum(),
                            A * (M * ds.abs()).sum() + 2 * A * (My * dy.abs()).sum()])
    up, down = losses(1), losses(-1)
    got, plain = ((up - down) / 2)[:2]
    want, exact = (d * step).sum(), (formula * step).sum()
    bound = (up + down)[2] / 2 + exact / 100                         # (the gradient's own error: tested against the formula above)
    assert bound < exact / 20, (bound / exact).item()
    assert abs((got - plain) - (want - exact)) <= bound
    assert abs(got - want) <= bound + abs(plain - exact)
