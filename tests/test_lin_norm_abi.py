"""Refusals of linear attention's and the block norms' calls, and the plain forms that the kernels are tested against (no GPU: every
call returns from its argument checks)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hybrid_linear_attention_rule_gb300 as K
import lin_plain as P

A256, MIS4, MIS1 = 0x10000, 0x10004, 0x10001              # never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


def _host(*x):
    return (ctypes.c_int32 * len(x))(*x)


def _prefill(lib, **kw):
    a = dict(q=A256, k=A256, v=A256, dtype=1, g=A256, fixed=0, first=A256, idx=None, idx_h=None, slots=2, cu=A256, cu_h=None, N=2, T=10, Hk=2,
             H=4, dk=64, dv=64, scale=1.0, out=A256, odt=1, last=A256, ws=A256, size=None)
    a.update(kw)
    size = a["size"] if a["size"] is not None else max(1 << 20, lib.k3lin_prefill_workspace_size(a["N"], a["T"], a["Hk"], a["H"], a["dk"], a["dv"], a["dtype"]))
    return lib.k3lin_prefill(a["q"], a["k"], a["v"], a["dtype"], a["g"], a["fixed"], a["first"], a["idx"], a["idx_h"], a["slots"], a["cu"], a["cu_h"],
                             a["N"], a["T"], a["Hk"], a["H"], a["dk"], a["dv"], a["scale"], a["out"], a["odt"], a["last"], a["ws"], size, None)


def test_prefill_refusals(lib):
    for bad in (dict(dtype=2), dict(odt=-1), dict(scale=NAN), dict(scale=INF), dict(N=0), dict(T=-1), dict(Hk=0), dict(H=0), dict(H=3),
                dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(out=None), dict(cu=None), dict(cu_h=_host(0, 5, 9)),
                dict(cu_h=_host(1, 5, 10)), dict(cu_h=_host(0, 11, 10)), dict(idx=A256, slots=0), dict(idx_h=_host(0, 1)),
                dict(idx=A256, idx_h=_host(0, 2)), dict(idx=A256, idx_h=_host(1, 1)), dict(idx=A256, idx_h=_host(-1, 1))):
        assert _prefill(lib, **bad) == -1, bad
    for bad in (dict(dk=8), dict(dk=24), dict(dk=144), dict(dv=0), dict(dv=256), dict(H=70000, Hk=1), dict(N=1 << 14, H=1 << 15),
                dict(idx=A256, slots=1 << 30)):
        assert _prefill(lib, **bad) == -2, bad
    for bad in (dict(q=MIS4), dict(k=MIS1), dict(v=MIS4), dict(out=MIS4), dict(first=MIS4), dict(last=MIS4), dict(g=MIS1), dict(cu=0x10002),
                dict(idx=MIS1)):
        assert _prefill(lib, **bad) == -3, bad
    for bad in (dict(ws=None), dict(ws=0x10010), dict(size=255)):
        assert _prefill(lib, **bad) == -4, bad


def test_workspace_sizes(lib):
    for size in (lib.k3lin_prefill_workspace_size, lib.k3lin_backward_workspace_size):
        assert size(1, 100, 1, 1, 128, 128, 1) >= 256
        assert size(1, 100, 1, 1, 128, 128, 2) == 0 and size(1, 100, 1, 1, 100, 128, 1) == 0 and size(0, 1, 1, 1, 64, 64, 1) == 0
        assert size(4, 1 << 30, 64, 64, 128, 128, 1) > 0                       # no product wraps


def _decode(lib, **kw):
    a = dict(q=A256, k=A256, v=A256, dtype=1, g=A256, fixed=0, state=A256, idx=None, idx_h=None, slots=2, N=2, Hk=2, H=4, dk=64, dv=64, scale=1.0,
             out=A256, odt=1)
    a.update(kw)
    return lib.k3lin_decode_step(a["q"], a["k"], a["v"], a["dtype"], a["g"], a["fixed"], a["state"], a["idx"], a["idx_h"], a["slots"], a["N"], a["Hk"],
                                 a["H"], a["dk"], a["dv"], a["scale"], a["out"], a["odt"], None)


def test_decode_refusals(lib):
    assert _decode(lib, N=0) == 0
    for bad in (dict(dtype=3), dict(odt=2), dict(scale=INF), dict(N=-1), dict(H=5), dict(q=None), dict(state=None), dict(out=None), dict(g=None),
                dict(idx=A256, idx_h=_host(1, 1)), dict(idx=A256, slots=0)):
        assert _decode(lib, **bad) == -1, bad
    assert _decode(lib, dk=20) == -2 and _decode(lib, dv=144) == -2
    for bad in (dict(state=MIS4), dict(q=MIS1), dict(g=MIS1), dict(out=MIS4), dict(idx=MIS1)):
        assert _decode(lib, **bad) == -3, bad


def _backward(lib, **kw):
    a = dict(q=A256, k=A256, v=A256, dtype=1, g=A256, first=A256, cu=A256, cu_h=None, N=2, T=10, Hk=2, H=4, dk=64, dv=64, scale=1.0, do=A256,
             dlast=A256, dq=A256, dk_=A256, dv_=A256, dg=A256, ds=A256, ws=A256, size=1 << 30)
    a.update(kw)
    return lib.k3lin_backward(a["q"], a["k"], a["v"], a["dtype"], a["g"], 0, a["first"], a["cu"], a["cu_h"], a["N"], a["T"], a["Hk"], a["H"], a["dk"],
                              a["dv"], a["scale"], a["do"], a["dlast"], a["dq"], a["dk_"], a["dv_"], a["dg"], a["ds"], a["ws"], a["size"], None)


def test_backward_refusals(lib):
    for bad in (dict(dtype=9), dict(scale=NAN), dict(N=0), dict(H=3), dict(do=None), dict(dq=None), dict(dk_=None), dict(dv_=None), dict(q=None),
                dict(cu=None), dict(cu_h=_host(0, 11, 10))):
        assert _backward(lib, **bad) == -1, bad
    assert _backward(lib, dk=40) == -2
    for bad in (dict(do=MIS4), dict(dlast=MIS4), dict(dq=MIS1), dict(ds=MIS4), dict(dg=MIS1)):
        assert _backward(lib, **bad) == -3, bad
    assert _backward(lib, ws=None) == -4 and _backward(lib, size=1000) == -4


def _norm(lib, **kw):
    a = dict(x=A256, dtype=1, res=A256, gate=A256, act=0, post=A256, pre=A256, rows=4, D=64, alpha=1.0, eps=1e-6, s=A256, y=A256)
    a.update(kw)
    return lib.k3blk_norm(a["x"], a["dtype"], a["res"], a["gate"], a["act"], a["post"], a["pre"], a["rows"], a["D"], a["alpha"], a["eps"], a["s"], a["y"],
                          None)


def test_norm_refusals(lib):
    assert _norm(lib, rows=0) == 0
    for bad in (dict(dtype=2), dict(rows=-1), dict(D=0), dict(alpha=NAN), dict(eps=-1.0), dict(eps=INF), dict(act=2), dict(pre=None), dict(y=None),
                dict(pre=None, y=None, s=None), dict(x=None)):
        assert _norm(lib, **bad) == -1, bad
    assert _norm(lib, D=16385) == -2 and _norm(lib, rows=1 << 31) == -2
    for bad in (dict(x=MIS1), dict(gate=MIS1), dict(res=MIS1), dict(s=MIS1), dict(y=MIS1), dict(post=0x10002), dict(dtype=0, x=0x10002)):
        assert _norm(lib, **bad) == -3, bad


def _norm_back(lib, **kw):
    a = dict(x=A256, dtype=1, ds=A256, dy=A256, sum=A256, gate=A256, act=1, post=A256, pre=A256, rows=4, D=64, alpha=1.0, eps=1e-6, dx=A256, dres=A256,
             dgate=A256, dpost=A256, dpre=A256, ws=A256, size=1 << 20)
    a.update(kw)
    return lib.k3blk_norm_backward(a["x"], a["dtype"], a["ds"], a["dy"], a["sum"], a["gate"], a["act"], a["post"], a["pre"], a["rows"], a["D"], a["alpha"],
                                   a["eps"], a["dx"], a["dres"], a["dgate"], a["dpost"], a["dpre"], a["ws"], a["size"], None)


def test_norm_backward_refusals(lib):
    for bad in (dict(dtype=2), dict(D=0), dict(alpha=INF), dict(act=-1), dict(ds=None), dict(dx=None), dict(x=None), dict(sum=None), dict(dy=None),
                dict(gate=None), dict(dgate=None), dict(dpost=None), dict(post=None), dict(pre=None), dict(dpre=None)):
        assert _norm_back(lib, **bad) == -1, bad
    assert _norm_back(lib, D=20000) == -2
    assert _norm_back(lib, dx=MIS1) == -3 and _norm_back(lib, dpre=0x10002) == -3
    assert _norm_back(lib, ws=None) == -4 and _norm_back(lib, size=100) == -4 and _norm_back(lib, ws=0x10010) == -4
    assert lib.k3blk_norm_backward_workspace_size(10, 0) == 0 and lib.k3blk_norm_backward_workspace_size(10, 64) >= 2 * 64 * 4


def test_outputs_that_are_inputs_are_refused(lib):
    at = lambda n: 0x10000 + 0x10000 * n  # noqa: E731
    for name in ("q", "k", "v", "g"):
        assert _prefill(lib, **{**dict(q=at(1), k=at(2), v=at(3), g=at(4), out=at(5)), name: at(5)}) == -1, name
        assert _decode(lib, **{**dict(q=at(1), k=at(2), v=at(3), g=at(4), state=at(6), out=at(5)), name: at(5)}) == -1, name
    assert _decode(lib, q=at(1), k=at(2), v=at(3), g=at(4), state=at(5), out=at(5)) == -1
    apart = dict(q=at(1), k=at(2), v=at(3), g=at(4), do=at(5), dq=at(6), dk_=at(7), dv_=at(8), dg=at(9), first=at(10), dlast=at(11), ds=at(12))
    for out in ("dq", "dk_", "dv_", "dg"):
        for name in ("q", "k", "v", "do", "g"):
            assert _backward(lib, **{**apart, out: apart[name]}) == -1, (out, name)
    assert _backward(lib, **{**apart, "ds": apart["first"]}) == -1 and _backward(lib, **{**apart, "ds": apart["dlast"]}) == -1
    apart = dict(x=at(1), ds=at(2), dy=at(3), sum=at(4), gate=at(5), dx=at(6), dgate=at(8))
    assert _norm_back(lib, **apart, dres=at(1)) == -1 and _norm_back(lib, **apart, dres=at(5)) == -1
    assert _prefill(lib, T=(1 << 31) - 100, size=1 << 62) == -2


def test_the_binding_refuses_cpu_tensors_and_wrong_shapes():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        K.k3lin_decode_step(q, q, q, torch.zeros(4, 2), torch.zeros(4, 2, 64, 64), 1.0, q)
    with pytest.raises(ValueError):
        K.k3blk_norm(q, None, None, "sigmoid", None, None, 1.0, 1e-6, q, None)
    with pytest.raises(ValueError):
        K.lin_prefill(q[0], q, q, torch.zeros(4, 2))
    with pytest.raises(K.K3KDAError):
        K.lin_prefill_workspace(1, 10, 1, 1, 100, 64)


# ---- the plain forms --------------------------------------------------------------------------

def test_plain_backward_is_the_gradient_of_plain_prefill():
    torch.manual_seed(0)
    T, hk, h, dk, dv, cu = 23, 2, 4, 3, 5, torch.tensor([0, 9, 9, 23])
    rand = lambda *s: torch.randn(s, dtype=torch.float64)  # noqa: E731
    for g in (-torch.rand(T, h, dtype=torch.float64), -torch.rand(h, dtype=torch.float64)):
        leaves = [rand(T, hk, dk), rand(T, hk, dk), rand(T, h, dv), g, rand(3, h, dk, dv)]
        for x in leaves:
            x.requires_grad_()
        q, k, v, g_, first = leaves
        out, last = P.prefill(q, k, v, g_, cu, first, 0.7)
        do, dlast = rand(T, h, dv), rand(3, h, dk, dv)
        want = torch.autograd.grad((out, last), leaves, (do, dlast))
        got = P.backward(*(x.detach() for x in (q, k, v, g_)), do, cu, first.detach(), dlast, 0.7)
        for a, b in zip(want, (got[x] for x in ("dq", "dk", "dv", "dg", "dS0"))):
            assert torch.allclose(a, b, rtol=1e-11, atol=1e-11)


def test_the_decays_gradient_is_a_running_sum():
    """dg_t = sum over u >= t of (q . dq - k . dk)_u + <S_T, dS_T>, pairs of a token with itself left out of both."""
    torch.manual_seed(1)
    T, h, dk, dv = 30, 2, 4, 3
    rand = lambda *s: torch.randn(s, dtype=torch.float64)  # noqa: E731
    q, k, v, g, do, first, dlast = rand(T, h, dk), rand(T, h, dk), rand(T, h, dv), -torch.rand(T, h, dtype=torch.float64), rand(T, h, dv), \
        rand(1, h, dk, dv), rand(1, h, dk, dv)
    d = P.backward(q, k, v, g, do, None, first, dlast, 0.5)
    _, last = P.prefill(q, k, v, g, None, first, 0.5)
    own = 0.5 * (q * k).sum(-1) * (do * v).sum(-1)
    x = ((q * d["dq"]).sum(-1) - own) - ((v * d["dv"]).sum(-1) - own)
    assert torch.allclose(x.flip(0).cumsum(0).flip(0) + (last * dlast).sum((0, 2, 3)), d["dg"], rtol=1e-11, atol=1e-11)


def test_plain_norm_backward_against_differences():
    torch.manual_seed(2)
    rand = lambda *s: torch.randn(s, dtype=torch.float64)  # noqa: E731
    x, res, gate, post, pre, ds, dy = rand(4, 6), rand(4, 6), rand(4, 6), rand(6), rand(6), rand(4, 6), rand(4, 6)
    for kind in ("sigmoid", "silu"):
        s, _ = P.block_norm(x, res, gate, kind, post, pre, 0.3)
        d = P.block_norm_backward(x, ds, dy, s, gate, kind, post, pre, 0.3)

        def loss(x, res, gate, post, pre):
            s, y = P.block_norm(x, res, gate, kind, post, pre, 0.3)
            return (s * ds).sum() + (y * dy).sum()
        at = dict(x=x, res=res, gate=gate, post=post, pre=pre)
        for name, grad in (("x", "dx"), ("res", "dresidual"), ("gate", "dgate"), ("post", "dpost"), ("pre", "dpre")):
            step, h = torch.randn_like(at[name]), 1e-5
            diff = (loss(**{**at, name: at[name] + h * step}) - loss(**{**at, name: at[name] - h * step})) / (2 * h)
            assert abs(diff - (d[grad] * step).sum()) < 1e-7 * (1 + abs(diff)), (kind, name)
