"""Linear attention with a decay a head on the GPU against the definition in 64 bits.

Tolerances.  An output is off by its own rounding, at most half a step of its type relative to its value, and by what the
kernel's arithmetic adds.  That is bounded through M, the same sum over absolute values (of q, k, v, the states): the weights'
exponentials are off by less than 2^-20 of themselves, an operand in two BF16 parts by 2^-16 and in three by 2^-24, and every
addition by 2^-23 of a partial sum (tensor cores may cut instead of round), of which an output has no more in a row than its
sequence has tokens, and the products' 128 terms twice.  What is below 2^-126 FP32 holds with fewer bits or not at all: an
exponential, a state or a product that is lost so takes at most 2^-126 times a factor from each of the terms of a sum.  The inputs
here are below 2^3, so the factors (products of three of them at most, over 128 channels) are below 2^16; with fewer than 2^14 terms
that is 2^-96 in all."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import lin_plain as P  # noqa: E402

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)


def _case(lens, hk, h, dk, dv, dtype, first=True, fixed=False, seed=0, decay=1.0):
    g = torch.Generator(DEV).manual_seed(1000 + seed)
    T, N = sum(lens), len(lens)
    rand = lambda *s, dt=dtype: torch.randn(s, generator=g, device=DEV).to(dt)  # noqa: E731
    slope = decay * torch.exp2(-8 * (torch.arange(h, device=DEV) + 0.5) / h)
    c = dict(q=rand(T, hk, dk), k=rand(T, hk, dk), v=rand(T, h, dv), do=rand(T, h, dv), scale=dk ** -0.5,
             g=-slope if fixed else -slope * torch.rand((T, h), generator=g, device=DEV) * 2,
             first=rand(N, h, dk, dv, dt=F32) if first else None, dlast=rand(N, h, dk, dv, dt=F32) if first else None,
             cu=None if N == 1 else _cu(lens).to(DEV))
    return c


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _arith(dtype, longest, three=False):
    return (2.0 ** -20 if dtype == F32 or three else 2.0 ** -15) + (longest + 256) * 2.0 ** -23


def _near(got, want, M, arith, what):
    bound = _half(got.dtype) * want.abs() + arith * M + 2.0 ** -96
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= bound).all(), f"{what}: {(off / bound.clamp_min(1e-300)).max().item():.3g} times the bound"


def _check_prefill(c, out_dtype=None):
    dt = c["q"].dtype
    longest = max(b - a for a, b in P.sequences(c["cu"], c["q"].shape[0]))
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"], out_dtype=out_dtype)
    want, wlast = P.prefill(c["q"], c["k"], c["v"], c["g"], c["cu"], c["first"], c["scale"])
    M, Mlast = P.prefill(c["q"].abs(), c["k"].abs(), c["v"].abs(), c["g"], c["cu"], None if c["first"] is None else c["first"].abs(), c["scale"])
    _near(out, want, M, _arith(dt, longest, out.dtype == F32), "out")
    _near(last, wlast, Mlast, _arith(dt, longest, True), "state")


DIMS = [(128, 128), (64, 128), (128, 64), (16, 16), (48, 112), (112, 48)]
LENS = [[1], [37], [64], [65], [127, 1, 0, 129], [200, 0, 63, 512, 1], [1100]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_lengths(lens, dtype):
    _check_prefill(_case(lens, 3, 3, 128, 128, dtype))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_widths_and_shared_heads(dk, dv, dtype):
    _check_prefill(_case([150, 90], 2, 6, dk, dv, dtype, seed=1))


@pytest.mark.parametrize("dtype,out", [(BF, F32), (F32, BF)], ids=["bf16 in", "f32 in"])
def test_prefill_output_of_another_type(dtype, out):
    _check_prefill(_case([300], 2, 2, 128, 64, dtype, seed=2), out)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_one_decay_a_head_without_first_state(dtype):
    _check_prefill(_case([257, 70], 4, 4, 128, 128, dtype, first=False, fixed=True, seed=3))


@pytest.mark.parametrize("decay", [0.0, 30.0, 3000.0])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_decays_from_none_to_strong(decay, dtype):
    _check_prefill(_case([400], 2, 2, 64, 64, dtype, seed=4, decay=decay))


def test_prefill_many_heads_and_sequences():
    _check_prefill(_case([(7 * i) % 90 for i in range(70)], 8, 8, 64, 64, BF, seed=5))


@pytest.mark.parametrize("heads", [1, 5])
def test_prefill_one_long_sequence_is_cut_and_joined(heads):
    _check_prefill(_case([9001], heads, heads, 128, 128, BF, seed=6, decay=0.02))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_decay_of_minus_infinity_starts_anew(dtype):
    c = _case([300], 2, 2, 128, 128, dtype, seed=7)
    at = [0, 100, 128, 299]
    c["g"][at] = -float("inf")
    _check_prefill(c)
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"])
    cut = slice(100, 128)
    alone, _ = K.lin_prefill(*(c[x][cut].contiguous() for x in "qkvg"), c["first"])
    _near(alone, out[cut].double(), P.prefill(*(c[x][cut].abs() for x in "qkv"), c["g"][cut], None, None, c["scale"])[0],
          _half(out.dtype) + 2 * _arith(dtype, 64), "from the reset on")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_reaches_only_what_follows(dtype, which, value):
    lens, bad = [150, 130, 60], 150 + 77                    # within the second sequence, inside a chunk
    c = _case(lens, 2, 2, 128, 128, dtype, seed=8)
    ref, rlast = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    x = c[which].clone()
    x[(bad, 1) if which == "g" else (bad, 1, 5)] = value
    c[which] = x
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    same = torch.ones_like(out, dtype=torch.bool)
    if which == "q":
        same[bad, 1] = False
    elif which == "v":
        same[bad:280, 1, 5] = False
    else:
        same[bad:280, 1] = False
    assert torch.equal(out[same], ref[same])
    assert not torch.isfinite(out[~same]).any()
    slast = torch.ones_like(last, dtype=torch.bool)
    if which == "k":
        slast[1, 1, 5] = False
    if which == "v":
        slast[1, 1, :, 5] = False
    if which == "g":
        slast[1, 1] = False
    assert torch.equal(last[slast], rlast[slast])
    assert not torch.isfinite(last[~slast]).any()


def test_a_state_that_is_not_finite_stays_with_its_sequence():
    c = _case([70, 70], 1, 1, 64, 64, BF, seed=9)
    ref, _ = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    c["first"][0, 0, 3, 7] = float("nan")
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    assert torch.equal(out[70:], ref[70:]) and torch.isnan(out[:70, 0, 7]).all()
    keep = [i for i in range(64) if i != 7]
    assert torch.equal(out[:70, :, keep], ref[:70, :, keep])


def test_tokens_behind_the_last_sequence_are_left_alone():
    c = _case([100, 60], 2, 2, 128, 128, BF, seed=10)
    cu = _cu([90, 40]).to(DEV)
    out = torch.full_like(c["v"], 7.0)
    for x in "qkv":
        c[x][130:] = float("nan")
    last = torch.empty_like(c["first"])
    ws = K.lin_prefill_workspace(2, 160, 2, 2, 128, 128)
    K.k3lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], cu, c["scale"], out, last, ws)
    assert (out[130:] == 7).all() and torch.isfinite(out).all() and torch.isfinite(last).all()


def test_a_device_array_of_lengths_is_never_trusted():
    c = _case([100, 60], 1, 1, 64, 64, BF, seed=11)
    for cu in ([0, 1000, 160], [-5, 80, 160], [0, 90, 40]):
        bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
        out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], bad)
        K.lin_backward(c["q"], c["k"], c["v"], c["g"], c["do"], c["first"], c["dlast"], bad)
        torch.cuda.synchronize()
        assert torch.isfinite(last).all()


def test_no_tokens_hand_the_state_on():
    for dtype in (BF, F32):
        c = _case([0], 2, 4, 64, 32, dtype, seed=12)
        out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"])
        assert out.shape == (0, 4, 32) and torch.equal(last, c["first"])
        d = K.lin_backward(c["q"], c["k"], c["v"], c["g"], c["do"], c["first"], c["dlast"])
        assert torch.equal(d["dS0"], c["dlast"]) and d["dg"].shape == (0, 4)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_then_tokens_one_by_one(dtype):
    c = _case([100, 31], 2, 4, 64, 96, dtype, seed=13)
    want, _ = P.prefill(c["q"], c["k"], c["v"], c["g"], c["cu"], c["first"], c["scale"])
    M, _ = P.prefill(c["q"].abs(), c["k"].abs(), c["v"].abs(), c["g"], c["cu"], c["first"].abs(), c["scale"])
    pool = torch.full((5, 4, 64, 96), float("nan"), device=DEV)
    idx = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    pool[idx.long()] = c["first"]
    head = [90, 20]
    rows = torch.cat([torch.arange(0, 90), torch.arange(100, 120)]).to(DEV)
    out, same = K.lin_prefill(*(c[x][rows] for x in "qkvg"), pool, _cu(head).to(DEV), state_idx=idx)
    assert same is pool and torch.isnan(pool[[0, 2, 4]]).all()
    _near(out, want[rows], M[rows], _arith(dtype, 100), "prompt")
    for i in range(10):
        at = torch.tensor([90 + i, 120 + i], device=DEV)
        o = K.lin_decode_step(*(c[x][at] for x in "qkvg"), pool, idx)
        _near(o, want[at], M[at], _arith(dtype, 110), f"token {i}")
    assert torch.isnan(pool[[0, 2, 4]]).all()


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n,hk,h,fixed", [(1, 1, 1, False), (3, 2, 4, True), (70, 4, 8, False)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_decode(dk, dv, n, hk, h, fixed, dtype):
    c = _case([1] * n, hk, h, dk, dv, dtype, fixed=fixed, seed=14)
    cu = _cu([1] * n)
    want, wlast = P.prefill(c["q"], c["k"], c["v"], c["g"], cu, c["first"], c["scale"])
    M, Ml = P.prefill(c["q"].abs(), c["k"].abs(), c["v"].abs(), c["g"], cu, c["first"].abs(), c["scale"])
    state = c["first"].clone()
    o = K.lin_decode_step(c["q"], c["k"], c["v"], c["g"], state)
    _near(o, want, M, _arith(F32, 1), "out")
    _near(state, wlast, Ml, 2.0 ** -20, "state")


def test_decode_of_a_slot_outside_the_pool():
    c = _case([1, 1, 1], 2, 2, 128, 128, BF, seed=15)
    pool = c["first"].clone()
    idx = torch.tensor([2, 7, -1], dtype=torch.int32, device=DEV)
    o = K.lin_decode_step(c["q"], c["k"], c["v"], c["g"], pool, idx)
    assert torch.equal(pool[:2], c["first"][:2]) and not torch.equal(pool[2], c["first"][2])
    assert (o[1:] == 0).all() and (o[0] != 0).any()
    p = c["first"].clone()
    out, _ = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], p, _cu([1, 1, 1]).to(DEV), state_idx=idx)
    assert torch.equal(p[:2], c["first"][:2])
    alone, _ = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], None, _cu([1, 1, 1]).to(DEV))
    assert torch.equal(out[1:], alone[1:])


def test_a_state_may_be_its_own_successor():
    c = _case([130, 66], 2, 2, 128, 128, BF, seed=16)
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    state, o = c["first"].clone(), torch.empty_like(out)
    K.k3lin_prefill(c["q"], c["k"], c["v"], c["g"], state, c["cu"], c["scale"], o, state, K.lin_prefill_workspace(2, 196, 2, 2, 128, 128))
    assert torch.equal(o, out) and torch.equal(state, last)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_pool_of_states_in_place_under_sequences_that_are_cut(dtype):
    c = _case([2500, 0, 1, 1100], 1, 2, 64, 64, dtype, seed=17)
    out, last = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], c["first"], c["cu"])
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=DEV)
    pool = torch.full((6, 2, 64, 64), 7.0, device=DEV)
    pool[slots.long()] = c["first"]
    o, p = K.lin_prefill(c["q"], c["k"], c["v"], c["g"], pool, c["cu"], state_idx=slots)
    assert p is pool and torch.equal(o, out) and torch.equal(pool[slots.long()], last)
    assert (pool[[2, 4]] == 7).all()
    _check_prefill(c)


# ---- gradients ----------------------------------------------------------------------------------

def _check_backward(c):
    dt = c["q"].dtype
    seqs = P.sequences(c["cu"], c["q"].shape[0])
    longest = max(b - a for a, b in seqs)
    d = K.lin_backward(c["q"], c["k"], c["v"], c["g"], c["do"], c["first"], c["dlast"], c["cu"])
    args = [c[x] for x in ("q", "k", "v", "g", "do")]
    want = P.backward(*args, c["cu"], c["first"], c["dlast"], c["scale"])
    size = lambda x: None if x is None else x.abs()  # noqa: E731
    M = P.backward(*(size(a) for a in args[:3]), c["g"], size(c["do"]), c["cu"], size(c["first"]), size(c["dlast"]), c["scale"])
    for x in ("dq", "dk", "dv"):
        _near(d[x], want[x], M[x], _arith(dt, longest), x)
    _near(d["dS0"], want["dS0"], M["dS0"], _arith(dt, longest, True), "dS0")
    # dg: a running sum over at most 512 tokens of differences, each off by its terms' rounding (no term is larger than that with
    # absolute values), from an anchor's product of two states on
    reach = torch.zeros_like(M["each"])
    for a, b in seqs:
        for s in range(a, b, 512):
            e = min(s + 512, b)
            reach[s:e] = M["each"][s:e].flip(0).cumsum(0).flip(0)
    bound = reach + M["dg_token"]
    _near(d["dg"], want["dg"], bound.sum(0) if c["g"].dim() == 1 else bound, _arith(dt, longest, True), "dg")


@pytest.mark.parametrize("lens", [[1], [37], [64], [65, 1, 0, 129], [511, 513], [1100]], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_lengths(lens, dtype):
    _check_backward(_case(lens, 2, 2, 128, 128, dtype, seed=20))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_widths_and_shared_heads(dk, dv, dtype):
    _check_backward(_case([150, 90], 2, 6, dk, dv, dtype, seed=21))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_of_one_decay_a_head_without_states(dtype):
    _check_backward(_case([600, 70], 2, 4, 64, 64, dtype, first=False, fixed=True, seed=22))


@pytest.mark.parametrize("decay", [0.0, 30.0, 3000.0])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_decays_from_none_to_strong(decay, dtype):
    _check_backward(_case([700], 2, 2, 64, 64, dtype, seed=23, decay=decay))


def test_backward_one_long_sequence_is_cut_and_joined():
    _check_backward(_case([6000], 3, 3, 128, 128, BF, seed=24, decay=0.02))


@pytest.mark.parametrize("lens", [[300, 64, 1, 0, 900], [10] * 25, [64] * 38 + [65]], ids=lambda x: f"{len(x)} sequences")
def test_backward_of_more_pairs_than_ctas(lens):
    """Pieces of dk's launch that are halves of the others', and too few chunks for halves."""
    h = 40 if len(lens) == 5 else 4
    _check_backward(_case(lens, h // 2, h, 64, 48, BF, seed=27))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward_of_no_tokens(dtype):
    c = _case([0, 0], 2, 4, 64, 48, dtype, seed=28)
    for g in (c["g"], torch.tensor([-1.0, -2.0, 0.0, -0.5], device=DEV)):
        d = K.lin_backward(c["q"], c["k"], c["v"], g, c["do"], c["first"], c["dlast"], c["cu"])
        assert torch.equal(d["dS0"], c["dlast"]) and d["dq"].shape == (0, 2, 64) and (d["dg"] == 0).all() and d["dg"].shape == g.shape


def test_backward_without_the_decays_gradient():
    c = _case([140, 80], 2, 4, 128, 64, BF, seed=25)
    args = [c[x] for x in ("q", "k", "v", "g", "do", "first", "dlast", "cu")]
    a, b = K.lin_backward(*args), K.lin_backward(*args, need_dg=False)
    assert b["dg"] is None
    M = P.backward(*(c[x].abs() for x in "qkv"), c["g"], c["do"].abs(), c["cu"], c["first"].abs(), c["dlast"].abs(), c["scale"])
    for x in ("dq", "dk", "dv"):
        _near(b[x], a[x].double(), M[x], _half(BF) + 2 * _arith(BF, 140), x)


def test_gradients_against_differences():
    """o and the last state are linear in q, k and v one at a time, so a difference over any step is the derivative; for g the step's
    square remains: |f'''| h^2 / 6, with f''' no larger than the same sum of absolute values (every term is an exponential of a sum
    of at most all decays, moved by less than h in all)."""
    c = _case([90, 41], 2, 4, 64, 48, F32, seed=26)
    w, dl = c["do"].double(), c["dlast"].double()

    def loss(**kw):
        x = {**c, **kw}
        o, s = K.lin_prefill(x["q"], x["k"], x["v"], x["g"], x["first"], x["cu"])
        return ((o.double() * w).sum() + (s.double() * dl).sum()).item()
    d = K.lin_backward(c["q"], c["k"], c["v"], c["g"], c["do"], c["first"], c["dlast"], c["cu"])
    gen = torch.Generator(DEV).manual_seed(5)
    M, Ml = P.prefill(c["q"].abs() + 4, c["k"].abs() + 4, c["v"].abs() + 4, c["g"], c["cu"], c["first"].abs() + 4, c["scale"])
    size = ((M * w.abs()).sum() + (Ml * dl.abs()).sum()).item()          # all terms of either loss by size, steps below 4 included
    for x, y in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("first", "dS0")):
        step = torch.randn(c[x].shape, generator=gen, device=DEV).clamp(-4, 4)
        got = (loss(**{x: c[x] + step}) - loss(**{x: c[x] - step})) / 2
        want = (d[y].double() * step).sum().item()
        assert abs(got - want) <= 2 * _arith(F32, 90) * size, x
    h = 2.0 ** -9
    step = torch.rand(c["g"].shape, generator=gen, device=DEV) * 2 - 1
    got = (loss(g=c["g"] + h * step) - loss(g=c["g"] - h * step)) / (2 * h)
    want = (d["dg"].double() * step).sum().item()
    assert abs(got - want) <= (2 * _arith(F32, 90) / h + (90 ** 3) * h * h / 6) * size


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_of_what_is_not_finite_stay_where_they_belong(dtype):
    c = _case([100, 90], 2, 2, 64, 64, dtype, seed=27)
    args = [c[x] for x in ("q", "k", "v", "g")]
    ref = K.lin_backward(*args, c["do"], c["first"], c["dlast"], c["cu"])
    do = c["do"].clone()
    do[40, 1, 3] = float("inf")
    d = K.lin_backward(*args, do, c["first"], c["dlast"], c["cu"])
    assert torch.equal(d["dq"][torch.arange(190) != 40], ref["dq"][torch.arange(190) != 40])
    assert torch.equal(d["dk"][41:], ref["dk"][41:]) and torch.equal(d["dv"][41:], ref["dv"][41:])
    assert torch.equal(d["dS0"][1], ref["dS0"][1]) and torch.equal(d["dv"][:, 0], ref["dv"][:, 0])
    assert not torch.isfinite(d["dv"][:41, 1, 3]).any()


# ---- streams, graphs, order ---------------------------------------------------------------------

def test_results_do_not_change_from_run_to_run():
    c = _case([3500, 800], 3, 6, 128, 128, BF, seed=30, decay=0.1)
    args = [c[x] for x in ("q", "k", "v", "g")]
    a = K.lin_prefill(*args, c["first"], c["cu"])
    da = K.lin_backward(*args, c["do"], c["first"], c["dlast"], c["cu"])
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, K.lin_prefill(*args, c["first"], c["cu"])))
        db = K.lin_backward(*args, c["do"], c["first"], c["dlast"], c["cu"])
        assert all(torch.equal(da[x], db[x]) for x in da)


def test_captured_calls_that_share_a_workspace():
    c, e = _case([900, 60], 2, 2, 128, 128, BF, seed=31), _case([33, 700], 4, 4, 128, 64, BF, seed=32)
    ws = K.lin_backward_workspace(2, 960, 4, 4, 128, 128)

    def all_of(x, w):
        a = [x[y] for y in ("q", "k", "v", "g")]
        return [*K.lin_prefill(*a, x["first"], x["cu"], workspace=w),
                *K.lin_backward(*a, x["do"], x["first"], x["dlast"], x["cu"], workspace=w).values()]
    want = [all_of(x, None) for x in (c, e)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for x in (c, e):
            all_of(x, ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = all_of(x, ws)
            graphs.append((g, got))
        for _ in range(3):
            for g, _ in graphs:
                g.replay()
        fresh = torch.randn_like(c["v"])
        c["v"].copy_(fresh)                                # a replay takes what its inputs hold then
        graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[1], graphs[1][1]))
    assert all(torch.equal(a, b) for a, b in zip(all_of(c, None), graphs[0][1]))
    assert K.k3kda_workspace_status(ws) == 0


def test_another_stream():
    c = _case([500], 2, 2, 128, 128, BF, seed=33)
    a = [c[x] for x in ("q", "k", "v", "g")]
    want = [*K.lin_prefill(*a, c["first"]), *K.lin_backward(*a, c["do"], c["first"], c["dlast"]).values()]
    state, state2 = c["first"].clone(), c["first"].clone()
    one = [x[:1].contiguous() for x in a]
    w = K.lin_decode_step(*one, state)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20_000_000)                      # the current stream is busy: nothing below waits for it
        got = [*K.lin_prefill(*a, c["first"], stream=s), *K.lin_backward(*a, c["do"], c["first"], c["dlast"], stream=s).values(),
               K.lin_decode_step(*one, state2, stream=s)]
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want + [w], got))
    torch.cuda.synchronize()
    assert torch.equal(state, state2)
