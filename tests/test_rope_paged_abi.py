"""The rotary positions' table and the refusals of the rotation and of the paged cache's calls (no GPU: every
call returns from its argument checks)."""
import ctypes
import math

import numpy as np
import pytest

import hybrid_linear_attention_rule_gb300 as K
import paged_plain as PP

A16, MIS4, MIS1 = 0x10000, 0x10004, 0x10001           # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


SCALINGS = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=16.0, original_length=4096.0, beta_fast=32.0, beta_slow=1.0)]


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k["scaling"])
@pytest.mark.parametrize("dim", [2, 4, 48, 64, 128, 512])
def test_table_holds_turns_in_units_of_2_to_minus_64(lib, dim, kw):
    if dim == 2 and kw["scaling"] == "ntk":
        pytest.skip("refused")
    phase, m = K.k3mla_rope_table(dim, 10000.0, **kw)
    f, want_m = PP.frequencies(dim, **kw)
    turns = phase.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = np.mod(f / (2 * math.pi), 1.0)
    # pow and one division: a few units of 2^-53
    assert np.abs(turns - want).max() <= 8 * 2.0 ** -53 * np.abs(want).max()
    assert abs(m - want_m) <= 2.0 ** -23 * want_m


def test_table_of_a_frequency_beyond_a_whole_turn(lib):
    # theta < 1: pairs turn faster than 1 radian a position, here by more than a whole turn
    phase, _ = K.k3mla_rope_table(4, 0.001)
    want = math.pow(0.001, -0.5) / (2 * math.pi)
    assert want > 1
    got = phase.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert abs(got[1] - want % 1.0) < 1e-14


def test_table_refusals():
    for bad in (dict(dim=0), dict(dim=3), dict(dim=514), dict(dim=8, theta=0.0), dict(dim=8, theta=float("nan")),
                dict(dim=8, scaling="linear", factor=0.0), dict(dim=8, scaling="linear", factor=float("inf")),
                dict(dim=2, scaling="ntk", factor=2.0), dict(dim=8, scaling="by_parts", factor=2.0),
                dict(dim=8, scaling="by_parts", factor=2.0, original_length=10.0, beta_fast=1.0, beta_slow=1.0)):
        kw = dict(dim=8, theta=10000.0)
        kw.update(bad)
        with pytest.raises(K.K3KDAError) as e:
            K.k3mla_rope_table(**kw)
        assert e.value.status == -1, bad


def _v(data=A16, ts=128, hs=64):
    return K._View(data, ts, hs)


def _rope(lib, back=False, **kw):
    a = dict(q=_v(), qo=_v(0x20000), hq=2, k=None, ko=None, hk=0, shared=0, dtype=1, pos=A16, T=4, d=64, phase=A16, dim=64,
             off=0, layout=0, mscale=1.0)
    a.update(kw)
    r = K._RopeArgs(a["phase"], a["dim"], a["off"], a["layout"], a["mscale"]) if a["phase"] != "none" else None
    if back:
        return lib.k3mla_rope_backward(a["q"], a["qo"], a["hq"], a["k"], a["ko"], a["hk"], a["shared"], a["dtype"], a["pos"],
                                       a["T"], a["d"], r, None)
    return lib.k3mla_rope(a["q"], a["qo"], a["hq"], a["k"], a["ko"], a["hk"], a["dtype"], a["pos"], a["T"], a["d"], r, None)


def test_rope_refusals(lib):
    assert _rope(lib, T=0) == 0
    assert _rope(lib, T=-1) == -1
    assert _rope(lib, phase="none") == -1
    assert _rope(lib, phase=None) == -1
    assert _rope(lib, dim=63) == -1
    assert _rope(lib, dim=66) == -1                        # past the head
    assert _rope(lib, dim=32, off=34) == -1
    assert _rope(lib, off=-2, dim=32) == -1
    assert _rope(lib, layout=2) == -1
    assert _rope(lib, mscale=float("inf")) == -1
    assert _rope(lib, dtype=2) == -1
    assert _rope(lib, d=0) == -2 and _rope(lib, d=1025) == -2
    assert _rope(lib, pos=None) == -1
    assert _rope(lib, pos=0x10002) == -3
    assert _rope(lib, phase=MIS4) == -3
    assert _rope(lib, q=None) == -1
    assert _rope(lib, hq=0) == -1                          # q given, no heads of it
    assert _rope(lib, hk=2) == -1                          # heads of a k that is not there
    assert _rope(lib, q=_v(MIS1)) == -3
    assert _rope(lib, q=_v(ts=-1)) == -1
    assert _rope(lib, qo=_v(0x20000, hs=0)) == -1          # an output's rows must differ
    assert _rope(lib, qo=_v(0x20000, ts=0)) == -1
    k = _v(0x30000)
    assert _rope(lib, back=True, k=k, ko=k, hk=4, shared=1) == -1     # the sum in place of its terms
    assert _rope(lib, back=True, shared=1) == -1


def _cache(**kw):
    a = dict(pool=A16, table=A16, kv_len=A16, table_h=None, kv_len_h=None, format=2, pages=8, page=16, width=4, N=2, heads=2,
             dqk=128, dv=128)
    a.update(kw)
    return K._PagedArgs(a["pool"], a["table"], a["kv_len"], a["table_h"], a["kv_len_h"], a["format"], a["pages"], a["page"],
                        a["width"], a["N"], a["heads"], a["dqk"], a["dv"])


def _calls(lib, cu=A16, cu_h=None, T=3, dtype=1, k=_v(), v=_v(), rope=None, **kw):
    """(append, read) on the same arguments."""
    c = _cache(**kw)
    return (lib.k3mla_paged_append(c, k, v, dtype, cu, cu_h, T, rope, None),
            lib.k3mla_paged_read(c, k, v, dtype, cu, cu_h, T, None))


def _host(*x):
    return (ctypes.c_int32 * len(x))(*x)


def _adr(a):
    return ctypes.cast(a, ctypes.c_void_p).value


BAD_CACHES = [
    (dict(format=0), -1), (dict(format=3), -1), (dict(page=8), -2), (dict(page=24), -2), (dict(page=272), -2),
    (dict(dqk=96), -2), (dict(dv=192), -2), (dict(heads=0), -1), (dict(N=-1), -1), (dict(pages=-1), -1),
    (dict(width=1 << 27), -2), (dict(pool=None), -1), (dict(table=None), -1), (dict(kv_len=None), -1),
    (dict(pool=MIS4), -3), (dict(table=0x10002), -3), (dict(kv_len=MIS1), -3), (dict(cu=0x10002), -3), (dict(N=0), -1),
    (dict(cu=None), -1), (dict(T=-1), -1), (dict(dtype=5), -1), (dict(v=_v(MIS1)), -3), (dict(k=_v(hs=-4)), -1)]


@pytest.mark.parametrize("kw,want", BAD_CACHES, ids=[str(b[0])[:40] for b in BAD_CACHES])
def test_cache_refusals(lib, kw, want):
    assert _calls(lib, **kw) == (want, want)


def test_append_and_read_refusals(lib):
    assert lib.k3mla_paged_append(None, _v(), _v(), 1, A16, None, 3, None, None) == -1
    c = _cache()
    assert lib.k3mla_paged_append(c, None, _v(), 1, A16, None, 3, None, None) == -1
    assert lib.k3mla_paged_read(c, None, None, 1, A16, None, 3, None) == -1
    assert lib.k3mla_paged_read(c, _v(hs=0), None, 1, A16, None, 3, None) == -1
    assert lib.k3mla_paged_append(c, _v(), _v(), 1, A16, None, 3, K._RopeArgs(A16, 64, 96, 0, 1.0), None) == -1
    assert _calls(lib, T=0) == (0, 0)


def test_host_copies_are_checked(lib):
    good = dict(T=3, cu_h=_adr(_host(0, 1, 3)))
    # (a good call would launch; each of these differs from it in one number)
    for cu in ((0, 1, 2), (1, 1, 3), (0, 4, 3)):
        assert _calls(lib, T=3, cu_h=_adr(_host(*cu))) == (-1, -1)
    for lens in ((-1, 2), (1, 65), (0, 2), (1, 1)):        # negative, past the table, fewer than the new tokens
        assert _calls(lib, kv_len_h=_adr(_host(*lens)), **good) == (-1, -1)
    pages = [0, 1, 2, 3, 4, 5, 6, 7]
    for at, page in ((0, -1), (4, 8), (5, 99)):            # a page that some length reaches
        p = list(pages)
        p[at] = page
        assert _calls(lib, kv_len_h=_adr(_host(16, 17)), table_h=_adr(_host(*p)), **good) == (-1, -1)


def test_block_bytes(lib):
    assert K.k3mla_paged_block_bytes("i4", 64, 128, 128) == 64 * 256 * 9 // 16
    assert K.k3mla_paged_block_bytes("bf16", 16, 192, 128) == 16 * 320 * 2
    for bad in (("i4", 8, 128, 128), ("i4", 64, 100, 128), ("i4", 512, 128, 128), (7, 64, 128, 128)):
        assert K.k3mla_paged_block_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    q = torch.zeros(2, 2, 64)
    table = K.RopeTable(torch.zeros(32, dtype=torch.int64), 64, 0, "half", 1.0)
    with pytest.raises(ValueError):
        K.rope(q, torch.zeros(2, dtype=torch.int32), table)
    with pytest.raises(ValueError):
        K.k3mla_rope(q, torch.zeros(2, 3, 64), None, None, torch.zeros(2, dtype=torch.int32), table)
    with pytest.raises(ValueError):
        K.PagedCache(torch.zeros(2, 2, 2304, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32),
                     torch.zeros(1, dtype=torch.int32), 16, 128, 128)


def test_plain_forms_agree_with_each_other():
    """The tests' own 64-bit forms: a rotation and its inverse, packing and unpacking."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64))
    for layout in ("half", "interleaved"):
        y = PP.rotate(x, np.arange(5), 32, 16, layout)
        assert np.abs(PP.rotate(y, np.arange(5), 32, 16, layout, sign=-1.0) - x).max() < 1e-12
        assert np.array_equal(y[..., :16], x[..., :16]) and np.array_equal(y[..., 48:], x[..., 48:])
    rows = rng.standard_normal((2, 32, 128))
    v = PP.unpack_i4(PP.strips_i4(rows), 32, 128)
    step = (rows.reshape(2, 32, 2, 64).max(-1) - rows.reshape(2, 32, 2, 64).min(-1)) / 15
    # half a step of the code, and fp16's rounding of the scale (15 of it) and the minimum (2^-11 of each)
    assert (np.abs(v - rows).reshape(2, 32, 2, 64).max(-1) <= 0.5 * step + 15 * step * 2.0 ** -11 + 4 * 2.0 ** -11).all()


def _attend(lib, q=_v(), dtype=1, Hq=4, cu=A16, cu_h=None, T=3, max_new=2, rope=None, scale=1.0, gate=None, out=A16, out_dtype=0,
            ws=0x10000, ws_bytes=1 << 30, **kw):
    return lib.k3mla_paged_attend(_cache(**kw), q, dtype, Hq, cu, cu_h, T, max_new, rope, scale, gate, out, out_dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [b for b in BAD_CACHES if "v" not in b[0] and "k" not in b[0]], ids=str)
def test_attend_refuses_bad_caches(lib, kw, want):
    assert _attend(lib, **kw) == want


def test_attend_refusals(lib):
    assert _attend(lib, T=0) == 0
    assert _attend(lib, Hq=3) == -1 and _attend(lib, Hq=0) == -1       # not a multiple of the key heads
    assert _attend(lib, heads=1, Hq=1 << 17) == -2
    assert _attend(lib, max_new=0) == -1 and _attend(lib, max_new=1 << 25) == -2
    assert _attend(lib, scale=float("nan")) == -1
    assert _attend(lib, out_dtype=3) == -1
    assert _attend(lib, q=None) == -1 and _attend(lib, q=_v(MIS1)) == -3
    assert _attend(lib, gate=_v(MIS1)) == -3 and _attend(lib, gate=_v(None)) == -1
    assert _attend(lib, out=None) == -1 and _attend(lib, out=MIS4) == -3
    assert _attend(lib, ws=None) == -4 and _attend(lib, ws=0x10010) == -4
    assert _attend(lib, rope=K._RopeArgs(A16, 64, 96, 0, 1.0)) == -1
    assert _attend(lib, max_new=1, cu_h=_adr(_host(0, 1, 3))) == -1    # a sequence has more than max_new
    need = K.k3mla_paged_attend_workspace_size(4, 2, 128, 128)
    assert _attend(lib, ws_bytes=need - 1) == -4
    assert need % 16 == 0 and need > 0
    for bad in ((3, 2, 128, 128), (4, 0, 128, 128), (4, 2, 100, 128), (4, 2, 128, 192)):
        assert K.k3mla_paged_attend_workspace_size(*bad) == 0


def test_handles_are_fixed_and_names_are_checked():
    import torch
    table = K.RopeTable(torch.zeros(32, dtype=torch.int64), 64, 0, "half", 1.0)
    with pytest.raises(AttributeError):
        table.phase = None
    with pytest.raises(ValueError):
        K.RopeTable(torch.zeros(32, dtype=torch.int64), 64, 0, "quarter", 1.0)
    with pytest.raises(ValueError):
        K.k3mla_rope_table(64, 10000.0, scaling="other")
