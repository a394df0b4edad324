"""Sizes at which the paged cache's calls are refused and accepted (no GPU: every call returns from its argument checks, an accepted
attention from the one on its workspace)."""
import pytest

import hybrid_linear_attention_rule_gb300 as K
from test_rope_paged_abi import _adr, _attend, _calls, _host, _v

UNSUPPORTED, WORKSPACE = -2, -4


@pytest.fixture(scope="module")
def lib():
    return K.load_library()


def _call(lib, T, heads, group, table, fmt=2, d=(128, 128), N=1, max_new=None, page=64, **kw):
    return _attend(lib, Hq=heads * group, heads=heads, q=_v(ts=heads * group * d[0], hs=d[0]), T=T, max_new=max_new or T, width=table // page,
                   pages=table // page, page=page, N=N, format=fmt, dqk=d[0], dv=d[1], ws_bytes=0, **kw)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T,heads,group,table,N", [
    (32768, 32, 1, 131072, 1), (8192, 32, 4, 131072, 1), (8192, 8, 8, 1 << 20, 1), (65536, 32, 1, 65536, 1), (16384, 8, 8, 131072, 1),
    (2048, 8, 8, 1 << 20, 4), (65536, 32, 1, 1 << 20, 16), (4096, 32, 1, 1 << 20, 1), (131072, 4, 8, 131072, 1)])
def test_prompts_over_long_tables_are_accepted(lib, T, heads, group, table, N, fmt):
    assert _call(lib, T, heads, group, table, fmt, N=N) == WORKSPACE


def _units(T, heads, group, table, N, rows, tile, extra):
    return (T * group // rows + min(N, T)) * heads * (-(-table // tile) + extra)


@pytest.mark.parametrize("fmt,d,group,new,rows,tile,extra", [
    (2, (128, 128), 8, 0, 128, 64, 10), (1, (64, 64), 16, 0, 128, 64, 10), (2, (192, 128), 4, 8, 128, 64, 10), (2, (192, 128), 4, 7, 8, 32, 2),
    (1, (128, 128), 1, 9, 128, 64, 10), (1, (128, 128), 1, 8, 8, 16, 2), (1, (64, 64), 1, 8, 8, 32, 2), (2, (256, 128), 4, 0, 8, 32, 2),
    (2, (64, 256), 1, 0, 8, 32, 2), (2, (128, 128), 1, 36, 8, 64, 2), (2, (128, 128), 1, 37, 128, 64, 10), (2, (128, 128), 4, 1, 4, 64, 2)])
def test_the_limit_is_that_of_the_kernel_that_runs(lib, fmt, d, group, new, rows, tile, extra):
    """new: max_new (0: all tokens are one sequence's)."""
    heads, table = 128, 1 << 19
    per = heads * (table // tile + extra)
    N = 1 if new == 0 else 300
    last = ((2 ** 31 - 1) // per - N + 1) * rows // group - 1          # the most tokens whose blocks fit
    assert _units(last, heads, group, table, N, rows, tile, extra) < 2 ** 31 <= _units(last + 1, heads, group, table, N, rows, tile, extra)
    assert _call(lib, last, heads, group, table, fmt, d, N=N, max_new=new or last) == WORKSPACE
    assert _call(lib, last + 1, heads, group, table, fmt, d, N=N, max_new=new or last + 1) == UNSUPPORTED


def test_no_tokens_and_one_each(lib):
    assert _call(lib, 0, 128, 8, 1 << 24, N=100000, max_new=1) == 0
    assert _call(lib, 4096, 8, 4, 1 << 20, N=4096, max_new=1, cu=None) == WORKSPACE
    assert _call(lib, 65536, 32, 4, 1 << 20, N=65536, max_new=1, cu=None) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(theta=1e-320), dict(scaling="linear", factor=1e-310), dict(theta=1e-300, scaling="linear", factor=1e-20),
                                dict(theta=1e-300, scaling="by_parts", factor=1e-300, original_length=4096.0)], ids=str)
def test_table_refuses_frequencies_that_are_not_finite(kw):
    """Their turns have no fraction to hold."""
    with pytest.raises(K.K3KDAError) as e:
        K.k3mla_rope_table(**{"dim": 128, "theta": 10000.0, **kw})
    assert e.value.status == -1


def test_table_takes_frequencies_up_to_the_largest():
    """Whole turns a position leave a phase of 0, and an infinite base the first pair alone."""
    phase, _ = K.k3mla_rope_table(4, 1e-300)
    assert phase[1] == 0 and phase[0] != 0
    phase, _ = K.k3mla_rope_table(8, 1e300, scaling="ntk", factor=1e30)
    assert phase[0] != 0 and not phase[1:].any()


@pytest.mark.parametrize("page,width,want", [(16, (1 << 27) - 16, 0), (16, (1 << 27) - 15, UNSUPPORTED), (16, (1 << 27) - 1, UNSUPPORTED), (256, (1 << 23) - 1, 0),
                                             (240, (1 << 31) // 240, UNSUPPORTED)])
def test_tables_whose_last_tile_would_pass_31_bits_are_refused(lib, page, width, want):
    """A tile holds up to 64 tokens: with 2^31 - 16 positions the last one's end has no int."""
    assert _attend(lib, T=0, page=page, width=width) == want


def test_a_host_packing_alone_is_not_taken_for_one_token_each(lib):
    """Without the device array every sequence has one token, whatever the host copy says; one that says otherwise is refused."""
    for cu, want in (((0, 2, 2), -1), ((0, 0, 2), -1), ((0, 1, 2), WORKSPACE)):
        assert _attend(lib, T=2, cu=None, cu_h=_adr(_host(*cu)), ws_bytes=0) == want
    assert _calls(lib, T=2, cu=None, cu_h=_adr(_host(0, 2, 2))) == (-1, -1)


@pytest.mark.parametrize("tokens,sequences,packed,want", [(64, 64, True, 1), (5, 64, True, 1), (65, 64, True, 65), (64, 64, False, 1), (0, 3, True, 1)])
def test_what_a_call_without_max_new_takes(monkeypatch, tokens, sequences, packed, want):
    """A decode batch that is packed is one token a sequence, not one sequence of all tokens: the kernel for few rows."""
    import types

    import torch
    taken = []
    monkeypatch.setattr(K, "k3mla_paged_attend", lambda cache, q, gate, out, ws, scale, cu, cu_host, max_new, rope, stream: taken.append(max_new))
    cache, q = types.SimpleNamespace(N=sequences, dqk=64, dv=64), torch.zeros(tokens, 1, 64)
    K.paged_attend(cache, q, torch.zeros(sequences + 1, dtype=torch.int32) if packed else None, out=q, workspace=q)
    assert taken == [want]
