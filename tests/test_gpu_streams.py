"""Calls on a stream other than the current one: what they allocate is that stream's, so that kernels still pending on the current stream
cannot write into it before the call has, nor the current stream's next allocations while it runs."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import kda_inputs as KI  # noqa: E402
from parity_utils import case_to_device  # noqa: E402

DEV = "cuda:0"
LONG = 40_000_000                                    # cycles: some 20 ms, longer than any of the calls


def _i(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rand(*s):
    return torch.randn(s, device=DEV).bfloat16()


def _paged(fmt="i4"):
    cache = K.PagedCache(K.paged_pool(8, 64, 4, 128, 128, fmt, DEV), _i(3, 1, 5, 0).view(2, 2), _i(100, 70), 64, 128, 128, fmt)
    K.paged_append(cache, _rand(170, 4, 128), _rand(170, 4, 128), _i(0, 100, 170))
    return cache


def _calls():
    torch.manual_seed(0)
    table, pos = K.rope_table(64, offset=64, device=DEV), _i(*range(300))
    q, k, cache, cu = _rand(300, 8, 128), _rand(300, 2, 128), _paged(), _i(0, 100, 170)
    ws = K.paged_attend_workspace(cache, 8)
    c = KI.prefill_case("streams", [200, 90], 2, 128, 128, 64, "bf16", seed=3, s0_std=0.02, gate=True)
    d = case_to_device(c)
    unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).bfloat16()
    dO = torch.randn(c.T, c.H, 128, device=DEV)
    args = [d[x] for x in ("q", "k", "v", "g", "beta")]
    unit_q, unit_k = unit(d["q"]), unit(d["k"])              # (the backward's recurrence takes keys of length 1)
    x, w = _rand(300, 64), torch.randn(64, 4, device=DEV)
    state = torch.zeros(2, 2, 128, 128, device=DEV)
    one = [t[:2].contiguous() for t in args]
    caches = iter([(torch.zeros(2, 2, 50, 128, device=DEV).bfloat16(), torch.zeros(2, 2, 50, 128, device=DEV).bfloat16(), _i(0, 7)) for _ in range(2)])
    held = []

    def step(s):
        held.append(next(caches))                          # (updated in place: a pair for each call)
        return K.mla_decode_step(*one[:3], *held[-1], stream=s)
    return {
        "rope": lambda s: K.rope(q, pos, table, k=k, stream=s),
        "rope backward": lambda s: K.rope_backward(q, pos, table, dk_out=k, k_shared=True, stream=s),
        "paged read": lambda s: K.paged_read(cache, 170, cu, stream=s),
        "paged attend, workspace": lambda s: K.paged_attend(cache, q[:170], cu, 100, table, workspace=ws, stream=s),
        "paged attend": lambda s: K.paged_attend(cache, q[:170], cu, 100, table, stream=s),
        "short conv": lambda s: K.short_conv(x, w, stream=s),
        "prefill": lambda s: K.prefill(*args, d["S0"], d["cu"], gate=d["gate"], stream=s),
        "backward": lambda s: tuple(K.backward(unit_q, unit_k, *args[2:], dO, d["S0"], cu_seqlens=d["cu"], stream=s).values()),
        "decode": lambda s: K.decode_step(*one, state, stream=s),
        "attention decode": step}, state


NAMES = ["rope", "rope backward", "paged read", "paged attend, workspace", "paged attend", "short conv", "prefill", "backward", "decode", "attention decode"]


def _flat(o):
    return [o] if torch.is_tensor(o) else [t for t in o if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_pending_kernels_of_the_current_stream_cannot_reach_the_outputs(name):
    """Blocks of the outputs' sizes are freed while a fill of them is still pending."""
    calls, state = _calls()
    call, zero = calls[name], state.clone()
    want = [t.clone() for t in _flat(call(None))]
    state.copy_(zero)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    victims = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(LONG)
    for v in victims:
        v.fill_(7)
    del victims, v
    got = call(s)
    torch.cuda.synchronize()
    for a, b in zip(_flat(got), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_scratches_in_stays_its_own_until_it_has_run(name):
    """The call's stream is busy; what the current stream allocates and fills meanwhile is not the call's memory."""
    calls, state = _calls()
    call, zero = calls[name], state.clone()
    want = [t.clone() for t in _flat(call(None))]
    state.copy_(zero)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    got = call(s)
    junk = [torch.full((1 << 10 << i,), 0xFF, dtype=torch.uint8, device=DEV) for i in range(16)] + \
           [torch.full((K.k3mla_paged_attend_workspace_size(8, 4, 128, 128),), 0xFF, dtype=torch.uint8, device=DEV)]
    del junk
    torch.cuda.synchronize()
    for a, b in zip(_flat(got), want):
        assert torch.equal(a, b)
