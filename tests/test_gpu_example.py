"""The example that runs the attention layers' operators together (it checks its own results)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
def test_attention_layer_example(fmt):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    errors = mod.main(["--fmt", fmt, "--steps", "8"])
    assert set(errors) == {"rope q", "rope k", "rope dq", "rope dk", "prompts", "tokens"}


def test_many_short_sequences():
    """More sequences than a CTA has threads: each gets its own."""
    import hybrid_linear_attention_rule_gb300 as K
    dev = "cuda:0"
    N, H, page = 1500, 2, 16
    g = torch.Generator(dev).manual_seed(3)
    lens = torch.randint(0, 40, (N,), generator=g, device=dev, dtype=torch.int32)
    table = torch.randperm(3 * N, generator=g, device=dev).to(torch.int32).view(N, 3)
    for fmt in ("i4", "bf16"):
        cache = K.PagedCache(K.paged_pool(3 * N, page, H, 64, 64, fmt, dev), table, lens, page, 64, 64, fmt)
        T = int(lens.sum())
        cu = torch.cat([torch.zeros(1, device=dev, dtype=torch.int32), lens.cumsum(0).to(torch.int32)])
        K.paged_append(cache, torch.randn(T, H, 64, device=dev), torch.randn(T, H, 64, device=dev), cu)
        k, v = K.paged_read(cache, T, cu, torch.float32)
        for group in (1, 60):                                # warps' runs, and blocks of 128 rows
            q = torch.randn(N, H * group, 64, device=dev)
            out = K.paged_attend(cache, q, out_dtype=torch.float32)
            kp, vp = torch.zeros(N, 40, H, 64, device=dev, dtype=torch.float64), torch.zeros(N, 40, H, 64, device=dev, dtype=torch.float64)
            n = torch.repeat_interleave(torch.arange(N, device=dev), lens.long())
            i = torch.arange(T, device=dev) - cu[n].long()
            kp[n, i], vp[n, i] = k.double(), v.double()
            s = torch.einsum("nhgd,nlhd->nhgl", q.double().unflatten(1, (H, group)), kp) * 0.125
            s = s.masked_fill((torch.arange(40, device=dev)[None] >= lens[:, None])[:, None, None], -float("inf"))
            want = torch.einsum("nhgl,nlhd->nhgd", torch.nan_to_num(torch.softmax(s, -1)), vp).flatten(1, 2)
            # values of a few units: FP32 with operands split in two (bf16 pages: 16 bits of them)
            assert float((out.double() - want).abs().max()) <= (1e-4 if fmt == "i4" else 1e-3)
            assert (out[lens == 0] == 0).all()
