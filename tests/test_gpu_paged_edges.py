"""The paged cache's operators at values, arrays and streams where they could go wrong: against the 64-bit forms, or against what the header
says of such data."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
import paged_plain as PP  # noqa: E402
from test_gpu_paged_append import Case as Append  # noqa: E402

DEV = "cuda:0"


def _np(t):
    return t.detach().cpu().double().numpy()


def _stored(c, k):
    """What the definition stores for keys k (float64, turned) and the case's values."""
    want = np.concatenate([k, _np(c.v)], -1)
    code, s, m = PP.quantise(want.reshape(len(want), c.heads, -1, 64))
    return (code * s[..., None] + m[..., None]).reshape(want.shape)


@pytest.mark.parametrize("base,step", [(20000.0, 2.0 ** -9), (-60000.0, 2.0 ** -8), (2048.0, 2.0 ** -12), (512.0, 2.0 ** -14), (-1040.0, 2.0 ** -13)])
@pytest.mark.parametrize("most", [8, 40, 300])
def test_groups_far_from_zero_and_narrow(base, step, most):
    """FP32 channels of one large value plus 0..most units of its last place: the minimum over the scale has more bits than FP32."""
    rng = np.random.default_rng(most)
    c = Append([0, 9], [64, 30], 4, 128, 64, 32, "i4", torch.float32, make=lambda *s: base + step * rng.integers(0, most + 1, s))
    K.paged_append(c.cache, c.k, c.v, c.cu)
    assert np.array_equal(c.rows(), _stored(c, _np(c.k)))
