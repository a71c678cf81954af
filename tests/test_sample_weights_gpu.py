"""The stated precision of a weight: 2^-28 of its own value."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from step_util import up
from test_sample_gpu import draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab,spread", [(2, 1.0), (2, 7.0), (6000, 4.0)])
def test_min_p_beside_a_weight(vocab, spread):
    """Rows of a zero and one other finite logit, min_p the fp32 number nearest to its weight. The token
    is kept where its weight is min_p or more; it may err only within 2^-28 (a unit of 2^-44 is 2^-32 of
    weights above 2^-12)."""
    torch_cuda()
    rng = np.random.default_rng(vocab)
    n = 40000 if vocab == 2 else 3000
    t = np.exp2(rng.uniform(-4, 4, n)).astype(np.float32).astype(np.float64)
    l = (-spread * rng.random(n) * t).astype(np.float32).astype(np.float64)
    w = np.exp(l / t)
    m = w.astype(np.float32).astype(np.float64)
    gap = w / m - 1
    pick = (np.abs(gap) >= 2.0 ** -28) & (w > 2.0 ** -12) & (m < 1)
    t, l, w, m, gap = (a[pick] for a in (t, l, w, m, gap))
    assert (np.abs(gap) < 2.0 ** -26).sum() > len(gap) // 50  # many beside the border
    x = np.full((len(t), vocab), -np.inf, dtype=np.float32)
    x[:, 0], x[:, -1] = 0.0, l
    token, _, status = draw(up(x), "f32", vocab, t=t, m=m, u=np.full(len(t), 1 - 2.0 ** -24))
    assert status == 0
    kept = np.array(token) == vocab - 1
    np.testing.assert_array_equal(kept, gap > 0)
