"""Sampling where the last token kept lies among zeros and denormal logits: the bounds of the ranges
that are searched fall on every key there, the one below zero too."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from step_util import up
from test_sample_gpu import compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by", ["top_k", "top_p"])
@pytest.mark.parametrize("io,rows,unit,steps", [("bf16", 256, 2.0 ** -133, 15),
                                                ("f32", 2048, 2.0 ** -149, 511)])
def test_denormals_below_zero(by, io, rows, unit, steps):
    """The temperature moves the ranges' ends: one row in 16 (bf16) or 512 (fp32) has a range that
    ends just below zero, with the zeros outside it and more tokens inside than are ranked."""
    torch_cuda()
    rng = np.random.default_rng(rows)
    vocab = 1400
    x = np.zeros((rows, vocab), dtype=np.float32)
    x[:, 500:] = -rng.integers(1, steps + 1, (rows, 900)) * unit
    x[:, 100:200] = -0.0
    x = rng.permuted(x, axis=1)
    x[:, 7] = rng.choice([0.5, 1.0, 2.0, 3.0], rows)
    t, ones = 0.5 + rng.random(rows), np.ones(rows)
    u = rng.random(rows)
    if by == "top_k":
        compare(up(x, io), io, vocab, t, rng.integers(600, 1300, rows), ones, 0 * ones, u)
    else:
        compare(up(x, io), io, vocab, t, 0 * ones.astype(int), 0.45 + 0.5 * rng.random(rows), 0 * ones, u)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_values_around_zero_in_pairs(io):
    """Rows whose keys lie evenly around zero, many equal: ranges halved in the middle."""
    torch_cuda()
    rng = np.random.default_rng(8)
    rows, vocab = 512, 3000
    a = np.exp2(rng.uniform(-30, 3, (rows, 1)))
    x = a * rng.choice([-1.0, 0.0, -0.0, 1.0], (rows, vocab))
    t, ones = np.exp2(rng.uniform(-2, 5, rows)), np.ones(rows)
    compare(up(x, io), io, vocab, t, rng.integers(1, vocab, rows), rng.random(rows), 0 * ones,
            rng.random(rows))
    compare(up(x, io), io, vocab, t, 0 * ones.astype(int), rng.random(rows), 0 * ones, rng.random(rows))
