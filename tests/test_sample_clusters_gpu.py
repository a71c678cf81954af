"""Sampling by the number of rows: many rows of a real vocabulary share the GPU in clusters of four, two
or one block a row where a few rows have eight each. Tokens and log-probabilities are the same bits."""
import numpy as np
import pytest

from gpu_util import torch_cuda
from step_util import up
from test_sample_gpu import compare, draw, settings

pytestmark = pytest.mark.gpu

# (io, rows, vocab): four blocks a row, two, one
SHAPES = [("bf16", 80, 50257), ("f32", 100, 50257), ("bf16", 160, 32003), ("f32", 160, 20011),
          ("bf16", 310, 20003), ("f32", 310, 9001)]


@pytest.mark.parametrize("kind", ["plain", "top_k", "top_p", "min_p", "all", "mixed"])
@pytest.mark.parametrize("io,rows,vocab", SHAPES)
def test_clusters(kind, io, rows, vocab):
    torch = torch_cuda()
    rng = np.random.default_rng(rows + vocab)
    logits = up(2.5 * rng.standard_normal((rows, vocab)) + 2.0, io)
    set_, u = settings(rng, rows, kind), rng.random(rows)
    few = rng.choice(rows, 40, replace=False)  # against the reference
    pick = lambda x: None if x is None else x[few]  # noqa: E731
    token, lp, status = draw(logits, io, vocab, *set_, u)
    assert status == 0
    part = logits[torch.from_numpy(few).cuda()].contiguous()
    want, _ = compare(part, io, vocab, *(pick(x) for x in set_), u[few])  # 40 rows: eight blocks each
    assert [token[i] for i in few] == want
    for a in range(0, rows, 32):
        cut = [None if x is None else x[a:a + 32] for x in set_]
        same, same_lp, _ = draw(logits[a:a + 32], io, vocab, *cut, u[a:a + 32])
        assert token[a:a + 32] == same and lp[a:a + 32] == same_lp


@pytest.mark.parametrize("io,rows,vocab", SHAPES[::2])
def test_ties_across_the_blocks_of_a_row(io, rows, vocab):
    """Many equal logits, cut by every filter at places in any block's slice."""
    torch_cuda()
    rng = np.random.default_rng(vocab)
    logits = up(rng.integers(-1, 2, (rows, vocab)), io)
    k, ones, u = rng.integers(1, vocab, rows), np.ones(rows), rng.random(rows)
    for set_ in ((ones, k, ones, 0 * ones), (ones, 0 * k, rng.random(rows), 0 * ones)):
        token, lp, _ = draw(logits, io, vocab, *set_, u)
        for a in range(0, rows, 32):
            same, same_lp, _ = draw(logits[a:a + 32], io, vocab, *(x[a:a + 32] for x in set_), u[a:a + 32])
            assert token[a:a + 32] == same and lp[a:a + 32] == same_lp
        compare(logits[:24], io, vocab, *(x[:24] for x in set_), u[:24])
