"""Value scales far apart: what a row gives follows from the tokens that it sees and their
weights (probability times value scale) alone, to the stated precision of the row's own
largest weight, wherever other pages' scales lie."""
import numpy as np
import pytest

from oracle import attn_ref as A

from gpu_util import torch_cuda
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu

# query heads, key/value heads, head dim, page size
SHAPES = [(8, 2, 128, 16), (8, 1, 256, 16), (4, 2, 64, 16), (16, 2, 256, 64), (4, 4, 128, 32)]


def _reference(c):
    """fp64: o, lse, mean |v| under the probabilities, largest scale * sum |q_d k_d|, largest
    weight times the largest code (448), and tokens seen, of every row and head."""
    values = A.e4m3_values()
    shape = (c.tokens, c.hq)
    o, mean = np.zeros(shape + (c.dim,)), np.zeros(shape + (c.dim,))
    lse, size, top, seen = (np.zeros(shape) for _ in range(4))
    group = c.hq // c.hkv
    for b, (n, kv) in enumerate(zip(c.q_len, c.kv_len)):
        ids = c.table[b][:-(-kv // c.page)]
        for h in range(c.hkv):
            ks, vs = (np.repeat(s[ids, h].astype(np.float64), c.page)[:kv] for s in c.scales)
            k, v = (values[x[ids, h]].reshape(-1, c.dim)[:kv] for x in c.codes)
            for i in range(n):
                see = kv - n + i + 1
                for x in range(h * group, (h + 1) * group):
                    r = c.cu[b] + i
                    s = c.scale * ks[:see] * (k[:see] @ c.q64[r, x])
                    p = np.exp(s - s.max())
                    w = p / p.sum() * vs[:see]
                    o[r, x], mean[r, x] = w @ v[:see], w @ np.abs(v[:see])
                    lse[r, x] = s.max() + np.log(p.sum())
                    size[r, x] = (c.scale * ks[:see] * (np.abs(k[:see]) @ np.abs(c.q64[r, x]))).max()
                    top[r, x], seen[r, x] = w.max() * 448.0, see
    return o, lse, mean, size, top, seen


def _check(torch, c):
    o, lse, status = c.run(torch)
    assert status == 0
    want, want_lse, mean, size, top, seen = _reference(c)
    # A score is a sum of D products in fp32 and is scaled twice; log2 of the value scale (at most
    # 126, off by 2^-22 of it) is added, the hardware's 2^x is off by 2^-22.
    prob = 2 * (c.dim + 8) * 2.0 ** -24 * size + 2.0 ** -21 + 126 * (2.0 ** -24 + 2.0 ** -22)
    # weights: 11 bits (fp32: 22), or half of fp16's smallest step, 2^-25, where the row's
    # largest is at least 2^6; sums; the output's own rounding
    term, half = (2.0 ** -11, 2.0 ** -8) if c.io == "bf16" else (2.0 ** -22, 2.0 ** -24)
    sums = (seen + 64) * 2.0 ** -24
    bound = np.abs(want) * half + mean * (term + 2 * prob + 2 * sums)[..., None] \
        + (seen * 2.0 ** -31 * top)[..., None]
    err = np.abs(o - want)
    worst = np.unravel_index(np.argmax(err / bound), err.shape)
    assert (err <= bound).all(), (worst, err[worst], bound[worst], want[worst])
    assert (np.abs(lse - want_lse) <= prob + sums + np.abs(want_lse) * 2.0 ** -22).all()


def _scales(c, b, exponents):
    """The value scales of request b's pages, one exponent a page (the last for the rest)."""
    for j, page in enumerate(c.table[b][:-(-c.kv_len[b] // c.page)]):
        c.scales[1][page] = 2.0 ** exponents[min(j, len(exponents) - 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-24, -28, -32, -40, -60])
def test_rows_in_front_of_a_page_of_large_values(shape, io, low):
    """A prompt and a draft whose early rows see only pages of small values, while a later page,
    in the same tile of 64 tokens, holds large ones."""
    hq, hkv, dim, page = shape
    c = Case(40 - low, [150, 4], [150, 4 * page + 2], hq, hkv, dim, page, io)
    _scales(c, 0, [low, low - 3, low + 2, 0, low, low, 4, low])
    _scales(c, 1, [low, low, low, low, 0])
    _check(torch_cuda(), c)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_pages_of_large_values_without_weight(shape, io):
    """Pages of large values whose keys point away from the queries: their weights are far below
    those of small values. Decode steps, a draft and a prompt."""
    hq, hkv, dim, page = shape
    q_len = [1, 1, 3, 120]
    c = Case(50, q_len, [90, 700, 200, 200], hq, hkv, dim, page, io, scale=1.0)
    c.q = np.abs(c.q) + 0.5
    for b in range(4):
        _scales(c, b, [0, -30, -28, -36] * 3 + [3, -30])
        pages = c.table[b][:-(-c.kv_len[b] // page)]
        c.scales[0][pages] = 2.0 ** -9
        # scores of the large pages: at most -0.5 * 64 * 2 = -64, of the others 64 at most less
        far = [p for p in pages if c.scales[1][p, 0] >= 1]
        c.codes[0][far] = 0x80 | 0x78            # -256 times 2^-7
        c.scales[0][far] = 2.0 ** -7
        near = [p for p in pages if c.scales[1][p, 0] < 1]
        c.codes[0][near] &= 0x3F                 # small keys, 0 to 1.875
    _check(torch_cuda(), c)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES[:3])
def test_scales_over_the_whole_range(shape, io):
    """2^-100 to 2^100 from page to page, first pages of zeros with the smallest scale, scales
    that are no powers of two."""
    hq, hkv, dim, page = shape
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    c = Case(60, [1, 5, 130], [400, 333, 260], hq, hkv, dim, page, io)
    c.scales[1] = (2.0 ** rng.integers(-100, 101, c.scales[1].shape)).astype(np.float32)
    _check(torch, c)
    first = [c.table[b][0] for b in range(3)]
    c.scales[1] = (2.0 ** rng.uniform(-9, 3, c.scales[1].shape)).astype(np.float32)
    c.codes[1][first] = 0
    c.scales[1][first] = 2.0 ** -100
    _check(torch, c)
    for e in (-100, 112):  # all of a size
        c.scales[1][:] = 2.0 ** e
        _check(torch, c)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nearly_one_hot_rows(io, dim):
    """Scores of hundreds."""
    _check(torch_cuda(), Case(8, [1, 2, 40, 130], [100, 77, 200, 130], 4, 2, dim, 16, io, scale=3.0))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scales_of_zero(io, shape):
    """A value scale of 0, or below 2^-100, makes zeros of any codes, and the tokens keep their
    part of the softmax sum; everywhere, in first pages, and in turns."""
    hq, hkv, dim, page = shape
    torch = torch_cuda()
    c = Case(65, [1, 5, 140], [300, 70, 140], hq, hkv, dim, page, io)
    c.scales[1][:] = 0
    o, lse, status = c.run(torch)
    assert status == 0 and (o == 0).all()
    _, want_lse, _, size, _, _ = _reference(c)
    assert (np.abs(lse - want_lse) <= 2 * (dim + 8) * 2.0 ** -24 * size + 2.0 ** -13).all()
    for small in (0.0, 2.0 ** -101, 2.0 ** -140):
        c.scales[1][:] = 2.0 ** -7
        for b in range(3):
            pages = c.table[b][:-(-c.kv_len[b] // page)]
            c.scales[1][pages[:1]] = small
            c.scales[1][pages[2::2]] = small
        keep = c.scales[1]
        c.scales[1] = np.where(keep == 2.0 ** -7, keep, 0).astype(np.float32)
        want = _reference(c)[0]
        c.scales[1] = keep
        o, _, status = c.run(torch)
        none = (want == 0).all(-1)
        assert status == 0 and none.any() and (o[none] == 0).all()
        c.scales[1] = np.where(keep == 2.0 ** -7, keep, 0).astype(np.float32)
        _check(torch, c)
