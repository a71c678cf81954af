"""Sampling against the plain fp64 reference: the same tokens, wherever no border is nearer than the
weights' own error."""
import numpy as np
import pytest

from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import IO, dtype, i32, num, up

pytestmark = pytest.mark.gpu

# weights are right to 2^-30 of themselves: shares of a total to 2^-28 with room
NEAR = 2.0 ** -28


def draw(logits, io, vocab, t=None, k=None, p=None, m=None, u=None, stride=None):
    torch = torch_cuda()
    n = len(u)
    f = lambda x: None if x is None else up(x)  # noqa: E731
    token = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    lp, status = torch.full((n,), 9.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = [f(t), None if k is None else i32(k), f(p), f(m), f(u)]
    gdn.gdn_sample(handle(), IO[io][0], n, vocab, logits, stride or vocab, *keep, token, lp, status)
    torch.cuda.synchronize()
    return token.tolist(), lp.tolist(), status.item()


def compare(logits, io, vocab, t, k, p, m, u, stride=None):
    """Every row's token and log-probability; at most one row in 50 may lie near a border."""
    token, lp, status = draw(logits, io, vocab, t, k, p, m, u, stride)
    rows = num(logits).reshape(len(u), -1)[:, :vocab]
    f32 = lambda x, i, d: float(np.float32(x[i])) if x is not None else d  # noqa: E731
    near = 0
    for i in range(len(u)):
        want, want_lp, gap = R.sample_row(rows[i], f32(t, i, 1.0), 0 if k is None else int(k[i]),
                                          f32(p, i, 1.0), f32(m, i, 0.0), f32(u, i, 0.0))
        if gap < NEAR:
            near += 1
            continue
        assert token[i] == want, i
        if np.isinf(want_lp):
            assert lp[i] == want_lp
        else:
            assert abs(lp[i] - want_lp) <= 2.0 ** -27 + abs(want_lp) * 2.0 ** -23, i
    assert near <= 1 + len(u) // 50
    return token, status


def settings(rng, n, kind):
    t, k = 0.3 + 1.5 * rng.random(n), rng.integers(1, 400, n)
    p, m = 0.05 + 0.95 * rng.random(n), 0.3 * rng.random(n)
    off = dict(plain=(t, None, None, None), top_k=(t, k, None, None), top_p=(t, None, p, None),
               min_p=(t, None, None, m), all=(t, k, p, m), ones=(None, None, None, None))
    if kind == "mixed":
        return (t * (rng.random(n) < 0.8), k * (rng.random(n) < 0.6),
                np.where(rng.random(n) < 0.5, p, 1.0), m * (rng.random(n) < 0.5))
    return off[kind]


@pytest.mark.parametrize("kind", ["ones", "plain", "top_k", "top_p", "min_p", "all", "mixed"])
@pytest.mark.parametrize("io,rows,vocab,spread", [
    ("f32", 40, 50257, 2.5), ("bf16", 30, 151936, 3.0), ("f32", 60, 1000, 1.0), ("bf16", 50, 4097, 0.2),
    ("f32", 64, 17, 2.0), ("bf16", 3, 262144, 2.0), ("f32", 2, 262144, 4.0)])
def test_rows(kind, io, rows, vocab, spread):
    rng = np.random.default_rng(vocab + rows)
    logits = up(spread * rng.standard_normal((rows, vocab)) - 3.0, io)
    compare(logits, io, vocab, *settings(rng, rows, kind), rng.random(rows))


@pytest.mark.parametrize("kind", ["top_k", "top_p", "all"])
@pytest.mark.parametrize("io,vocab,spread", [
    ("f32", 20000, 1e-3), ("bf16", 20000, 1e-3), ("f32", 60000, 0.05), ("bf16", 60000, 0.3),
    ("f32", 60000, 30.0), ("bf16", 60000, 30.0)])
def test_logits_around_zero(kind, io, vocab, spread):
    """The last token kept among many whose keys span the exponents."""
    rng = np.random.default_rng(int(spread * 1000))
    logits = up(spread * rng.standard_normal((16, vocab)), io)
    t, k, p, m = settings(rng, 16, kind)
    k = None if k is None else rng.integers(1, vocab, 16)
    compare(logits, io, vocab, t, k, p, m, rng.random(16))


@pytest.mark.parametrize("io,rows,vocab", [("f32", 700, 1000), ("bf16", 1023, 300), ("f32", 4100, 40)])
def test_many_rows_as_few(io, rows, vocab):
    """Rows in any order of their settings: each as in a call of a few rows, refused ones too."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    logits = up(2.0 * rng.standard_normal((rows, vocab)), io)
    t, k, p, m = settings(rng, rows, "mixed")
    p[rng.random(rows) < 0.02] = np.nan
    u = rng.random(rows)
    for setting in ((t, k, p, m), (t, None, p, None), (None, None, p, None), (t, k, np.ones(rows), m),
                    (t, k, np.full(rows, 0.5), m)):
        token, lp, status = draw(logits, io, vocab, *setting, u)
        cut = lambda x, a: None if x is None else x[a:a + 32]  # noqa: E731
        refused = 0
        for a in range(0, rows, 32):
            few, few_lp, bad = draw(logits[a:a + 32].contiguous(), io, vocab,
                                    *(cut(x, a) for x in setting), u[a:a + 32])
            assert token[a:a + 32] == few and lp[a:a + 32] == few_lp
            refused = max(refused, bad)
        assert status == refused
    torch.cuda.synchronize()


def test_rows_off_16_byte_boundaries():
    torch = torch_cuda()
    rng = np.random.default_rng(1)
    for io in ("f32", "bf16"):
        for off, stride in ((1, 5003), (3, 5001), (7, 5000)):
            flat = up(2 * rng.standard_normal(10 + 20 * stride), io)
            view = flat[off:off + 20 * stride].view(20, stride)
            assert view.data_ptr() % 16 != 0
            compare(view, io, 4999, *settings(rng, 20, "mixed"), rng.random(20), stride)
    assert torch.cuda.is_available()


def test_ties():
    """Many equal logits: a filter that cuts them keeps those of the lowest index."""
    rng = np.random.default_rng(2)
    vocab, rows = 30000, 32
    x = rng.integers(-2, 3, (rows, vocab)).astype(np.float64)
    x[:8] = 1.0           # a row of one value
    x[8:12, ::2] = -0.0   # equal to the zeros between them
    x[8:12, 1::2] = 0.0
    logits = up(x)
    u = rng.random(rows)
    k = rng.integers(1, vocab, rows)
    ones = np.ones(rows)
    compare(logits, "f32", vocab, ones, k, ones, 0 * ones, u)
    compare(logits, "f32", vocab, ones, 0 * k, rng.random(rows), 0 * ones, u)
    compare(logits, "f32", vocab, ones, k, rng.random(rows), 0.02 * ones, u)
    compare(logits, "f32", vocab, 0 * ones, k, ones, 0 * ones, u)
    # all equal, powers of two: top-k of 4,096 and u = j / 4,096 are exact
    even = up(np.zeros((64, 8192)))
    token, _, _ = draw(even, "f32", 8192, k=[4096] * 64, u=np.arange(64) * 64 / 4096.0)
    assert token == [64 * j for j in range(64)]
    token, _, _ = draw(even, "f32", 8192, p=[0.25] * 64, u=np.arange(64) * 32 / 2048.0)
    assert token == [32 * j for j in range(64)]


def test_infinities_nan_and_refused_rows():
    torch = torch_cuda()
    inf, nan = float("inf"), float("nan")
    x = np.zeros((12, 600))
    x[0] = -inf
    x[1] = nan
    x[2, 5:] = -inf
    x[3, [100, 300]] = inf
    x[4, ::2] = nan
    x[5, 77] = 3.0e38
    x[6, 10] = -inf
    t = [1.0, 1.0, 1.0, 1.0, 1.0, 0.5, inf, -1.0, nan, 1.0, 1.0, 0.0]
    p = [1.0] * 9 + [nan, 1.0, 1.0]
    m = [0.0] * 10 + [nan, 0.0]
    for io in ("f32", "bf16"):
        token, lp, status = draw(up(x, io), io, 600, t=t, p=p, m=m, u=[0.99999] * 12)
        assert status == gdn.GDN_ERR_INVALID_ARGUMENT
        assert token == [-1, -1, 4, 300, 599, 77, 599, -1, -1, -1, -1, 0]
        for i in (0, 1, 7, 8, 9, 10):
            assert lp[i] == -inf
        assert abs(lp[2] + np.log(5)) < 1e-6 and abs(lp[3] + np.log(2)) < 1e-6
        assert abs(lp[4] + np.log(300)) < 1e-6 and lp[5] == 0 and abs(lp[6] + np.log(599)) < 1e-6
        assert lp[11] == 0
        token, lp, status = draw(up(x[2:7], io), io, 600, t=t[2:7], k=[3] * 5, p=[0.5] * 5, u=[0.0] * 5)
        assert status == 0 and token == [0, 100, 1, 77, 0]
    assert torch.cuda.is_available()


def test_settings_at_their_ends():
    rng = np.random.default_rng(4)
    x = up(rng.standard_normal((1, 5000)))
    best = int(np.argmax(num(x)))
    order = np.argsort(-num(x)[0], kind="stable")
    one = lambda **kw: draw(x, "f32", 5000, **kw)[0][0]  # noqa: E731
    last = 1.0 - 2.0 ** -24
    for u in (0.0, 0.5, last, 1.0, 7.0, -3.0):
        assert one(u=[u], k=[1]) == best and one(u=[u], p=[0.0]) == best
        assert one(u=[u], p=[-1.0]) == best and one(u=[u], m=[1.0]) == best
        assert one(u=[u], m=[5.0]) == best and one(u=[u], t=[0.0]) == best
        assert one(u=[u], t=[1e-30]) == best and one(u=[u], p=[1e-30]) == best
    assert one(u=[0.0]) == 0 and one(u=[last], t=[float("inf")]) == 4999
    assert one(u=[1.0]) == 4999 and one(u=[5.0]) == 4999 and one(u=[-1.0]) == 0
    assert one(u=[1.0], k=[2]) == max(order[:2]) and one(u=[0.0], k=[2]) == min(order[:2])
    for k in (0, -5, 5000, 6000):  # off
        assert one(u=[0.37], k=[k]) == one(u=[0.37])
    for p in (1.0, 2.0, float("inf")):
        assert one(u=[0.37], p=[p]) == one(u=[0.37])
    for m in (0.0, -1.0):
        assert one(u=[0.37], m=[m]) == one(u=[0.37])
    single = up(np.array([[0.3]]))
    assert draw(single, "f32", 1, u=[0.9], k=[1], p=[0.3])[0] == [0]


def test_frequencies():
    """Over an even grid of u every token is drawn as often as its share says, to one count."""
    rng = np.random.default_rng(5)
    n = 4096
    x = 1.5 * rng.standard_normal(40)
    logits = up(np.tile(x, (n, 1)))
    token, _, _ = draw(logits, "f32", 40, t=[0.8] * n, u=(np.arange(n) + 0.5) / n)
    row = num(logits)[0]
    w = np.exp((row - row.max()) / float(np.float32(0.8)))
    count = np.bincount(token, minlength=40)
    assert (np.abs(count - n * w / w.sum()) <= 1.001).all()
    assert token == sorted(token)


def test_the_same_bits_again_and_from_a_graph():
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    n, vocab = 16, 32000
    logits = up(2 * rng.standard_normal((n, vocab)), "bf16")
    t, k, p, m = (up(x) if i != 1 else i32(x) for i, x in enumerate(settings(rng, n, "all")))
    u = up(rng.random(n))
    out = [(torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda"))
           for _ in range(2)]
    args = (handle(), gdn.GDN_BF16, n, vocab, logits, vocab, t, k, p, m, u)
    gdn.gdn_sample(*args, *out[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gdn.gdn_sample(*args, *out[1], None, s)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    u.copy_(torch.flip(u, [0]))
    g.replay()
    gdn.gdn_sample(*args, *out[0])
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0])
    assert dtype("bf16") == logits.dtype
