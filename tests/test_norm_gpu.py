"""The RMS norm with residual, gate and 8-bit output against the plain fp64 reference."""
import numpy as np
import pytest

from oracle import attn_ref as A
from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import IO, empty_rows, num, rows, up

pytestmark = pytest.mark.gpu


def value_tolerance(v, gate, s_err):
    """A mean of squares is off by at most 2^-18 of itself (chains of 64 and a tree of 10 more
    roundings, all terms positive), so the root by half of that; reciprocal root, mean and two
    products: 2^-21. silu: 2^-20 and the rounding of its exponent."""
    rel = 2.0 ** -18
    if gate is not None:
        rel = rel + 2.0 ** -20 + np.abs(gate) * 2.0 ** -22
    return np.abs(v) * rel + s_err


class Case:
    def __init__(self, rng, tokens, heads, dim, io, residual, gate):
        self.tokens, self.heads, self.dim, self.io, width = tokens, heads, dim, io, heads * dim
        self.x = rows(rng, tokens, width, io)
        self.r = rows(rng, tokens, width, io, gap=16, scale=4.0) if residual else None
        self.g = rows(rng, tokens, width, io, gap=24, scale=3.0) if gate else None
        self.w = up(rng.standard_normal(dim))
        self.sum = empty_rows(tokens, width, io) if residual else None

    def run(self, y=None, codes=None, scales=None, sum=None, offset=0.0, weight=True, **kw):
        torch = torch_cuda()
        st = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
        cfg = gdn.make_norm_config(self.dim, self.w if weight else None, num_heads=self.heads,
                                   weight_offset=offset, io_dtype=IO[self.io][0], **kw)
        s = self.sum if sum is None else sum
        gdn.gdn_rms_norm(handle(), cfg, self.tokens, self.x, st(self.x), self.r, st(self.r), s,
                         st(s), self.g, st(self.g), y, st(y), codes, st(codes), scales)
        torch.cuda.synchronize()

    def want(self, offset=0.0, eps=1e-6, weight=True):
        opt = lambda t: None if t is None else num(t)  # noqa: E731
        s, v = R.rms_norm(num(self.x), opt(self.r), num(self.w) if weight else None, offset, eps,
                          self.heads, opt(self.g))
        # the residual's sum is rounded once in fp32: 2^-24 of itself, as much of v
        return s, v, value_tolerance(v, opt(self.g), np.abs(v) * 2.0 ** -23)


SHAPES = [(1, 1, 2048), (3, 1, 1), (5, 1, 77), (2, 1, 8), (130, 1, 1000), (7, 1, 8192), (2, 1, 16392),
          (1, 1, 32768), (33, 4, 128), (9, 3, 64), (5, 2, 256), (1100, 32, 128), (1500, 1, 515)]


@pytest.mark.parametrize("tokens,heads,dim", SHAPES)
@pytest.mark.parametrize("io,residual,gate", [("bf16", True, False), ("f32", False, True),
                                              ("bf16", False, True), ("f32", True, False)])
def test_values(tokens, heads, dim, io, residual, gate):
    rng = np.random.default_rng(tokens + dim)
    c = Case(rng, tokens, heads, dim, io, residual, gate)
    y = empty_rows(tokens, heads * dim, io)
    offset = 1.0 if tokens % 2 else 0.0
    c.run(y=y, offset=offset)
    s, v, tol = c.want(offset)
    half = IO[io][1]
    assert (np.abs(num(y) - v) <= tol + (np.abs(v) + tol) * half + 1e-37).all()
    if residual:
        assert (np.abs(num(c.sum) - s) <= np.abs(s) * (half + 2.0 ** -24)).all()


@pytest.mark.parametrize("tokens,heads,dim,group", [
    (1, 1, 2048, 0), (4, 1, 77, 0), (130, 1, 1024, 128), (3, 1, 96, 32), (2, 1, 8192, 64),
    (5, 4, 128, 0), (6, 3, 256, 128), (9, 2, 64, 32), (1200, 8, 128, 0), (1030, 1, 640, 128),
    (2, 1, 20000, 0), (3, 1, 24576, 64)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("pow2", [False, True])
def test_codes(tokens, heads, dim, group, io, pow2):
    torch = torch_cuda()
    rng = np.random.default_rng(dim + group)
    c = Case(rng, tokens, heads, dim, io, heads == 1, heads > 1)
    width = heads * dim
    n = width // group if group else 1
    codes = torch.full((tokens, -(-width // 16) * 16), 9, dtype=torch.uint8, device="cuda")[:, :width]
    scales, y = torch.zeros(tokens, n, device="cuda"), empty_rows(tokens, width, io)
    c.run(y=y, codes=codes, scales=scales, scale_group=group, scale_pow2=pow2)
    _, v, tol = c.want()
    assert (np.abs(num(y) - v) <= tol + (np.abs(v) + tol) * IO[io][1] + 1e-37).all()
    wide, err = v.reshape(tokens, n, -1), tol.reshape(tokens, n, -1)
    top, got = np.abs(wide).max(-1), num(scales)
    most = err.max(-1)
    if pow2:
        least = lambda t: np.exp2(np.ceil(np.log2(t / 448.0)))  # noqa: E731
        assert ((got == least(top - most)) | (got == least(top + most))).all()
    else:
        assert (np.abs(got - top / 448.0) <= most / 448.0 + top / 448.0 * 2.0 ** -23).all()
    value = A.e4m3_values()[codes.cpu().numpy()].reshape(tokens, n, -1) * got[..., None]
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normal numbers); the
    # quotient is a product with a reciprocal, 2^-23
    room = np.abs(wide) * (2.0 ** -4 + 2.0 ** -22) + got[..., None] * 2.0 ** -10 + err * 1.1
    assert (np.abs(value - wide) <= room).all()


@pytest.mark.parametrize("over", ["x", "r", "g"])
def test_in_place(over):
    torch = torch_cuda()
    rng = np.random.default_rng(21)
    a = Case(rng, 40, 1, 520, "bf16", True, True)
    y = empty_rows(40, 520, "bf16")
    a.run(y=y)
    s = a.sum.clone()
    # sum over the residual stream, y over x or gate; or y over the residual alone
    target = getattr(a, over)
    if over == "r":
        a.run(y=target)
        assert torch.equal(target, y)
    else:
        a.run(y=target, sum=a.r)
        assert torch.equal(target, y) and torch.equal(a.r, s)


def test_zeros_infinities_and_nan():
    torch = torch_cuda()
    width = 256
    x = torch.zeros(5, width, device="cuda")
    x[1] = torch.linspace(-1, 1, width, device="cuda")
    x[2, 7] = float("nan")
    x[3, :] = 3.0e38  # the squares' sum overflows: zeros
    x[4, 9] = float("inf")
    w = torch.ones(width, device="cuda")
    w[3], w[4], w[5] = float("inf"), float("-inf"), float("nan")
    for pow2 in (False, True):
        y = torch.empty(5, width, device="cuda")
        codes = torch.empty(5, width, dtype=torch.uint8, device="cuda")
        scales = torch.empty(5, 2, device="cuda")
        cfg = gdn.make_norm_config(width, w, scale_group=128, scale_pow2=pow2, io_dtype=gdn.GDN_F32)
        gdn.gdn_rms_norm(handle(), cfg, 5, x, width, y=y, y_stride=width, codes=codes,
                         codes_stride=width, scales=scales)
        torch.cuda.synchronize()
        val = torch.from_numpy(A.e4m3_values()).cuda()[codes.long()]
        assert (scales[0] == 2.0 ** -100).all() and (val[0, 6:] == 0).all()
        # the weights' infinities: the largest finite value, out of the scale; NaN stays NaN
        assert val[1, 3] == -448 and val[1, 4] == 448 and torch.isnan(val[1, 5])
        assert torch.isfinite(scales).all() and 0 < scales[1, 0] < 1
        assert torch.isnan(val[2]).all() and (scales[2] == 2.0 ** -100).all()
        assert torch.isnan(y[2]).all() and (y[3, 6:] == 0).all()
        assert torch.isnan(y[4, 9]) and (y[4, 10:] == 0).all()


def test_no_weight_no_tokens_and_a_large_eps():
    torch = torch_cuda()
    rng = np.random.default_rng(22)
    c = Case(rng, 6, 1, 100, "f32", False, False)
    y = empty_rows(6, 100, "f32")
    c.run(y=y, weight=False, eps=2.0)
    _, v, tol = c.want(weight=False, eps=2.0)
    assert (np.abs(num(y) - v) <= tol + np.abs(v) * 2.0 ** -23).all()
    c.tokens = 0
    y.fill_(7.0)
    c.run(y=y)
    assert (y == 7).all()


def test_past_four_gib():
    """Rows whose offsets pass 32 bits."""
    torch = torch_cuda()
    n, width = 280000, 8192
    x = torch.ones(n, width, dtype=torch.bfloat16, device="cuda")
    x[-1, ::2] = 3.0
    w = torch.ones(width, device="cuda")
    cfg = gdn.make_norm_config(width, w)
    gdn.gdn_rms_norm(handle(), cfg, n, x, width, y=x, y_stride=width)
    torch.cuda.synchronize()
    assert (x[:-1] == 1).all()
    want = torch.tensor([3.0, 1.0], device="cuda") / 5.0 ** 0.5
    assert torch.allclose(x[-1].float().view(-1, 2), want.expand(width // 2, 2), rtol=2.0 ** -7)
