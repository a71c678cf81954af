"""Attention over the paged 8-bit cache against the plain fp64 reference."""
import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu


class Case:
    """A pack of requests with `q_len` queries behind `kv_len` cached tokens each."""

    def __init__(self, seed, q_len, kv_len, hq, hkv, dim, page, io="bf16", causal=True, scale=None,
                 spread=6, extra_rows=0, gap=0):
        rng = np.random.default_rng(seed)
        self.q_len, self.kv_len, self.io, self.causal = q_len, kv_len, io, causal
        self.hq, self.hkv, self.dim, self.page = hq, hkv, dim, page
        self.scale = dim ** -0.5 if scale is None else scale
        blocks = [-(-x // page) for x in kv_len]
        self.pages = sum(blocks) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((len(q_len), max(max(blocks), 1) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = order[at:at + n]
            at += n
        # anything may stand in unused places of a page: NaN codes among them
        self.codes = [rng.integers(0, 256, (self.pages, hkv, page, dim)).astype(np.uint8)
                      for _ in range(2)]
        self.scales = [(2.0 ** rng.integers(-spread, 1, (self.pages, hkv)) / 64).astype(np.float32)
                       for _ in range(2)]
        for b, n in enumerate(kv_len):
            for j in range(blocks[b]):
                rows = min(page, n - j * page)
                for c in self.codes:
                    live = c[self.table[b, j], :, :rows]
                    live[(live & 127) == 127] -= 1
        self.tokens = sum(q_len) + extra_rows
        self.cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.gap = gap
        self.q = (rng.standard_normal((self.tokens, hq, dim))
                  * 2.0 ** rng.integers(-3, 3, (self.tokens, hq, 1))).astype(np.float32)

    def run(self, torch, max_q=None, max_kv=None, stream=None, lse=True, keep=None):
        t = torch.bfloat16 if self.io == "bf16" else torch.float32
        code = gdn.GDN_BF16 if self.io == "bf16" else gdn.GDN_F32
        row = self.hq * self.dim
        wide = torch.full((self.tokens, row + self.gap), 3.0, dtype=t, device="cuda")
        wide[:, :row] = torch.from_numpy(self.q).cuda().to(t).view(self.tokens, row)
        q = wide[:, :row]
        self.q64 = q.double().cpu().numpy().reshape(self.tokens, self.hq, self.dim)
        o = torch.full((self.tokens, row + 2 * self.gap), 5.0, dtype=t, device="cuda")
        ls = torch.full((self.tokens, self.hq), 7.0, device="cuda")
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        c, s = [up(x) for x in self.codes], [up(x) for x in self.scales]
        cache = gdn.make_kv_cache(c[0], c[1], s[0], s[1])
        cfg = gdn.make_attn_config(self.hq, scale=self.scale, causal=self.causal, io_dtype=code)
        mq = max(self.q_len) if max_q is None else max_q
        mk = max(self.kv_len) if max_kv is None else max_kv
        n = len(self.q_len)
        bytes_ = gdn.gdn_attn_workspace_size(cfg, cache, n, self.tokens, mq, mk)
        ws = torch.full((bytes_,), 0xA5, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = (handle(), cfg, cache, n, self.tokens, mq, mk, up(self.cu),
                up(np.asarray(self.kv_len, np.int32)), up(self.table), self.table.shape[1], q,
                row + self.gap, o, row + 2 * self.gap, ls if lse else None, ws, bytes_, status,
                stream)
        if keep is not None:
            keep.append((args, c, s, wide))
        gdn.gdn_attn_paged(*args)
        torch.cuda.synchronize()
        out = o.float().cpu().numpy()
        assert (out[:, row:] == 5).all()
        return (out[:, :row].reshape(self.tokens, self.hq, self.dim).astype(np.float64),
                ls.cpu().numpy().astype(np.float64), int(status.item()))

    def check(self, torch, **kw):
        o, lse, status = self.run(torch, **kw)
        assert status == 0
        self.compare(o, lse)
        return o, lse

    def compare(self, o, lse, kv_len=None, cu=None):
        kv_len = self.kv_len if kv_len is None else kv_len
        cu = self.cu if cu is None else cu
        want, want_lse, mean, size, vmax = A.attention(self.q64, *self.codes, *self.scales,
                                                       self.table, cu, kv_len, self.scale,
                                                       self.causal)
        n = max(max(kv_len), 1)
        # a score is a sum of D products in fp32 (each partial sum within the sum of magnitudes),
        # two scalings and the hardware's 2^x (2^-22): relative error of a probability
        prob = 2 * (self.dim + 8) * 2.0 ** -24 * size + 2.0 ** -21
        term, half = (2.0 ** -11, 2.0 ** -8) if self.io == "bf16" else (2.0 ** -22, 2.0 ** -24)
        sums = (n + 64) * 2.0 ** -24  # accumulation of the weighted sum and of the total
        bound = np.abs(want) * half + mean * (term + 2 * prob + 2 * sums)[..., None] \
            + (n * 2.0 ** -31 * vmax)[..., None]
        rows = int(cu[-1])
        live = np.isfinite(want_lse[:rows])
        err = np.abs(o[:rows] - want[:rows])
        worst = (err / np.maximum(bound[:rows], 1e-300)).max() if rows else 0.0
        assert (err <= bound[:rows] + 1e-30).all(), f"{worst:.3f} of the bound"
        assert (lse[:rows][~live] == -np.inf).all()
        el = np.abs(lse[:rows] - want_lse[:rows])[live]
        assert (el <= (prob + sums)[:rows][live] + np.abs(want_lse[:rows][live]) * 2.0 ** -22).all()
        assert (o[:rows][~live] == 0).all()
        assert (o[rows:] == 5).all() and (lse[rows:] == 7).all()


HEADS = [(16, 2, 256), (8, 8, 64), (7, 1, 64), (32, 4, 128), (24, 1, 256), (12, 4, 128)]


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decode_lengths(hq, hkv, dim, page, io):
    """One query behind no token, one, lengths about the tile and page borders, a long one."""
    kv = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 130, 700]
    Case(1, [1] * len(kv), kv, hq, hkv, dim, page, io).check(torch_cuda())


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_few_queries(hq, hkv, dim, io, causal):
    """Drafts of 1 to 9 tokens, some behind fewer cached tokens than queries (rows that see
    nothing), requests without queries, rows past the last request."""
    q = [2, 1, 4, 0, 9, 3, 5]
    kv = [50, 200, 2, 30, 9, 0, 131]
    Case(2, q, kv, hq, hkv, dim, 16, io, causal, extra_rows=3, gap=32).check(torch_cuda())


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("io,page", [("bf16", 16), ("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_prompts(hq, hkv, dim, io, page):
    q, kv = [100, 1, 33, 257], [100, 300, 161, 300]
    Case(3, q, kv, hq, hkv, dim, page, io, gap=8).check(torch_cuda())


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 1, 256, 64), (8, 1, 256, 16), (4, 2, 128, 128),
                                             (3, 1, 128, 32), (2, 2, 64, 16), (7, 1, 64, 128)])
def test_long_prompts(hq, hkv, dim, page):
    """Prompts of several row and column tiles, behind prefixes that end inside a tile, beside
    a decoding request and a draft."""
    Case(20, [530, 1, 260, 3], [530, 700, 1413, 90], hq, hkv, dim, page, gap=8).check(torch_cuda())


def test_many_prompts_of_one_pass():
    """More units than blocks, of very different sizes."""
    rng = np.random.default_rng(21)
    q = rng.integers(1, 120, 90).tolist()
    kv = [n + int(rng.integers(0, 400)) for n in q]
    Case(21, q, kv, 8, 2, 64, 32).check(torch_cuda())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prompts_without_causal_mask(io):
    Case(4, [130, 40], [70, 333], 16, 2, 128, 32, io, causal=False).check(torch_cuda())


@pytest.mark.parametrize("dim,hq,hkv", [(256, 8, 1), (128, 4, 2), (64, 6, 2)])
def test_one_long_request_is_split(dim, hq, hkv):
    Case(5, [1], [20000], hq, hkv, dim, 64).check(torch_cuda())


def test_scales_of_very_different_size():
    """Page scales 2^-40 to 1: small pages count for their share."""
    torch = torch_cuda()
    for io in ("bf16", "f32"):
        c = Case(6, [1, 3, 70], [300, 500, 200], 8, 2, 128, 16, io, spread=6)
        rng = np.random.default_rng(0)
        c.scales[1] = (2.0 ** rng.integers(-20, 10, c.scales[1].shape)).astype(np.float32)
        c.check(torch)


def test_large_and_zero_queries_and_scores_far_apart():
    torch = torch_cuda()
    for io in ("bf16", "f32"):
        c = Case(7, [1, 2, 40], [100, 77, 200], 4, 2, 64, 16, io)
        c.q[0] *= 2.0 ** 40        # far outside fp16
        c.scale = 2.0 ** -44
        c.q[1] = 0
        c.q[2] *= 2.0 ** -60
        c.q[3, :, 5] = 2.0 ** 30   # one channel dwarfs the others
        c.check(torch)
        c = Case(8, [1, 2, 40], [100, 77, 200], 4, 2, 64, 16, io, scale=3.0)
        o, lse, status = c.run(torch)  # scores of hundreds: nearly one-hot rows, no overflow
        assert np.isfinite(o).all() and np.isfinite(lse).all() and status == 0


def test_result_does_not_depend_on_the_pack_or_the_stream():
    """The same bits again, on another stream; and a request alone within rounding."""
    torch = torch_cuda()
    c = Case(9, [1, 1, 4, 1], [900, 33, 500, 4000], 16, 2, 256, 64)
    o, lse = c.check(torch)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, lse2, _ = c.run(torch, stream=side)
    np.testing.assert_array_equal(o, o2)
    np.testing.assert_array_equal(lse, lse2)
    o3, _, _ = c.run(torch, lse=False)
    np.testing.assert_array_equal(o, o3)


def test_a_query_with_an_infinity_or_nan_spoils_its_own_rows_only():
    torch = torch_cuda()
    for q, kv in (([3], [50]), ([200], [200])):
        for bad in (np.inf, np.nan):
            c = Case(16, q, kv, 8, 2, 128, 16)
            c.q[1, 2, 5] = bad
            o, lse, _ = c.run(torch)
            assert np.isnan(o[1, 2]).all()
            o[1, 2] = 0
            assert np.isfinite(o).all()


def test_a_nan_key_reaches_only_those_who_see_it():
    torch = torch_cuda()
    for q, kv in (([4], [40]), ([70], [90]), ([300], [300])):
        c = Case(10, q, kv, 8, 2, 128, 16)
        j = kv[0] - 2  # seen by the last two queries
        c.codes[0][c.table[0, j // 16], :, j % 16, 3] = 0x7F
        o, lse, _ = c.run(torch)
        assert np.isnan(o[-2:]).all() and np.isnan(lse[-2:]).all()
        assert np.isfinite(o[:-2]).all() and np.isfinite(lse[:-2]).all()


def test_absent_pages_count_as_masked_and_are_flagged():
    torch = torch_cuda()
    for q, kv in (([1, 2, 1], [100, 300, 60]), ([1, 200, 90], [100, 300, 90])):
        for page in (16, 64):
            c = Case(11, q, kv, 8, 2, 128, page)
            c.table[0, 0] = -1
            c.table[1, 2] = c.pages
            c.table[2, 0] = 2**31 - 1
            if page == 64:
                c.table[2, 1] = -2**31  # the third request has no page left
            o, lse, status = c.run(torch)
            assert status == gdn.GDN_ERR_INVALID_ARGUMENT
            c.compare(o, lse)


def test_lengths_out_of_range_are_cut_and_flagged():
    torch = torch_cuda()
    c = Case(12, [1, 3, 2], [100, 50, 64], 8, 2, 128, 16)
    for x in c.codes:
        x[(x & 127) == 127] -= 1  # tokens past the stated length are read here
    c.kv_len = [100, 10**9, -5]
    o, lse, status = c.run(torch, max_kv=100)
    assert status == gdn.GDN_ERR_INVALID_ARGUMENT  # the second also runs off its pages
    c.compare(o, lse, kv_len=[100, 100, 0])
    # first rows out of range: rows outside the arrays are neither read nor written
    c = Case(13, [1, 3, 2], [100, 50, 64], 8, 2, 128, 16)
    c.cu = np.array([0, 1, 4, 9], np.int32)
    o, lse, status = c.run(torch, max_q=3)
    assert status == gdn.GDN_ERR_INVALID_ARGUMENT
    c.compare(o, lse, cu=np.array([0, 1, 4, 6]))
    c.cu = np.array([-7, 1, 4, 6], np.int32)
    o, lse, status = c.run(torch, max_q=3)
    assert status == gdn.GDN_ERR_INVALID_ARGUMENT
    c.cu = np.array([2**31 - 1, -2**31, 4, 6], np.int32)
    o, lse, status = c.run(torch, max_q=3)
    assert status == gdn.GDN_ERR_INVALID_ARGUMENT


def test_many_requests():
    """4,096 requests, most of them short: prefix sums over all of them."""
    torch = torch_cuda()
    rng = np.random.default_rng(14)
    kv = rng.integers(0, 40, 4096).tolist()
    kv[77], kv[4095] = 3000, 1000
    c = Case(14, rng.integers(0, 3, 4096).tolist(), kv, 2, 1, 64, 16)
    c.check(torch)


def test_append_then_attend_replays_from_a_graph():
    """Plan, append with rotation and attention of one decode step captured in a CUDA graph:
    three replays give the bits of three direct steps."""
    torch = torch_cuda()
    rng = np.random.default_rng(15)
    B, hq, hkv, dim, page, width, pages = 5, 8, 2, 128, 16, 8, 40
    T = B
    i32 = dict(dtype=torch.int32, device="cuda")
    qkv = torch.from_numpy(rng.standard_normal((T, (hq + 2 * hkv) * dim)).astype(np.float32)
                           ).cuda().to(torch.bfloat16)
    row = qkv.shape[1]
    rope = gdn.gdn_rope_init(dim, 64, [32], theta=1e6)
    cfg = gdn.make_attn_config(hq, scale=dim ** -0.5)
    h = handle()
    ones = torch.ones(B, **i32)

    class World:
        def __init__(self):
            self.ctx = torch.tensor([0, 3, 15, 16, 40], **i32)
            self.table = torch.full((B, width), -1, **i32)
            self.table[1, 0], self.table[2, 0], self.table[3, 0] = 0, 1, 2
            self.table[4, :3] = torch.tensor([3, 4, 5], **i32)
            self.free = torch.arange(6, pages, **i32)
            self.free = torch.cat([self.free, torch.zeros(6, **i32)])
            self.count = torch.tensor([pages - 6], **i32)
            self.c = [torch.zeros(pages, hkv, page, dim, dtype=torch.uint8, device="cuda")
                      for _ in range(2)]
            self.s = [torch.ones(pages, hkv, device="cuda") for _ in range(2)]
            self.cache = gdn.make_kv_cache(*self.c, *self.s)
            self.cu, self.kv = torch.empty(B + 1, **i32), torch.empty(B, **i32)
            self.pos = torch.empty(T, **i32)
            self.slots = torch.empty(T, dtype=torch.int64, device="cuda")
            self.qo = torch.empty(T, hq, dim, dtype=torch.bfloat16, device="cuda")
            self.o = torch.empty_like(self.qo)
            n = gdn.gdn_attn_workspace_size(cfg, self.cache, B, T, 1, width * page)
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            self.status = torch.zeros(1, **i32)

        def step(self, stream=None):
            gdn.gdn_kv_plan(h, page, B, T, self.ctx, ones, self.table, width, pages, self.free,
                            self.count, self.count, self.cu, self.kv, self.pos, self.slots,
                            self.status, stream)
            gdn.gdn_kv_append(h, self.cache, gdn.GDN_BF16, T, self.slots, qkv[:, hq * dim:], row,
                              qkv[:, (hq + hkv) * dim:], row, rope, self.pos, T, qkv, row, hq,
                              self.qo, hq * dim, self.status, stream)
            gdn.gdn_attn_paged(h, cfg, self.cache, B, T, 1, width * page, self.cu, self.kv,
                               self.table, width, self.qo, hq * dim, self.o, hq * dim, None,
                               self.ws, self.ws.numel(), self.status, stream)

    a, b = World(), World()
    for _ in range(3):
        a.step()
        a.ctx.copy_(a.kv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            b.step(side)
            b.ctx.copy_(b.kv)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for x, y in ((a.o, b.o), (a.qo, b.qo), (a.c[0], b.c[0]), (a.c[1], b.c[1]), (a.s[0], b.s[0]),
                 (a.table, b.table), (a.count, b.count), (a.kv, b.kv)):
        assert torch.equal(x, y)
    assert int(a.status.item()) == 0 == int(b.status.item())
    assert a.kv.tolist() == [3, 6, 18, 19, 43]
