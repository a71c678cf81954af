"""Packs of prompts, drafts and decoding requests, which run the split, join and tile kernels in one
call: the same bits from call to call on one workspace without a wait between them, between calls
of another shape, on a side stream, on two streams at once, and from a graph."""
import numpy as np
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu


class Call:
    """A case's arrays on the device; run() enqueues the call into the given output."""

    def __init__(self, torch, seed, q_len, kv_len, hq, hkv, dim, page):
        self.torch, c = torch, Case(seed, q_len, kv_len, hq, hkv, dim, page)
        self.case, self.row = c, hq * dim
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.q = up(c.q).bfloat16().view(c.tokens, self.row)
        c.q64 = self.q.double().cpu().numpy().reshape(c.tokens, hq, dim)
        self.codes, self.scales = [up(x) for x in c.codes], [up(x) for x in c.scales]
        self.cache = gdn.make_kv_cache(*self.codes, *self.scales)
        self.cfg = gdn.make_attn_config(hq, scale=c.scale)
        self.cu, self.table = up(c.cu), up(c.table)
        self.kv = up(np.asarray(kv_len, np.int32))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def size(self):
        c = self.case
        return gdn.gdn_attn_workspace_size(self.cfg, self.cache, len(c.q_len), c.tokens,
                                           max(c.q_len), max(c.kv_len))

    def outputs(self):
        return (self.torch.full_like(self.q, 5.0),
                self.torch.full((self.case.tokens, self.case.hq), 7.0, device="cuda"))

    def run(self, out, work, stream=None):
        c = self.case
        gdn.gdn_attn_paged(handle(), self.cfg, self.cache, len(c.q_len), c.tokens, max(c.q_len),
                           max(c.kv_len), self.cu, self.kv, self.table, c.table.shape[1], self.q,
                           self.row, out[0], self.row, out[1], work, work.numel(), self.status,
                           stream)

    def check(self, out):
        c = self.case
        assert self.status.item() == 0
        c.compare(out[0].double().cpu().numpy().reshape(c.tokens, c.hq, c.dim),
                  out[1].double().cpu().numpy())


def _pair(torch, hq, hkv, dim, page):
    """Prompts enough for more units than SMs beside drafts and decode, and decode alone."""
    rng = np.random.default_rng(70)
    q_len = rng.integers(130, 150, 1200 // (2 * hq)).tolist() + [1] * 12 + [3] * 4 + [0]
    kv_len = [n + int(rng.integers(0, 200)) for n in q_len]
    a = Call(torch, 71, q_len, kv_len, hq, hkv, dim, page)
    assert sum(-(-n * (hq // hkv) // 128) for n in q_len) * hkv > 152
    b = Call(torch, 72, [1] * 9, rng.integers(1, 1500, 9).tolist(), hq, hkv, dim, page)
    return a, b


def _same(x, y):
    return all(bool((p == q).all()) for p, q in zip(x, y))


SHAPES = [(16, 2, 256, 64), (32, 8, 128, 16), (16, 4, 64, 32)]


@pytest.mark.parametrize("shape", SHAPES)
def test_calls_in_a_row_on_one_workspace(shape):
    torch = torch_cuda()
    a, b = _pair(torch, *shape)
    work = torch.full((max(a.size(), b.size()),), 0xA5, dtype=torch.uint8, device="cuda")
    outs = [(c, c.outputs()) for c in (a, b, a, a, b, b, a)]
    torch.cuda.synchronize()
    for c, out in outs:
        c.run(out, work)
    torch.cuda.synchronize()
    for c in (a, b):
        mine = [out for x, out in outs if x is c]
        c.check(mine[0])
        assert all(_same(mine[0], out) for out in mine[1:])


@pytest.mark.parametrize("shape", SHAPES)
def test_calls_on_two_streams_and_from_a_graph(shape):
    torch = torch_cuda()
    a, b = _pair(torch, *shape)
    work = [torch.empty(max(a.size(), b.size()), dtype=torch.uint8, device="cuda")
            for _ in range(2)]
    first = {c: c.outputs() for c in (a, b)}
    for c in (a, b):
        c.run(first[c], work[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [(c, i, c.outputs()) for _ in range(4) for i, c in ((0, a), (1, b), (1, a), (0, b))]
    torch.cuda.synchronize()
    for c, i, out in outs:  # each stream has a workspace of its own
        c.run(out, work[i], streams[i])
    torch.cuda.synchronize()
    assert all(_same(first[c], out) for c, _, out in outs)
    # a graph of both calls, replayed without a wait
    out = {c: c.outputs() for c in (a, b)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        with torch.cuda.graph(graph, stream=streams[0]):
            for c in (a, b):
                c.run(out[c], work[0], streams[0])
    torch.cuda.synchronize()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for c in (a, b):
        assert _same(first[c], out[c]) and c.status.item() == 0
