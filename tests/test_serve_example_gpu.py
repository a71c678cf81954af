"""The serving example: plan, append with rotation, attention and release run together with the
linear layers. Every call's inputs and results are read back: cached values against the rows'
keys and values, outputs against fp64 attention over the cache they were computed from."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                    "serve_hybrid.py")


def example():
    spec = importlib.util.spec_from_file_location("serve_hybrid", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Watch:
    """Checks every append and attention call of a server as it happens."""

    def __init__(self, torch, m, monkeypatch):
        self.torch, self.m, self.history, self.calls, self.mixed = torch, m, {}, 0, 0
        self.append, self.attn = gdn.gdn_kv_append, gdn.gdn_attn_paged
        self.end = m.Server.end
        monkeypatch.setattr(gdn, "gdn_kv_append", self.on_append)
        monkeypatch.setattr(gdn, "gdn_attn_paged", self.on_attn)
        monkeypatch.setattr(m.Server, "end", lambda server, slots: self.on_end(server, slots))

    def on_end(self, server, slots):
        for key in [k for k in self.history if k[1] in slots]:
            del self.history[key]
        self.end(server, slots)

    def on_append(self, h, cache, io, rows, places, k, ks, v, vs, rope, pos, ps, q, qs, hq, *rest):
        m = self.m
        f = lambda x, n: x.double().cpu().numpy().reshape(rows, n, m.DIM)  # noqa: E731
        self.k, self.v, q64 = f(k, m.KV), f(v, m.KV), f(q, hq)
        p = pos.cpu().numpy()[None]
        turn = lambda x: A.rope(x, p, m.ROTARY, [m.ROTARY // 2], False, False, 10000.0)  # noqa
        self.k = turn(self.k)
        want = turn(q64)
        self.append(h, cache, io, rows, places, k, ks, v, vs, rope, pos, ps, q, qs, hq, *rest)
        got = f(q, hq)
        # a rounding to bf16, and fp32 arithmetic on values of the pair's size
        pair = np.abs(q64).max()
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + pair * 2.0 ** -20).all()

    def on_attn(self, h, cfg, cache, n, rows, mq, mk, cu, kv_len, table, blocks, q, qs, o, os_, *rest):
        m = self.m
        self.attn(h, cfg, cache, n, rows, mq, mk, cu, kv_len, table, blocks, q, qs, o, os_, *rest)
        layer = next(x for x in self.server.layers if getattr(x, "cache", None) is cache)
        codes = [x.cpu().numpy() for x in layer.codes]
        scales = [x.cpu().numpy() for x in layer.scales]
        c = Case.__new__(Case)
        c.io, c.causal, c.dim, c.scale = "bf16", True, m.DIM, m.DIM ** -0.5
        c.codes, c.scales, c.table = codes, scales, table.cpu().numpy()
        c.cu, c.kv_len = cu.cpu().numpy(), kv_len.cpu().numpy().tolist()
        live = [b for b in range(n) if c.cu[b + 1] > c.cu[b]]
        c.q64 = q.double().cpu().numpy().reshape(rows, m.QUERY, m.DIM)
        got = o.double().cpu().numpy().reshape(rows, m.QUERY, m.DIM)
        want_lse = A.attention(c.q64, *codes, *scales, c.table, c.cu, c.kv_len, c.scale, True)[1]
        c.compare(got, want_lse)
        # the cache: each live request's whole history, through its table row
        values, held = A.e4m3_values(), []
        for b in live:
            lo, hi = c.cu[b], c.cu[b + 1]
            key = (id(layer), b)
            old = self.history.get(key, (np.zeros((0, m.KV, m.DIM)),) * 2)
            now = [np.concatenate([old[0], self.k[lo:hi]]), np.concatenate([old[1], self.v[lo:hi]])]
            self.history[key] = now
            length = c.kv_len[b]
            assert len(now[0]) == length
            pages = c.table[b, :-(-length // m.PAGE)]
            held += pages.tolist()
            at, off = pages[np.arange(length) // m.PAGE], np.arange(length) % m.PAGE
            for x, code, s in zip(now, codes, scales):
                s = s[at][:, :, None].astype(np.float64)
                y = values[code[at, :, off]] * s
                # half an e4m3 step: 2^-4 of the value, or of the subnormals' 2^-9; where the scale
                # grew later, half a subnormal step more for each of the (geometric) growths
                assert (np.abs(y - x) <= np.abs(x) * (2.0 ** -4 + 2.0 ** -16) + s * 2.0 ** -9).all()
        assert len(set(held)) == len(held)
        self.calls += 1
        lens = [int(c.cu[b + 1] - c.cu[b]) for b in live]
        self.mixed += min(lens) == 1 and max(lens) > 64


def test_requests_come_and_go(monkeypatch):
    torch = torch_cuda()
    handle()  # builds the library
    m = example()
    watch = Watch(torch, m, monkeypatch)
    torch.manual_seed(1)
    server = m.Server(slots=3, num_pages=24, max_tokens=512, layers="LF")
    watch.server = server
    prompts = [torch.randn(n, m.HIDDEN, device="cuda").bfloat16() for n in (70, 1, 200, 130, 63)]
    last = m.serve(server, prompts, 5)
    assert all(torch.isfinite(x).all() for x in last)
    assert watch.calls >= 12 and watch.mixed >= 1
    assert int(server.pages.count.item()) == 24
    assert sorted(server.pages.free.tolist()) == list(range(24))
    assert (server.pages.table == -1).all()
    server.close()


def test_too_few_pages_are_reported():
    torch = torch_cuda()
    handle()
    m = example()
    torch.manual_seed(2)
    server = m.Server(slots=2, num_pages=2, max_tokens=512, layers="F")
    server.step({0: torch.randn(64, m.HIDDEN, device="cuda").bfloat16(),
                 1: torch.randn(65, m.HIDDEN, device="cuda").bfloat16()})
    with pytest.raises(gdn.GdnError) as e:
        server.check()
    assert e.value.status == gdn.GDN_ERR_POOL_EXHAUSTED
    assert server.pages.kv_len.tolist() == [64, 0]
    server.close()
