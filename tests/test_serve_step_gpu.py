"""The serving example with selective-scan layers and a vocabulary: convolution, scan, norm and
sampling run together with the linear and full-attention layers. Every call's results are checked
against the plain references on the inputs that it had."""
import numpy as np
import pytest

from oracle import attn_ref as A
from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import num
from test_conv_gpu import tolerance as conv_tolerance
from test_norm_gpu import value_tolerance
from test_sample_gpu import NEAR
from test_serve_example_gpu import example

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # a rounding to bf16


class Watch:
    def __init__(self, monkeypatch):
        self.calls = dict(conv=0, ssm=0, norm=0, sample=0)
        self.lengths, self.history = set(), {}
        for name in ("conv_packed", "ssm_packed", "rms_norm", "sample"):
            real = getattr(gdn, "gdn_" + name)
            monkeypatch.setattr(gdn, "gdn_" + name,
                                lambda *a, real=real, check=getattr(self, name), **k: check(real, *a, **k))

    def spans(self, req):
        cu, _, zero = req.tensors[:3]
        cu, zero = cu.tolist(), zero.tolist()
        return [(n, lo, hi, zero[n]) for n, (lo, hi) in enumerate(zip(cu, cu[1:]))]

    def conv_packed(self, real, h, cfg, req, x, xs, y, ys, pool, ckpt, status):
        old, xv = num(pool), num(x)
        real(h, cfg, req, x, xs, y, ys, pool, ckpt, status)
        w, b = (num(t) for t in cfg.tensors)
        got, new = num(y), num(pool)
        for n, lo, hi, zero in self.spans(req):
            want, mag, line = R.conv(xv[lo:hi], w, b, 1, old[n] * (1 - zero))
            assert (np.abs(got[lo:hi] - want) <= conv_tolerance(want, mag, HALF, 1)).all()
            np.testing.assert_array_equal(new[n], line[hi - lo:])
            self.lengths.add(hi - lo)
        self.calls["conv"] += 1

    def ssm_packed(self, real, h, cfg, req, rows, pool, *rest):
        old = num(pool)
        x, delta, b, c, z, y = (num(t) for t in rows.tensors)
        real(h, cfg, req, rows, pool, *rest)
        a, d, bias = (num(t) for t in cfg.tensors)
        got, new = num(rows.tensors[5]), num(pool)
        for n, lo, hi, zero in self.spans(req):
            want, hs, bound, es = R.ssm(x[lo:hi], delta[lo:hi], b[lo:hi, None], c[lo:hi, None],
                                        z[lo:hi], a, d, bias, True, old[n] * (1 - zero), 1)
            tol = 2 * bound  # long prompts are cut into segments
            assert (np.abs(got[lo:hi] - want) <= tol + (np.abs(want) + tol) * HALF + 1e-37).all()
            assert (np.abs(new[n] - hs[-1]) <= 2 * es[-1] + 1e-37).all()
        self.calls["ssm"] += 1

    def rms_norm(self, real, h, cfg, n, x, xs, residual=None, rs=0, sum=None, ss=0, **k):
        xv, rv = num(x), None if residual is None else num(residual)
        real(h, cfg, n, x, xs, residual, rs, sum, ss, **k)
        s, v = R.rms_norm(xv, rv, num(cfg.tensors[0]), 0.0, 1e-6, 1, None)
        tol = value_tolerance(v, None, np.abs(v) * 2.0 ** -23)
        if sum is not None:
            assert (np.abs(num(sum) - s) <= np.abs(s) * (HALF + 2.0 ** -24)).all()
        if k.get("y") is not None:
            assert (np.abs(num(k["y"]) - v) <= tol + (np.abs(v) + tol) * HALF).all()
        else:
            scale = num(k["scales"])
            top = np.abs(v).max(-1, keepdims=True)
            assert (np.abs(scale - top / 448) <= top / 448 * 2.0 ** -17).all()
            got = A.e4m3_values()[k["codes"].view(x.new_empty(0).byte().dtype).cpu().numpy()] * scale
            room = np.abs(v) * (2.0 ** -4 + 2.0 ** -22) + scale * 2.0 ** -10 + tol * 1.1
            assert (np.abs(got - v) <= room).all()
        self.calls["norm"] += 1

    def sample(self, real, h, io, n, vocab, logits, stride, t, k, p, m, u, token):
        real(h, io, n, vocab, logits, stride, t, k, p, m, u, token)
        l, got = num(logits), token.tolist()
        for i in range(n):
            want, _, gap = R.sample_row(l[i], float(t[i]), int(k[i]), float(p[i]), float(m[i]), float(u[i]))
            assert got[i] == want or gap < NEAR
        self.calls["sample"] += 1


def test_tokens_are_served(monkeypatch):
    torch = torch_cuda()
    handle()  # builds the library
    m = example()
    watch = Watch(monkeypatch)
    torch.manual_seed(4)
    server = m.Server(slots=3, num_pages=24, max_tokens=512, layers="SLSF", vocab=1009)
    prompts = [torch.randint(0, 1009, (n,), dtype=torch.int32, device="cuda")
               for n in (70, 1, 200, 130, 2)]
    last = m.serve(server, prompts, 4)
    assert all(x.shape == (1,) and 0 <= int(x) < 1009 for x in last)
    assert watch.calls["sample"] >= 10 and watch.calls["conv"] == watch.calls["ssm"] >= 20
    assert {0, 1, 70, 200} <= watch.lengths and watch.calls["norm"] >= 30
    assert int(server.pages.status.item()) == 0 and int(server.pages.count.item()) == 24
    server.close()


def test_rows_through_scan_layers_alone(monkeypatch):
    torch = torch_cuda()
    handle()
    m = example()
    watch = Watch(monkeypatch)
    torch.manual_seed(5)
    server = m.Server(slots=2, num_pages=24, max_tokens=1024, layers="SS")
    prompts = [torch.randn(n, m.HIDDEN, device="cuda").bfloat16() for n in (300, 3, 64)]
    last = m.serve(server, prompts, 3)
    assert all(torch.isfinite(x).all() for x in last) and watch.calls["ssm"] >= 8
    server.close()
