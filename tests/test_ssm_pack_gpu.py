"""The selective scan: what a request's results and a call's workspace owe to the calls around them."""
import numpy as np
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from oracle import step_ref as R
from step_util import IO, Pack, empty_rows, i32, num, up
from test_ssm_gpu import Layer, run

pytestmark = pytest.mark.gpu


def test_one_workspace_for_every_step():
    """Sized for the largest call, used by smaller ones, which are cut where that one is not."""
    torch = torch_cuda()
    rng = np.random.default_rng(31)
    layer = Layer(rng, 2048, 16, 1, "bf16")
    most = 12 * 600
    t = layer.inputs(rng, most)
    size = gdn.gdn_ssm_workspace_size(layer.cfg, gdn.make_requests(i32([0] * 13), most, 600, 12))
    work = torch.zeros(size + 512, dtype=torch.uint8, device="cuda")
    start = up(rng.standard_normal((12, 2048, 16)))
    for lens, rows, max_len in (([600] * 12, most, 600), ([600], 600, 600), ([600, 1, 500], most, 600),
                                ([130], most, 130), ([1] * 12, 12, 600), ([300] * 3, 900, 300)):
        req = gdn.make_requests(i32(np.concatenate([[0], np.cumsum(lens)])), rows, max_len, 12)
        part = {k: v[:rows] for k, v in t.items()}
        ys, pools = [empty_rows(rows, 2048, "bf16") for _ in range(2)], [start.clone() for _ in range(2)]
        work.fill_(255)  # NaN, and a mark behind the end
        gdn.gdn_ssm_packed(handle(), layer.cfg, req, gdn.make_ssm_rows(y=ys[0], **part), pools[0], None,
                           work, size)
        run(layer, req, part, ys[1], pools[1])
        assert torch.equal(*ys) and torch.equal(*pools) and (work[size:] == 255).all()
        assert torch.isfinite(pools[0]).all()


@pytest.mark.parametrize("single", [False, True])
def test_steps_of_far_inputs_keep_their_precision(single):
    """dt alone: one state that starts from 0, x = b = 1. 2^-20 of itself: 2^-22 from ex2, 2^-22 from the
    constant ln 2 at 87 and seven roundings of 2^-24."""
    torch = torch_cuda()
    n = 16384
    v = np.concatenate([np.linspace(-87, 40, n - 4), [-np.inf, np.inf, np.nan, -1e30]])
    delta = up(v[None])
    ones, low = torch.ones(1, n, device="cuda"), torch.ones(1, 1, device="cuda")
    cfg = gdn.make_ssm_config(-torch.ones(n, 1, device="cuda"), io_dtype=gdn.GDN_F32)
    y, pool = torch.empty(1, n, device="cuda"), torch.zeros(1, n, 1, device="cuda")
    rows = gdn.make_ssm_rows(ones, delta, low, low, y)
    if single:
        gdn.gdn_ssm_step(handle(), cfg, 1, rows, pool, 1, i32([0]))
    else:
        req = gdn.make_requests(i32([0, 1]), 1, 1, 1)
        size = gdn.gdn_ssm_workspace_size(cfg, req)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        gdn.gdn_ssm_packed(handle(), cfg, req, rows, pool, None, work, size)
    torch.cuda.synchronize()
    for got in (num(pool)[0, :, 0], num(y)[0]):
        want = np.logaddexp(num(delta)[0, :-4], 0.0)
        rel = np.abs(got[:-4] - want) / want
        assert rel.max() <= 2.0 ** -20, np.log2(rel.max())
        assert got[-4] == 0 and np.isnan(got[-2]) and got[-1] == 0
        assert not np.isfinite(got[-3])  # an infinite step spoils its channel


class Some:
    """The fp64 reference of a few channels of a wide layer (one group)."""

    def __init__(self, rng, layer, t, count):
        self.at = np.sort(rng.choice(layer.ch, count, replace=False))
        self.layer, self.t = layer, {k: None if v is None else num(v[:, self.at] if k in "xz" or k == "delta" else v)
                                     for k, v in t.items()}

    def __call__(self, lo, hi, state):
        t, y = self.t, self.layer
        part = lambda k: None if t[k] is None else t[k][lo:hi]  # noqa: E731
        opt = lambda w: None if w is None else num(w)[self.at]  # noqa: E731
        return R.ssm(part("x"), part("delta"), part("b")[:, None], part("c")[:, None], part("z"),
                     num(y.a)[self.at], opt(y.d), opt(y.bias), y.soft, state, 1)


WIDE = [50 + 5 * (i % 3) for i in range(24)]  # 4,096 channels of them fill the GPU: 16 states a thread


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [16, 11])
def test_a_request_alone_and_among_others(io, n):
    """The same bits whichever plan the pack around it leads to: alone two lanes share a channel's
    states, among 24 one thread has them."""
    torch = torch_cuda()
    rng = np.random.default_rng(n)
    ch = 4096
    layer = Layer(rng, ch, n, 1, io)
    cu = np.concatenate([[0], np.cumsum(WIDE)])
    rows = int(cu[-1])
    t = layer.inputs(rng, rows)
    start = up(rng.standard_normal((24, ch, n)))
    pools, ys = [start.clone() for _ in range(2)], [empty_rows(rows, ch, io) for _ in range(2)]
    run(layer, gdn.make_requests(i32(cu), rows, 60, 24), t, ys[0], pools[0])
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        req = gdn.make_requests(i32([0, hi - lo]), int(hi - lo), int(hi - lo), 1)
        run(layer, req, {k: v[lo:hi] for k, v in t.items()}, ys[1][lo:hi], pools[1][i:i + 1])
    assert torch.equal(*pools) and torch.equal(*ys)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
def test_a_pack_that_fills_the_gpu(io, gate):
    """24 ragged requests of 4,096 channels, with slots, zero starts and checkpoints."""
    torch = torch_cuda()
    rng = np.random.default_rng(33)
    ch = 4096
    p = Pack(rng, WIDE[:22] + [1, 0] + WIDE[:3], max_len=60)
    layer = Layer(rng, ch, 16, 1, io, gate=gate)
    t, y = layer.inputs(rng, p.tokens), empty_rows(p.tokens, ch, io)
    pool, ckpt = up(rng.standard_normal((p.slots, ch, 16))), torch.zeros(max(1, p.num_ckpt), ch, 16, device="cuda")
    old, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    run(layer, p.requests, t, y, pool, ckpt, status)
    assert status.item() == 0
    some = Some(rng, layer, t, 24)
    half, got = IO[io][1], num(y)[:, some.at]
    states, marks, old = (num(s[:, some.at]) for s in (pool, ckpt, old))
    for n, (lo, hi) in enumerate(zip(p.cu, p.cu[1:])):
        want, hs, bound, es = some(lo, hi, old[p.slot[n]] * (1 - p.zero[n]))
        assert (np.abs(got[lo:hi] - want) <= bound + (np.abs(want) + bound) * half + 1e-37).all()
        assert (np.abs(states[p.slot[n]] - hs[-1]) <= es[-1] + 1e-37).all()
        for j, pos in zip(range(p.ckpt_cu[n], p.ckpt_cu[n + 1]), p.pos[n]):
            assert (np.abs(marks[j] - hs[pos]) <= es[pos] + 1e-37).all()
    left = [s for s in range(p.slots) if s not in p.slot]
    np.testing.assert_array_equal(states[left], old[left])
    assert (num(y)[p.cu[-1]:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_long_prompt_of_many_channels(io):
    """Cut into segments of 96 rows that fill the GPU: 16 states a thread; checkpoints in several of
    them and at their borders."""
    torch = torch_cuda()
    rng = np.random.default_rng(34)
    ch, n = 2048, 4096
    layer = Layer(rng, ch, 16, 1, io)
    t, y = layer.inputs(rng, n), empty_rows(n, ch, io)
    pos = [1, 95, 96, 97, 960, 2500, 4031, 4032, 4096]
    start = up(rng.standard_normal((1, ch, 16)))
    pool, ckpt = start.clone(), torch.zeros(len(pos), ch, 16, device="cuda")
    req = gdn.make_requests(i32([0, n]), n, n, 1, ckpt_cu=i32([0, len(pos)]), ckpt_pos=i32(pos),
                            num_ckpt=len(pos))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert run(layer, req, t, y, pool, ckpt, status) > 256 and status.item() == 0
    some = Some(rng, layer, t, 24)
    want, hs, bound, es = some(0, n, num(start)[0, some.at])
    tol = 2 * bound  # as where few channels are cut
    assert (np.abs(num(y)[:, some.at] - want) <= tol + (np.abs(want) + tol) * IO[io][1] + 1e-37).all()
    for got, at in zip(num(ckpt[:, some.at]), pos):
        assert (np.abs(got - hs[at]) <= 2 * es[at] + 1e-37).all()
    assert (np.abs(num(pool)[0, some.at] - hs[-1]) <= 2 * es[-1] + 1e-37).all()
    again, pool2 = empty_rows(n, ch, io), start.clone()
    run(layer, req, t, again, pool2, torch.zeros_like(ckpt))
    assert torch.equal(again, y) and torch.equal(pool, pool2)


@pytest.mark.parametrize("ch", [64, 2048])
def test_a_bound_of_the_lengths_that_says_nothing(ch):
    """max_len at its largest: the segments it leads to are longer than the requests, which run whole."""
    torch = torch_cuda()
    rng = np.random.default_rng(35)
    layer = Layer(rng, ch, 16, 1, "bf16")
    cu, rows = i32([0, 50, 51, 110]), 110
    t, start = layer.inputs(rng, rows), up(rng.standard_normal((3, ch, 16)))
    pools, ys = [start.clone() for _ in range(2)], [empty_rows(rows, ch, "bf16") for _ in range(2)]
    for max_len, y, pool in zip((59, 2 ** 31 - 1), ys, pools):
        run(layer, gdn.make_requests(cu, rows, max_len, 3), t, y, pool)
    assert torch.equal(*pools) and torch.equal(*ys)
