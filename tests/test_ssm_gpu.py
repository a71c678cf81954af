"""The selective scan against the plain fp64 recurrence, within bounds that follow it."""
import numpy as np
import pytest

from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import IO, Pack, dtype, empty_rows, i32, num, rows, up

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, rng, ch, n, groups, io, gate=True, skip=True, bias=True, soft=True):
        self.ch, self.n, self.groups, self.io, self.gate, self.soft = ch, n, groups, io, gate, soft
        self.a = up(-(0.2 + rng.random((ch, n))) * np.arange(1, n + 1))
        self.d = up(rng.standard_normal(ch)) if skip else None
        self.bias = up(rng.uniform(-7, -1, ch)) if bias else None
        self.cfg = gdn.make_ssm_config(self.a, self.d, self.bias, num_groups=groups,
                                       delta_softplus=soft, io_dtype=IO[io][0])

    def inputs(self, rng, tokens):
        g = self.groups * self.n
        low = up(rng.standard_normal((tokens, 3 + 2 * g + 1)), self.io)  # b and c off boundaries
        delta = rows(rng, tokens, self.ch, self.io, scale=1.5)
        if not self.soft:
            delta.abs_()  # in place: the rows keep their stride
        return dict(x=rows(rng, tokens, self.ch, self.io), delta=delta, b=low[:, 3:3 + g],
                    c=low[:, 3 + g:3 + 2 * g],
                    z=rows(rng, tokens, self.ch, self.io, scale=2.0) if self.gate else None)

    def reference(self, t, lo, hi, state):
        f = lambda k: None if t[k] is None else num(t[k])[lo:hi]  # noqa: E731
        g = lambda k: f(k).reshape(hi - lo, self.groups, self.n)  # noqa: E731
        opt = lambda x: None if x is None else num(x)  # noqa: E731
        return R.ssm(f("x"), f("delta"), g("b"), g("c"), f("z"), num(self.a), opt(self.d),
                     opt(self.bias), self.soft, state, self.groups)


def run(layer, requests, t, y, pool, ckpt=None, status=None):
    torch = torch_cuda()
    n = gdn.gdn_ssm_workspace_size(layer.cfg, requests)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_packed(handle(), layer.cfg, requests, gdn.make_ssm_rows(y=y, **t), pool, ckpt,
                       work, n, status)
    torch.cuda.synchronize()
    return n


def check(layer, p, t, y, old, pool, ckpt, cut=0):
    """cut: a longer pass joins segments; their states pass through sums of dt and products that
    round a few times more, which `cut` roundings of the states' bounds stand for."""
    half = IO[layer.io][1]
    got, states, marks, pool_left = num(y), num(pool), num(ckpt), set(range(p.slots))
    for n, (lo, hi) in enumerate(zip(p.cu, p.cu[1:])):
        s = p.slot[n]
        pool_left.discard(s)
        state = num(old)[s] * (1 - p.zero[n])
        want, hs, bound, es = layer.reference(t, lo, hi, state)
        tol = bound * (1 + cut)
        assert (np.abs(got[lo:hi] - want) <= tol + (np.abs(want) + tol) * half + 1e-37).all()
        assert (np.abs(states[s] - hs[-1]) <= es[-1] * (1 + cut) + 1e-37).all()
        for j, pos in zip(range(p.ckpt_cu[n], p.ckpt_cu[n + 1]), p.pos[n]):
            assert (np.abs(marks[j] - hs[pos]) <= es[pos] * (1 + cut) + 1e-37).all()
    left = sorted(pool_left)
    np.testing.assert_array_equal(states[left], num(old)[left])
    assert (got[p.cu[-1]:] == 7).all()


@pytest.mark.parametrize("lens", [[1], [33], [0, 1, 2, 3, 31, 32, 65, 0], [1] * 20, [5, 120, 64]])
@pytest.mark.parametrize("ch,n,groups,io,kw", [
    (64, 16, 1, "bf16", {}), (40, 8, 2, "f32", {}), (130, 16, 1, "f32", dict(gate=False)),
    (7, 3, 1, "bf16", dict(skip=False)), (66, 10, 3, "bf16", dict(bias=False)),
    (48, 64, 2, "bf16", dict(gate=False)), (36, 128, 1, "f32", {}), (24, 30, 1, "f32", {}),
    (33, 4, 1, "bf16", dict(soft=False, bias=False)), (1, 1, 1, "f32", {}),
    (18, 101, 2, "bf16", {})])
def test_packed(lens, ch, n, groups, io, kw):
    torch = torch_cuda()
    rng = np.random.default_rng(sum(lens) * 7 + ch + n)
    p = Pack(rng, lens)
    layer = Layer(rng, ch, n, groups, io, **kw)
    t, y = layer.inputs(rng, p.tokens), empty_rows(p.tokens, ch, io)
    pool = up(rng.standard_normal((p.slots, ch, n)))
    ckpt = torch.zeros(max(1, p.num_ckpt), ch, n, device="cuda")
    old, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    run(layer, p.requests, t, y, pool, ckpt, status)
    assert status.item() == 0
    check(layer, p, t, y, old, pool, ckpt)


@pytest.mark.parametrize("lens,ch,n,groups,io", [
    ([700], 40, 16, 1, "f32"), ([300, 1, 0, 900, 128, 129], 24, 16, 1, "bf16"),
    ([1200, 640], 12, 40, 2, "bf16"), ([513], 9, 5, 1, "f32")])
def test_requests_cut_into_segments(lens, ch, n, groups, io):
    torch = torch_cuda()
    rng = np.random.default_rng(sum(lens))
    p = Pack(rng, lens)
    layer = Layer(rng, ch, n, groups, io)
    t, y = layer.inputs(rng, p.tokens), empty_rows(p.tokens, ch, io)
    pool = up(rng.standard_normal((p.slots, ch, n)))
    ckpt = torch.zeros(max(1, p.num_ckpt), ch, n, device="cuda")
    old, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert run(layer, p.requests, t, y, pool, ckpt, status) > 256  # the call is cut
    assert status.item() == 0
    # the joined decay exp(a sum dt) is off by its exponent's error, as the rows' own decays are
    # together, and by one ex2 and one rounding where they have one each
    check(layer, p, t, y, old, pool, ckpt, cut=1)
    again, pool2 = empty_rows(p.tokens, ch, io), old.clone()
    run(layer, p.requests, t, again, pool2, ckpt)
    assert torch.equal(again, y) and torch.equal(pool, pool2)


@pytest.mark.parametrize("ch,n,groups,io,kw", [
    (4096, 16, 1, "bf16", {}), (70, 8, 2, "f32", dict(gate=False)), (33, 3, 1, "bf16", {}),
    (20, 128, 1, "f32", {}), (64, 64, 2, "bf16", {}), (30, 21, 1, "f32", dict(skip=False)),
    (12, 32, 1, "bf16", dict(soft=False, bias=False))])
@pytest.mark.parametrize("over", [None, "x", "delta", "z"])
def test_step(ch, n, groups, io, kw, over):
    torch = torch_cuda()
    rng = np.random.default_rng(ch + n)
    layer = Layer(rng, ch, n, groups, io, **kw)
    slot = np.array([3, -1, 0, 6, 2, 7])
    t = layer.inputs(rng, 6)
    if over == "z" and not layer.gate:
        pytest.skip("no gate")
    before = {k: None if v is None else v.clone() for k, v in t.items()}
    y = empty_rows(6, ch, io) if over is None else t[over]
    pool = up(rng.standard_normal((7, ch, n)))
    old, status = num(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_ssm_step(handle(), layer.cfg, 6, gdn.make_ssm_rows(y=y, **t), pool, 7, i32(slot),
                     status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT  # slot 7
    got, states, half = num(y), num(pool), IO[io][1]
    for r, s in enumerate(slot):
        if not 0 <= s < 7:
            assert (got[r] == (7 if over is None else num(before[over])[r])).all()
            continue
        want, hs, bound, es = layer.reference(before, r, r + 1, old[s])
        assert (np.abs(got[r] - want[0]) <= bound[0] + (np.abs(want[0]) + bound[0]) * half + 1e-37).all()
        assert (np.abs(states[s] - hs[-1]) <= es[-1] + 1e-37).all()
    left = [s for s in range(7) if s not in slot]
    np.testing.assert_array_equal(states[left], old[left])


@pytest.mark.parametrize("over", ["x", "delta", "z"])
@pytest.mark.parametrize("lens,ch", [([40, 3, 100], 36), ([800], 16)])
def test_in_place(over, lens, ch):
    torch = torch_cuda()
    rng = np.random.default_rng(len(over))
    p = Pack(rng, lens, ckpt=False)
    layer = Layer(rng, ch, 20, 1, "bf16")
    t, y = layer.inputs(rng, p.tokens), empty_rows(p.tokens, ch, "bf16")
    pools = [up(rng.standard_normal((p.slots, ch, 20)))]
    pools.append(pools[0].clone())
    run(layer, p.requests, t, y, pools[0])
    run(layer, p.requests, t, t[over], pools[1])
    rows_ = p.cu[-1]
    assert torch.equal(t[over][:rows_], y[:rows_]) and torch.equal(*pools)


def test_a_prompt_in_pieces_and_by_tokens():
    torch = torch_cuda()
    rng = np.random.default_rng(11)
    layer = Layer(rng, 48, 16, 1, "f32")
    n = 90
    t = layer.inputs(rng, n)
    start = up(rng.standard_normal((1, 48, 16)))
    want, hs, bound, es = layer.reference(t, 0, n, num(start)[0])
    pools = [start.clone() for _ in range(3)]
    ys = [empty_rows(n, 48, "f32") for _ in range(3)]
    part = lambda lo, hi: {k: v[lo:hi] for k, v in t.items()}  # noqa: E731
    for pieces, pool, y in (([(0, n)], pools[0], ys[0]),
                            ([(0, 1), (1, 35), (35, 90)], pools[1], ys[1])):
        for lo, hi in pieces:
            req = gdn.make_requests(i32([0, hi - lo]), hi - lo, hi - lo, 1)
            run(layer, req, part(lo, hi), y[lo:hi], pool)
    for r in range(n):
        gdn.gdn_ssm_step(handle(), layer.cfg, 1,
                         gdn.make_ssm_rows(y=ys[2][r:r + 1], **part(r, r + 1)), pools[2], 1, i32([0]))
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(pools[0], pools[1])
    for y, pool in zip(ys, pools):
        assert (np.abs(num(y) - want) <= bound + (np.abs(want) + bound) * 2.0 ** -24).all()
        assert (np.abs(num(pool)[0] - hs[-1]) <= es[-1]).all()


def test_extreme_steps():
    """Steps from where softplus is all exponential to where it is the identity; decays of 0."""
    torch = torch_cuda()
    rng = np.random.default_rng(12)
    layer = Layer(rng, 64, 16, 1, "f32", bias=False)
    t = layer.inputs(rng, 64)
    t["delta"].copy_(torch.linspace(-30, 60, 64, device="cuda")[torch.randperm(64)][None].T.expand(64, 64))
    y, pool = empty_rows(64, 64, "f32"), up(rng.standard_normal((1, 64, 16)))
    old = num(pool)
    run(layer, gdn.make_requests(i32([0, 64]), 64, 64, 1), t, y, pool)
    want, hs, bound, es = layer.reference(t, 0, 64, old[0])
    assert (np.abs(num(y) - want) <= bound + (np.abs(want) + bound) * 2.0 ** -24 + 1e-30).all()
    assert (np.abs(num(pool)[0] - hs[-1]) <= es[-1] + 1e-30).all()


def test_inputs_that_are_not_finite_stay_in_their_channel():
    torch = torch_cuda()
    rng = np.random.default_rng(13)
    layer = Layer(rng, 40, 20, 1, "bf16")
    req = gdn.make_requests(i32([0, 30, 60]), 60, 30, 2)
    t = layer.inputs(rng, 60)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        u = {k: v.clone() for k, v in t.items()}
        if bad is not None:
            u["x"][4, 3] = bad
            u["delta"][7, 11] = bad
            u["z"][2, 20] = bad
        y, pool = empty_rows(60, 40, "bf16"), torch.zeros(2, 40, 20, device="cuda")
        run(layer, req, u, y, pool)
        outs.append((y, pool))
    clean = [c for c in range(40) if c not in (3, 11, 20)]
    for y, pool in outs[1:]:
        assert torch.equal(y[:, clean], outs[0][0][:, clean])
        assert torch.equal(y[30:], outs[0][0][30:])
        assert torch.equal(pool[1], outs[0][1][1]) and torch.equal(pool[0, clean], outs[0][1][0, clean])


@pytest.mark.parametrize("rows_,max_len", [(64, 25), (3000, 1500)])
def test_requests_out_of_range_are_left_out(rows_, max_len):
    """The second shape is cut into segments."""
    torch = torch_cuda()
    rng = np.random.default_rng(14)
    layer = Layer(rng, 8, 16, 1, "f32")
    t = layer.inputs(rng, rows_)
    pool = up(rng.standard_normal((6, 8, 16)))
    k = max_len
    #         served    too long     backwards  past the rows  slot 6     skipped
    cu = i32([0, k // 2, k // 2 + k + 1, 10, rows_ + 1, 20, 40])
    y, status = empty_rows(rows_, 8, "f32"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mine, ckpt = pool.clone(), torch.full((2, 8, 16), 5.0, device="cuda")
    req = gdn.make_requests(cu, rows_, max_len, 6, slot_idx=i32([1, 2, 3, 4, 6, -1]),
                            ckpt_cu=i32([0, 2, 2, 2, 2, 2, 2]), ckpt_pos=i32([max_len, 0]), num_ckpt=2)
    run(layer, req, t, y, mine, ckpt, status)
    assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
    want, hs, bound, es = layer.reference(t, 0, k // 2, num(pool)[1])
    tol = 2 * bound + np.abs(want) * 2.0 ** -23
    assert (np.abs(num(y)[:k // 2] - want) <= tol).all() and (num(y)[k // 2:] == 7).all()
    keep = [0, 2, 3, 4, 5]
    assert torch.equal(mine[keep], pool[keep]) and not torch.equal(mine[1], pool[1])
    assert (ckpt == 5).all()


def test_overlapping_requests_stay_within_the_workspace():
    torch = torch_cuda()
    rng = np.random.default_rng(15)
    layer = Layer(rng, 8, 16, 1, "bf16")
    n = 1000
    t, y = layer.inputs(rng, n), empty_rows(n + 4, 8, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = torch.zeros(20, 8, 16, device="cuda")
    req = gdn.make_requests(i32([0, n] * 10), n, n, 20)
    size = gdn.gdn_ssm_workspace_size(layer.cfg, req)
    assert size > 256
    work = torch.full((size + 1024,), 3, dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_packed(handle(), layer.cfg, req, gdn.make_ssm_rows(y=y, **t), pool, None, work,
                       size, status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
    assert (num(y)[n:] == 7).all() and (work[size:] == 3).all()


def test_replayed_from_a_graph_with_other_lengths():
    """A captured pass reads lengths, slots and flags when it runs."""
    torch = torch_cuda()
    rng = np.random.default_rng(16)
    layer = Layer(rng, 24, 16, 1, "f32")
    rows_, b = 700, 3
    t, y = layer.inputs(rng, rows_), empty_rows(rows_, 24, "f32")
    pool = up(rng.standard_normal((4, 24, 16)))
    cu, slot, zero = i32([0, 0, 0, 0]), i32([-1] * 3), i32([0] * 3)
    req = gdn.make_requests(cu, rows_, 600, 4, slot_idx=slot, start_zero=zero)
    n = gdn.gdn_ssm_workspace_size(layer.cfg, req)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    rec = gdn.make_ssm_rows(y=y, **t)
    h, s = handle(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gdn.gdn_ssm_packed(h, layer.cfg, req, rec, pool, None, work, n, None, s)
    for lens, slots in (([600, 3, 97], [3, 0, 1]), ([1, 1, 1], [2, 1, 0]), ([0, 500, 0], [1, 3, 2])):
        cu.copy_(i32(np.concatenate([[0], np.cumsum(lens)])))
        slot.copy_(i32(slots))
        zero.copy_(i32([1, 0, 0]))
        y.fill_(7.0)
        old = num(pool)
        g.replay()
        torch.cuda.synchronize()
        lo = 0
        for k, (m, sl) in enumerate(zip(lens, slots)):
            want, hs, bound, es = layer.reference(t, lo, lo + m, old[sl] * (k != 0))
            tol = 2 * bound + np.abs(want) * 2.0 ** -23
            assert (np.abs(num(y)[lo:lo + m] - want) <= tol).all()
            assert (np.abs(num(pool)[sl] - hs[-1]) <= 2 * es[-1]).all()
            lo += m
        assert (num(y)[lo:] == 7).all()
    assert b == 3 and dtype("f32") == y.dtype
