"""The short causal convolution against the plain fp64 reference."""
import numpy as np
import pytest

from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import IO, Pack, empty_rows, i32, num, rows, up

pytestmark = pytest.mark.gpu


def tolerance(want, mag, half, act):
    """width + 1 roundings of the terms' absolute values, silu (slope at most 1.1) with its own
    error of 2^-20 and an exponent's rounding, |v| 2^-22 of the result; then one rounding to the
    output (bf16: half a step of what is rounded)."""
    err = mag * 6 * 2.0 ** -24 * 1.1
    if act:
        err = err + np.abs(want) * (2.0 ** -20 + mag * 2.0 ** -22)
    return err + (np.abs(want) + err) * half + 1e-37


def case(rng, ch, width, io, bias):
    w = up(rng.standard_normal((ch, width)))
    b = up(rng.standard_normal(ch)) if bias else None
    return w, b


@pytest.mark.parametrize("lens", [[1], [70], [0, 1, 2, 3, 33, 64, 5, 0], [1] * 40, [32, 31, 97, 1],
                                  [200, 1, 1, 1], [0], [0, 0, 4]])
@pytest.mark.parametrize("ch,width,io,bias,act", [
    (8, 4, "bf16", False, 1), (1, 2, "bf16", True, 1), (1028, 4, "bf16", True, 0),
    (96, 3, "f32", True, 1), (515, 4, "f32", False, 1), (77, 2, "f32", True, 0),
    (2056, 4, "bf16", False, 1)])
def test_packed(lens, ch, width, io, bias, act):
    torch = torch_cuda()
    code, half = IO[io]
    rng = np.random.default_rng(sum(lens) * 31 + ch + width)
    p = Pack(rng, lens)
    w, b = case(rng, ch, width, io, bias)
    x, y = rows(rng, p.tokens, ch, io), empty_rows(p.tokens, ch, io)
    pool = up(rng.standard_normal((p.slots, width - 1, ch)), io)
    ckpt = torch.full((max(1, p.num_ckpt), width - 1, ch), 9.0, dtype=pool.dtype, device="cuda")
    old, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = gdn.make_conv_config(w, b, activation=act, io_dtype=code)
    gdn.gdn_conv_packed(handle(), cfg, p.requests, x, x.stride(0), y, y.stride(0), pool, ckpt,
                        status)
    torch.cuda.synchronize()
    assert status.item() == 0
    want_pool, xs, got = num(old), num(x), num(y)
    for n, (lo, hi) in enumerate(zip(p.cu, p.cu[1:])):
        state = num(old)[p.slot[n]] * (1 - p.zero[n])
        want, mag, line = R.conv(xs[lo:hi], num(w), None if b is None else num(b), act, state)
        err = np.abs(got[lo:hi] - want)
        assert (err <= tolerance(want, mag, half, act)).all()
        want_pool[p.slot[n]] = line[len(line) - (width - 1):]
        for j, pos in zip(range(p.ckpt_cu[n], p.ckpt_cu[n + 1]), p.pos[n]):
            np.testing.assert_array_equal(num(ckpt)[j], line[pos:pos + width - 1])
    np.testing.assert_array_equal(num(pool), want_pool)  # copies; other slots untouched
    assert (got[p.cu[-1]:] == 7).all()  # rows behind the last request


@pytest.mark.parametrize("io,tokens", [("bf16", 60_000), ("bf16", 130_000), ("bf16", 260_000),
                                       ("bf16", 500_000), ("f32", 45_000), ("f32", 190_000)])
def test_packed_in_blocks_of_more_rows(io, tokens):
    """Calls large enough for blocks of 64 to 512 rows, requests that end beside their borders."""
    rng = np.random.default_rng(tokens)
    lens = [63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1, 0, 3, 1024, 7000]
    lens += list(rng.integers(0, 4000, 2000))
    total = np.cumsum(lens)
    cut = int(np.searchsorted(total, tokens))
    test_packed([int(n) for n in lens[:cut]], 8, 4, io, True, 1)


@pytest.mark.parametrize("ch,width,io", [(8192, 4, "bf16"), (13, 3, "bf16"), (260, 4, "f32"),
                                         (5, 2, "f32")])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(ch, width, io, in_place):
    torch = torch_cuda()
    code, half = IO[io]
    rng = np.random.default_rng(ch)
    w, b = case(rng, ch, width, io, True)
    slot = np.array([4, -1, 0, 9, 2, 3, 10, -7])  # skipped rows; 10 is out of range
    x = rows(rng, 8, ch, io)
    y = x if in_place else empty_rows(8, ch, io)
    before, pool = num(x), up(rng.standard_normal((10, width - 1, ch)), io)
    old, status = num(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = gdn.make_conv_config(w, b, io_dtype=code)
    gdn.gdn_conv_step(handle(), cfg, 8, x, x.stride(0), y, y.stride(0), pool, 10, i32(slot), status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
    got = num(y)
    for r, s in enumerate(slot):
        if not 0 <= s < 10:
            assert (got[r] == (before[r] if in_place else 7)).all()
            continue
        want, mag, line = R.conv(before[r:r + 1], num(w), num(b), 1, old[s])
        assert (np.abs(got[r:r + 1] - want) <= tolerance(want, mag, half, 1)).all()
        old[s] = line[1:]
    np.testing.assert_array_equal(num(pool), old)


def test_a_prompt_in_pieces_and_by_tokens():
    """The same outputs and states, bit for bit, whole, in slices and token by token."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    ch, n = 520, 75
    w, _ = case(rng, ch, 4, "bf16", False)
    cfg = gdn.make_conv_config(w)
    x, whole = rows(rng, n, ch, "bf16"), empty_rows(n, ch, "bf16")
    pools = [torch.ones(1, 3, ch, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(lo, hi, y, pool):
        req = gdn.make_requests(i32([0, hi - lo]), hi - lo, hi - lo, 1)
        gdn.gdn_conv_packed(handle(), cfg, req, x[lo:hi], x.stride(0), y[lo:hi], y.stride(0), pool)
        torch.cuda.synchronize()

    run(0, n, whole, pools[0])
    parts, steps = empty_rows(n, ch, "bf16"), empty_rows(n, ch, "bf16")
    for lo, hi in [(0, 1), (1, 3), (3, 40), (40, 75)]:
        run(lo, hi, parts, pools[1])
    for t in range(n):
        gdn.gdn_conv_step(handle(), cfg, 1, x[t:], x.stride(0), steps[t:], steps.stride(0),
                          pools[2], 1, zero)
    torch.cuda.synchronize()
    for y, pool in ((parts, pools[1]), (steps, pools[2])):
        assert torch.equal(whole, y) and torch.equal(pools[0], pool)


def test_requests_out_of_range_are_left_out():
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    ch = 40
    w, _ = case(rng, ch, 4, "f32", False)
    cfg = gdn.make_conv_config(w, io_dtype=gdn.GDN_F32)
    x = rows(rng, 64, ch, "f32")
    pool = up(rng.standard_normal((6, 3, ch)))
    #            served  too long  backwards  past the rows  slot 6  skipped
    cu = i32([0, 10, 40, 30, 65, 50, 60])
    slot, bad = i32([1, 2, 3, 4, 6, -1]), i32([0, 2, 2, 2, 2, 2, 2])
    for ckpt_cu, expect in ((bad, None), (None, None)):
        y, status = empty_rows(64, ch, "f32"), torch.zeros(1, dtype=torch.int32, device="cuda")
        mine = pool.clone()
        ckpt = torch.full((2, 3, ch), 5.0, device="cuda")
        req = gdn.make_requests(cu, 64, 25, 6, slot_idx=slot, ckpt_cu=ckpt_cu,
                                ckpt_pos=i32([11, -3]), num_ckpt=2)
        gdn.gdn_conv_packed(handle(), cfg, req, x, x.stride(0), y, y.stride(0), mine, ckpt, status)
        torch.cuda.synchronize()
        assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
        assert (num(y)[10:] == 7).all() and (num(y)[:10] != 7).any()
        keep = [0, 2, 3, 4, 5]
        assert torch.equal(mine[keep], pool[keep]) and not torch.equal(mine[1], pool[1])
        assert (ckpt == 5).all()  # positions behind the request and below 1


def test_overlapping_requests_stay_within_the_arrays():
    """Rows that several requests name (cu out of order): more work than the call has blocks for;
    everything around the arrays stays as it was."""
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    ch, n = 24, 130
    w, _ = case(rng, ch, 4, "bf16", False)
    x, y = rows(rng, n, ch, "bf16"), empty_rows(n + 4, ch, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = torch.zeros(30, 3, ch, dtype=torch.bfloat16, device="cuda")
    req = gdn.make_requests(i32([0, n] * 15), n, n, 30)
    gdn.gdn_conv_packed(handle(), gdn.make_conv_config(w), req, x, x.stride(0), y, y.stride(0),
                        pool, None, status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
    assert (num(y)[n:] == 7).all()


def test_many_requests():
    """4,096 requests: every thread of a block counts several."""
    torch = torch_cuda()
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 4, 4096)
    lens[[17, 4095]] = 50, 70
    p = Pack(rng, lens, ckpt=False)
    w, _ = case(rng, 8, 4, "f32", False)
    x, y = rows(rng, p.tokens, 8, "f32"), empty_rows(p.tokens, 8, "f32")
    pool = up(rng.standard_normal((p.slots, 3, 8)))
    old = num(pool)
    gdn.gdn_conv_packed(handle(), gdn.make_conv_config(w, io_dtype=gdn.GDN_F32), p.requests, x,
                        x.stride(0), y, y.stride(0), pool)
    torch.cuda.synchronize()
    xs, got, wn = num(x), num(y), num(w)
    for n, (lo, hi) in enumerate(zip(p.cu, p.cu[1:])):
        state = old[p.slot[n]] * (1 - p.zero[n])
        want, mag, line = R.conv(xs[lo:hi], wn, None, 1, state)
        assert (np.abs(got[lo:hi] - want) <= tolerance(want, mag, 2.0 ** -24, 1)).all()
        old[p.slot[n]] = line[len(line) - 3:]
    np.testing.assert_array_equal(num(pool), old)
