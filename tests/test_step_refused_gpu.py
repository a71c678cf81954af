"""A step planned on the device: the requests that there are no pages for keep their recurrent states."""
import numpy as np
import pytest

from oracle import step_ref as R
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import i32, num, up

pytestmark = pytest.mark.gpu


def test_requests_refused_by_the_plan_keep_their_states():
    """Plan, convolution and scan from one graph; slots follow kv_len. The third request finds the stack
    empty in the first step and is served in the second."""
    torch = torch_cuda()
    rng = np.random.default_rng(41)
    h, page, ch, n, rows, seqs = handle(), 16, 48, 16, 64, 3
    ctx, new = i32([5, 0, 16]), i32([1, 30, 3])
    table = torch.full((seqs, 8), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[2, 0] = 7, 6
    free, count = i32(list(range(6)) + [0, 0]), i32([2])
    left, cu, kv_len = i32([0]), i32([0] * 4), i32([0] * 3)
    places = torch.empty(rows, dtype=torch.int64, device="cuda")
    status, slots = i32([0]), i32([0] * 3)
    conv = gdn.make_conv_config(up(rng.standard_normal((ch, 4))), io_dtype=gdn.GDN_F32)
    a = up(-rng.random((ch, n)))
    scan = gdn.make_ssm_config(a, io_dtype=gdn.GDN_F32)
    x, delta, low = (up(rng.standard_normal((rows, k))) for k in (ch, ch, 2 * n))
    c, y = torch.zeros(rows, ch, device="cuda"), torch.zeros(rows, ch, device="cuda")
    inputs, states = up(rng.standard_normal((seqs, 3, ch))), up(rng.standard_normal((seqs, ch, n)))
    req = gdn.make_requests(cu, rows, 40, seqs, slot_idx=slots)
    record = gdn.make_ssm_rows(c, delta, low[:, :n], low[:, n:], y)
    size = gdn.gdn_ssm_workspace_size(scan, req)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    order = torch.arange(seqs, dtype=torch.int32, device="cuda")

    def step(s):
        gdn.gdn_kv_plan(h, page, seqs, rows, ctx, new, table, 8, 8, free, count, left, cu, kv_len, None,
                        places, status, s)
        slots.copy_(torch.where(kv_len > 0, order, torch.full_like(order, -1)))
        gdn.gdn_conv_packed(h, conv, req, x, ch, c, ch, inputs, None, status, s)
        gdn.gdn_ssm_packed(h, scan, req, record, states, None, work, size, status, s)

    before = num(inputs), num(states)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for served in ([0, 1], [2]):
        graph.replay()
        torch.cuda.synchronize()
        assert [b for b in range(3) if kv_len[b] > 0] == [b for b in range(3) if b in served or new[b] == 0]
        assert status.item() == (gdn.GDN_ERR_POOL_EXHAUSTED if served == [0, 1] else 0)
        xs, ds, lo_ = num(x), num(delta), num(low)
        got = num(inputs), num(states)
        for b in range(seqs):
            if b not in served:
                np.testing.assert_array_equal(got[0][b], before[0][b])
                np.testing.assert_array_equal(got[1][b], before[1][b])
                continue
            r = slice(int(cu[b]), int(cu[b + 1]))
            _, _, line = R.conv(xs[r], num(conv.tensors[0]), None, 1, before[0][b])
            np.testing.assert_array_equal(got[0][b], line[-3:])
            _, hs, _, es = R.ssm(num(c)[r], ds[r], lo_[r, None, :n], lo_[r, None, n:], None, num(a), None,
                                 None, True, before[1][b], 1)
            assert (np.abs(got[1][b] - hs[-1]) <= es[-1] + 1e-37).all()
        before = got
        ctx.copy_(torch.where(kv_len > 0, kv_len, ctx))
        new.copy_(i32([0, 0, 3]))
        count.copy_(i32([2]))
        status.zero_()
