"""Ranges of requests that are out of order or out of the arrays: rows in front of and behind
the call's rows, and rows of no request, are neither read nor written."""
import numpy as np
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu

GUARD = 8  # rows of q, o and lse on either side of the call's


def _run_between_guards(torch, c, cu, max_q):
    t, code = (torch.bfloat16, gdn.GDN_BF16) if c.io == "bf16" else (torch.float32, gdn.GDN_F32)
    row, n = c.hq * c.dim, len(c.q_len)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = torch.full((c.tokens + 2 * GUARD, row), float("nan"), dtype=t, device="cuda")
    q[GUARD:-GUARD] = up(c.q).to(t).view(c.tokens, row)
    o = torch.full_like(q, 5.0)
    lse = torch.full((c.tokens + 2 * GUARD, c.hq), 7.0, device="cuda")
    codes, scales = [up(x) for x in c.codes], [up(x) for x in c.scales]
    cache = gdn.make_kv_cache(*codes, *scales)
    cfg = gdn.make_attn_config(c.hq, scale=c.scale, causal=c.causal, io_dtype=code)
    size = gdn.gdn_attn_workspace_size(cfg, cache, n, c.tokens, max_q, max(c.kv_len))
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_paged(handle(), cfg, cache, n, c.tokens, max_q, max(c.kv_len),
                       up(np.asarray(cu, np.int32)), up(np.asarray(c.kv_len, np.int32)),
                       up(c.table), c.table.shape[1], q[GUARD:], row, o[GUARD:], row, lse[GUARD:],
                       work, size, status)
    torch.cuda.synchronize()
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARGUMENT
    for x, v in ((o, 5), (lse, 7)):
        assert (x[:GUARD] == v).all() and (x[-GUARD:] == v).all()
    return o[GUARD:-GUARD].float(), lse[GUARD:-GUARD]


@pytest.mark.parametrize("io,lengths,max_q", [("bf16", [1, 3, 2], 3), ("f32", [1, 3, 2], 3),
                                              ("bf16", [100, 200, 150], 200)])
def test_ends_far_out_of_range(io, lengths, max_q):
    torch = torch_cuda()
    c = Case(31, lengths, [n + 50 for n in lengths], 8, 2, 128, 16, io)
    n = c.tokens
    for cu in ([2**31 - 1, -2**31, 4, n], [n, -2**31, -2**31, -2**31], [5, -2**31, n, -2**31 + 4],
               [-2**31, -2**31, 2**31 - 1, -2**31], [n, n + 1, 2**31 - 1, -1]):
        o, lse = _run_between_guards(torch, c, cu, max_q)
        inside = np.zeros(n, bool)
        for r0, r1 in zip(cu, cu[1:]):
            r0 = min(max(r0, 0), n)
            inside[r0:min(max(min(r1, n) - r0, 0), max_q) + r0] = True
        outside = torch.from_numpy(~inside).cuda()
        assert (o[outside] == 5).all() and (lse[outside] == 7).all()
        assert torch.isfinite(o).all()  # the guard rows of q are NaN


def test_overlapping_requests_that_ask_for_too_much():
    """2,048 requests, each over all rows of the call: their work items pass 32 bits. Nothing is
    computed, the status is raised, and the next call is right."""
    torch = torch_cuda()
    seqs, tokens, hq, dim, page, kv = 4096, 2304, 16, 64, 16, 65536
    i32 = dict(dtype=torch.int32, device="cuda")
    codes = [torch.zeros(4, 1, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(4, 1, device="cuda") for _ in range(2)]
    cache = gdn.make_kv_cache(*codes, *scales)
    cfg = gdn.make_attn_config(hq, scale=1.0, io_dtype=gdn.GDN_F32)
    cu = torch.zeros(seqs + 1, **i32)
    cu[1::2] = tokens
    table = torch.zeros(seqs, kv // page, **i32)
    kv_len = torch.full((seqs,), kv, **i32)
    q = torch.zeros(tokens, hq * dim, device="cuda")
    o = torch.full_like(q, 5.0)
    size = gdn.gdn_attn_workspace_size(cfg, cache, seqs, tokens, tokens, kv)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, **i32)
    gdn.gdn_attn_paged(handle(), cfg, cache, seqs, tokens, tokens, kv, cu, kv_len, table,
                       kv // page, q, hq * dim, o, hq * dim, None, work, size, status)
    torch.cuda.synchronize()
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert (o == 5).all()
    Case(32, [3, 40], [100, 40], 8, 2, 64, 16, "f32").check(torch)
