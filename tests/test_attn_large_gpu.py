"""Offsets past 32 bits: a cache whose last pages lie beyond 4 GiB, and rows of q, k, v and o
that do. Few tokens, so that the plain reference stays small."""
import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu


def _attend(torch, case, cache, table, q, q_stride, o, o_stride):
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cfg = gdn.make_attn_config(case.hq, scale=case.scale)
    n, mq, mk = len(case.q_len), max(case.q_len), max(case.kv_len)
    size = gdn.gdn_attn_workspace_size(cfg, cache, n, case.tokens, mq, mk)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    lse = torch.full((case.tokens, case.hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_paged(handle(), cfg, cache, n, case.tokens, mq, mk, up(case.cu),
                       up(np.asarray(case.kv_len, np.int32)), up(table), table.shape[1], q,
                       q_stride, o, o_stride, lse, work, size, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return lse.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("q_len,kv_len", [([1, 3], [300, 65]), ([200, 1], [400, 64])])
def test_pages_beyond_four_gib(q_len, kv_len):
    torch = torch_cuda()
    hq, hkv, dim, page, pages = 8, 4, 256, 128, 34000
    assert pages * hkv * page * dim > 1 << 32 and pages * hkv * page <= (1 << 31) - 1
    c = Case(5, q_len, kv_len, hq, hkv, dim, page)
    first = pages - c.pages
    big = [torch.empty(pages, hkv, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.ones(pages, hkv, device="cuda") for _ in range(2)]
    for j in range(2):
        big[j][first:].copy_(torch.from_numpy(c.codes[j]))
        scale[j][first:].copy_(torch.from_numpy(c.scales[j]))
    cache = gdn.make_kv_cache(*big, *scale)
    table = np.where(c.table >= 0, c.table + first, -1).astype(np.int32)
    q = torch.from_numpy(c.q).cuda().bfloat16()
    c.q64 = q.double().cpu().numpy()
    o = torch.empty_like(q)
    lse = _attend(torch, c, cache, table, q, hq * dim, o, hq * dim)
    c.compare(o.double().cpu().numpy(), lse)
    # and the append: a page's first tokens, then more behind them
    rng = np.random.default_rng(6)
    k, v = (rng.standard_normal((70, hkv, dim)).astype(np.float32) for _ in range(2))
    k, v = (torch.from_numpy(x).cuda().bfloat16() for x in (k, v))
    slots = (np.arange(70) + (pages - 1) * page).astype(np.int64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lo, hi in ((0, 40), (40, 70)):
        gdn.gdn_kv_append(handle(), cache, gdn.GDN_BF16, hi - lo,
                          torch.from_numpy(slots[lo:hi].copy()).cuda(), k[lo:hi], hkv * dim,
                          v[lo:hi], hkv * dim, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    zero = np.zeros((1, hkv, page, dim), np.uint8)
    one = np.ones((1, hkv), np.float32)
    want = [zero, zero, one, one]
    for lo, hi in ((0, 40), (40, 70)):
        want = A.append(want[0], want[1], want[2], want[3], slots[lo:hi] - (pages - 1) * page,
                        k[lo:hi].double().cpu().numpy(), v[lo:hi].double().cpu().numpy())
    values = A.e4m3_values()
    for j in range(2):
        np.testing.assert_array_equal(scale[j][-1:].double().cpu().numpy(), want[2 + j])
        np.testing.assert_array_equal(values[big[j][-1, :, :70].cpu().numpy()],
                                      values[want[j][0][:, :70]])


@pytest.mark.parametrize("q_len", [[1, 3, 2], [120, 1, 90]])
def test_rows_beyond_four_gib(q_len):
    torch = torch_cuda()
    hq, hkv, dim, page = 4, 2, 64, 32
    c = Case(7, q_len, [n + 40 for n in q_len], hq, hkv, dim, page)
    row = hq * dim
    stride = ((1 << 32) // (c.tokens - 1) // 8 + 1) * 8  # elements of 2 bytes: the last row at 8 GiB
    wide = torch.empty((c.tokens - 1) * stride + 2 * row, dtype=torch.bfloat16, device="cuda")
    q = wide[:(c.tokens - 1) * stride + row].as_strided((c.tokens, row), (stride, 1))
    o = wide[row:].as_strided((c.tokens, row), (stride, 1))
    q.copy_(torch.from_numpy(c.q).cuda().bfloat16().view(c.tokens, row))
    c.q64 = q.double().cpu().numpy().reshape(c.tokens, hq, dim)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    codes, scales = [up(x) for x in c.codes], [up(x) for x in c.scales]
    cache = gdn.make_kv_cache(*codes, *scales)
    lse = _attend(torch, c, cache, c.table, q, stride, o, stride)
    c.compare(o.double().cpu().numpy().reshape(c.tokens, hq, dim), lse)
    # rotation and append from rows as far apart (k where o was)
    pos = np.arange(c.tokens, dtype=np.int32)[None] * 1000
    rope = gdn.gdn_rope_init(dim, dim, [dim // 2])
    k = o[:, :hkv * dim]
    k64 = k.double().cpu().numpy().reshape(c.tokens, hkv, dim)
    slots = np.arange(c.tokens, dtype=np.int64)
    fresh = [torch.zeros(-(-c.tokens // page), hkv, page, dim, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    size = [torch.ones(fresh[0].shape[0], hkv, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(handle(), gdn.make_kv_cache(*fresh, *size), gdn.GDN_BF16, c.tokens, up(slots),
                      k, stride, k, stride, rope, up(pos), c.tokens, q, stride, hq, q, stride,
                      status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    turned = A.rope(c.q64, pos, dim, [dim // 2], False, False, 10000.0)
    got = q.double().cpu().numpy().reshape(c.tokens, hq, dim)
    assert (np.abs(got - turned) <= np.abs(turned) * 2.0 ** -8
            + np.abs(c.q64).max() * 2.0 ** -20).all()
    values = A.e4m3_values()
    v = np.concatenate([values[x.cpu().numpy()] * s.double().cpu().numpy()[:, :, None, None]
                        for x, s in [(fresh[1], size[1])]])
    s = size[1].double().cpu().numpy()
    for t in range(c.tokens):
        p, at = divmod(t, page)
        want = k64[t]
        assert (np.abs(v[p, :, at] - want) <= np.abs(want) * 2.0 ** -4
                + s[p][:, None] * 2.0 ** -10).all()
