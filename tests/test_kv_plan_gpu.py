"""The step plan (pages, slots, positions) and the return of pages against the plain
reference: whole numbers, so every output is equal."""
import numpy as np
import pytest

from oracle import attn_ref as A
from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu


def _case(seed, seqs, page, ctx_hi, new_hi, *, short=0, pad=5, extra_blocks=2):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, seqs)
    new = rng.integers(0, new_hi + 1, seqs)
    have = [A.ceil_div(int(c), page) for c in ctx]
    need = sum(A.ceil_div(int(c + n), page) - h for c, n, h in zip(ctx, new, have))
    width = max(A.ceil_div(int(c + n), page) for c, n in zip(ctx, new)) + extra_blocks
    count = max(0, need + (7 if not short else -short))
    num_pages = sum(have) + max(count, 1) + 3
    ids = rng.permutation(num_pages)
    table = np.full((seqs, width), -1, np.int32)
    at = 0
    for b in range(seqs):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.full(num_pages, -7, np.int32)
    free[:count] = ids[at:at + count]
    return ctx, new, table, free, count, int(new.sum()) + pad, num_pages


def _run(torch, ctx, new, table, free, count, page, tokens, num_pages, in_place=False,
         positions=True):
    up = lambda x, t: torch.from_numpy(np.ascontiguousarray(x, t)).cuda()  # noqa: E731
    n = len(ctx)
    d = dict(ctx=up(ctx, np.int32), new=up(new, np.int32), table=up(table, np.int32),
             free=up(free, np.int32), count=up([count], np.int32))
    poison = lambda *s, dt=torch.int32: torch.full(s, -99, dtype=dt, device="cuda")  # noqa: E731
    out = d["count"] if in_place else poison(1)
    cu, kv, pos = poison(n + 1), poison(n), poison(max(tokens, 1))
    slots = poison(max(tokens, 1), dt=torch.int64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_plan(handle(), page, n, tokens, d["ctx"], d["new"], d["table"], table.shape[1],
                    num_pages, d["free"], d["count"], out, cu, kv, pos if positions else None,
                    slots, status)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(d["free"].cpu().numpy(), free)
    return (d["table"].cpu().tolist(), cu.cpu().tolist(), kv.cpu().tolist(),
            pos.cpu().tolist()[:tokens] if positions else None, slots.cpu().tolist()[:tokens],
            int(out.item()), int(status.item()))


@pytest.mark.parametrize("seed,seqs,page,ctx_hi,new_hi", [
    (0, 1, 16, 0, 1), (1, 1, 64, 100, 300), (2, 3, 16, 50, 1), (3, 37, 32, 500, 40),
    (4, 256, 64, 8192, 1), (5, 1000, 16, 64, 33), (6, 1025, 128, 300, 3), (7, 4096, 16, 40, 5),
    (8, 5, 128, 1000, 20000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_reference(seed, seqs, page, ctx_hi, new_hi, in_place):
    torch = torch_cuda()
    case = _case(seed, seqs, page, ctx_hi, new_hi)
    ctx, new, table, free, count, tokens, pages = case
    want = A.plan(ctx, new, table, free, count, page, tokens, pages)
    got = _run(torch, ctx, new, table, free, count, page, tokens, pages, in_place)
    assert got == tuple(want)
    assert want[-1] == 0


@pytest.mark.parametrize("short", [1, 5, 1000])
def test_plan_without_enough_pages(short):
    """Requests are served in order until the stack is empty; those that need no page go on."""
    torch = torch_cuda()
    ctx, new, table, free, count, tokens, pages = _case(11, 60, 16, 100, 30, short=short)
    want = A.plan(ctx, new, table, free, count, 16, tokens, pages)
    assert want[-1] == A.EXHAUSTED and 0 in want[2]
    assert _run(torch, ctx, new, table, free, count, 16, tokens, pages) == tuple(want)


def test_plan_refuses_bad_lengths_pages_and_rows_one_by_one():
    torch = torch_cuda()
    ctx, new, table, free, count, tokens, pages = _case(12, 12, 16, 100, 30)
    ctx, new = ctx.copy(), new.copy()
    ctx[1] = -5
    new[3] = -2
    ctx[5] = 16 * table.shape[1]          # no room behind it
    new[5] = 4
    ctx[6], new[6] = 2**31 - 1, 2**31 - 1  # sums pass 32 bits
    table[8, 0], ctx[8], new[8] = pages + 3, 10, 3   # its page is out of range
    free[count - 1] = -4                    # the first page handed out is none
    want = A.plan(ctx, new, table, free, count, 16, tokens, pages)
    assert want[-1] == A.INVALID
    assert _run(torch, ctx, new, table, free, count, 16, tokens, pages) == tuple(want)
    # a count out of range, and no positions wanted
    ctx, new, table, free, count, tokens, pages = _case(13, 4, 16, 100, 30)
    for bad in (-1, pages + 1):
        if bad > 0:
            free[:] = np.arange(pages)
        want = A.plan(ctx, new, table, free, bad, 16, tokens, pages)
        got = _run(torch, ctx, new, table, free, bad, 16, tokens, pages, positions=False)
        assert got == tuple(want[:3]) + (None,) + tuple(want[4:])


@pytest.mark.parametrize("seed,seqs,page,ctx_hi", [(0, 1, 16, 40), (1, 50, 16, 500),
                                                   (2, 300, 64, 3000), (3, 4096, 16, 30)])
def test_release_matches_the_reference(seed, seqs, page, ctx_hi):
    torch = torch_cuda()
    ctx, _, table, free, count, _, pages = _case(seed, seqs, page, ctx_hi, 1)
    rng = np.random.default_rng(seed + 100)
    flags = rng.integers(0, 2, seqs)
    if seqs > 10:
        table[3, 0] = -1 if ctx[3] else table[3, 0]  # a row that cannot be given back
        flags[3] = 1
    want = A.release(ctx, flags, table, free, count, page, pages)
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    t, f, c = up(table), up(free), up([count])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_release(handle(), page, seqs, up(ctx), up(flags), t, table.shape[1], pages, f, c,
                       status)
    torch.cuda.synchronize()
    got = (t.cpu().tolist(), f.cpu().tolist(), int(c.item()), int(status.item()))
    assert got == tuple(want)


def test_release_never_overfills_the_stack():
    torch = torch_cuda()
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    # 6 pages; 3 are free already, yet rows of 2, 2 and 1 pages claim to be given back
    table, free = np.array([[0, 1], [2, 3], [4, -1]]), np.array([5, 0, 1, -7, -7, -7])
    want = A.release([20, 32, 16], [1, 1, 1], table, free, 3, 16, 6)
    t, f, c = up(table), up(free), up([3])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_release(handle(), 16, 3, up([20, 32, 16]), up([1, 1, 1]), t, 2, 6, f, c, status)
    torch.cuda.synchronize()
    assert (t.cpu().tolist(), f.cpu().tolist(), int(c.item()), int(status.item())) == tuple(want)
    assert int(status.item()) == A.INVALID and int(c.item()) == 5


def test_pages_go_round():
    """Plan and release in turns: no page is ever owned twice, and all come back."""
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    seqs, page, width, pages = 24, 16, 20, 300
    ctx = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.empty(seqs + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(2000, dtype=torch.int64, device="cuda")
    for _ in range(12):
        new = torch.from_numpy(rng.integers(0, 25, seqs).astype(np.int32)).cuda()
        kv = torch.empty_like(ctx)
        gdn.gdn_kv_plan(handle(), page, seqs, 2000, ctx, new, table, width, pages, free, count,
                        count, cu, kv, None, slots, status)
        gone = torch.from_numpy((rng.random(seqs) < 0.2).astype(np.int32)).cuda()
        gdn.gdn_kv_release(handle(), page, seqs, kv, gone, table, width, pages, free, count,
                           status)
        ctx = torch.where(gone > 0, 0, kv).int()
        owned = table[table >= 0].cpu().tolist()
        left = free[:int(count.item())].cpu().tolist()
        assert sorted(owned + left) == list(range(pages))
    assert int(status.item()) == 0
