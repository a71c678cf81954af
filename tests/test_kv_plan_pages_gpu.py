"""Pages out of range, in a request's table row or on the free stack: the request that would use
one is refused whole (no page taken, no length, no slot), so that what the next step and the
release are told is what the cache holds."""
import numpy as np
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu

PAGE = 16


class World:
    def __init__(self, torch, rows, stack, num_pages, width=6):
        """rows: the requests' pages in order; stack: the free pages, the top last."""
        self.torch, self.num_pages, self.width, self.n = torch, num_pages, width, len(rows)
        table = np.full((self.n, width), -1, np.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = r
        up = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table = torch.from_numpy(table).cuda()
        self.free = up(list(stack) + [-9] * (num_pages - len(stack)))
        self.count = up([len(stack)])
        self.cu, self.kv = up([-9] * (self.n + 1)), up([-9] * self.n)
        self.status = up([0])
        self.up = up

    def plan(self, ctx, new, tokens=None):
        tokens = sum(new) if tokens is None else tokens
        pos = self.up([-9] * tokens)
        slots = pos.long()
        gdn.gdn_kv_plan(handle(), PAGE, self.n, tokens, self.up(ctx), self.up(new), self.table,
                        self.width, self.num_pages, self.free, self.count, self.count, self.cu,
                        self.kv, pos, slots, self.status)
        self.torch.cuda.synchronize()
        return self.kv.tolist(), slots.tolist(), pos.tolist()

    def release(self, flags):
        gdn.gdn_kv_release(handle(), PAGE, self.n, self.kv, self.up(flags), self.table,
                           self.width, self.num_pages, self.free, self.count, self.status)
        self.torch.cuda.synchronize()

    def owned(self):
        return [[p for p in r if p >= 0] for r in self.table.tolist()]

    def left(self):
        return self.free.tolist()[:self.count.item()]


def test_a_bad_page_where_new_tokens_go():
    """Request 1's half-filled page is out of range: it takes none of the two pages it asks for.
    Request 3 has a bad page too, but appends behind it."""
    for bad in (-1, 40, 2**31 - 1, -2**31):
        w = World(torch_cuda(), [[5], [6, bad], [7, 8], [bad, 9]], [0, 1, 2, 3, 4], 40)
        before = w.table.clone()
        kv, slots, pos = w.plan([10, 20, 32, 30], [3, 40, 1, 2])
        assert w.status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
        assert kv == [13, 0, 33, 32] and w.cu.tolist() == [0, 3, 43, 44, 46]
        assert slots == [90, 91, 92] + [-1] * 40 + [4 * 16, 9 * 16 + 14, 9 * 16 + 15]
        assert pos == [10, 11, 12] + [0] * 40 + [32, 30, 31]
        assert w.left() == [0, 1, 2, 3]
        before[2, 2] = 4
        assert (w.table == before).all()


def test_no_new_token_needs_no_page():
    w = World(torch_cuda(), [[-1], [3]], [0, 1], 8)
    kv, slots, _ = w.plan([10, 16], [0, 0], tokens=2)
    assert kv == [10, 16] and slots == [-1, -1] and w.status.item() == 0 and w.left() == [0, 1]


@pytest.mark.parametrize("bad", [-1, 60, -2**31])
def test_a_bad_page_on_the_stack(bad):
    """The third page from the top is out of range. The requests are served until one needs it;
    from there on those that need a page are refused, those that need none are not."""
    w = World(torch_cuda(), [[10], [11], [12], [13], [14]], [0, 1, 2, bad, 3, 4], 60)
    before = w.table.clone()
    kv, slots, _ = w.plan([16, 10, 16, 16, 5], [17, 2, 5, 1, 3])
    assert w.status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
    assert kv == [33, 12, 0, 0, 8]
    assert slots == [64 + i for i in range(16)] + [48, 11 * 16 + 10, 11 * 16 + 11] + [-1] * 6 + \
        [14 * 16 + 5, 14 * 16 + 6, 14 * 16 + 7]
    assert w.left() == [0, 1, 2, bad]
    before[0, 1], before[0, 2] = 4, 3
    assert (w.table == before).all()
    # what was served can be given back
    w.release([1, 1, 1, 1, 1])
    assert w.left() == [0, 1, 2, bad, 10, 4, 3, 11, 14]
    assert w.owned() == [[], [], [12], [13], []]


def test_a_bad_page_deep_in_the_stack():
    """Far more pages than threads: 600 requests of ten pages, one page that some of them would
    get is none. Where the requests end in front of it, nothing is wrong."""
    torch = torch_cuda()
    n, stack = 600, 6000
    for served in (150, 415, 416, 590):
        empty = [[] for _ in range(n)]
        w = World(torch, empty, range(stack), stack + 100, width=12)
        at = stack - 10 * served - 3  # the third page of the first request that is not served
        w.free[at] = -1
        kv, slots, _ = w.plan([0] * n, [160] * n)
        assert kv == [160] * served + [0] * (n - served)
        assert w.status.item() == gdn.GDN_ERR_INVALID_ARGUMENT
        assert (np.array(slots[served * 160:]) == -1).all() and min(slots[:served * 160]) >= 0
        left = list(range(stack - 10 * served))
        left[at] = -1
        assert w.left() == left
        assert sorted(sum(w.owned(), [])) == list(range(stack - 10 * served, stack))
        w = World(torch, empty, range(stack), stack + 100, width=12)
        w.free[stack - 10 * served - 1] = -1
        kv, _, _ = w.plan([0] * n, [160] * served + [0] * (n - served))
        assert kv == [160] * served + [0] * (n - served) and w.status.item() == 0


def test_stack_ends_before_the_bad_page():
    """The stack runs out: that is what is reported."""
    w = World(torch_cuda(), [[], []], [0, 99, 1], 8)
    kv, _, _ = w.plan([0, 0], [16, 64])
    assert kv == [16, 0] and w.status.item() == gdn.GDN_ERR_POOL_EXHAUSTED and w.left() == [0, 99]
