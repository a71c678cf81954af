"""The serving example when its pages run out: a request that gets none keeps its context, its
pages and its linear states, goes on when there are pages again, and no page is lost."""
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from test_serve_example_gpu import example

pytestmark = pytest.mark.gpu


def _server(m, torch, pages, slots=2, layers="LF"):
    torch.manual_seed(4)
    return m.Server(slots=slots, num_pages=pages, max_tokens=512, layers=layers)


def _pool(server):
    """Every page once: owned by a table row or free."""
    owned = [p for r in server.pages.table.tolist() for p in r if p >= 0]
    return sorted(owned + server.pages.free.tolist()[:server.pages.count.item()])


def test_a_running_request_that_gets_no_page():
    torch = torch_cuda()
    handle()
    m = example()
    a, b = (torch.randn(n, m.HIDDEN, device="cuda").bfloat16() for n in (64, 60))
    row = torch.randn(1, m.HIDDEN, device="cuda").bfloat16()
    tight, ample = _server(m, torch, 2), _server(m, torch, 8)
    for s in (tight, ample):
        s.step({0: a, 1: b})
    state = tight.layers[0].pool[0].clone()
    table = tight.pages.table.clone()
    out = tight.step({0: row, 1: row})  # request 0 needs a second page
    assert sorted(out) == [1]
    assert tight.pages.ctx.tolist() == [64, 61]
    assert torch.equal(tight.pages.table, table) and torch.equal(tight.layers[0].pool[0], state)
    with pytest.raises(gdn.GdnError) as e:
        tight.check()
    assert e.value.status == gdn.GDN_ERR_POOL_EXHAUSTED
    assert _pool(tight) == [0, 1]
    tight.end([1])
    got = tight.step({0: row})[0]
    tight.check()
    want = ample.step({0: row})[0]
    assert tight.pages.ctx.tolist() == [65, 0] and _pool(tight) == [0, 1]
    # the same step in another pack: bf16 rows of a few units, through two layers
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -4
    tight.end([0])
    assert sorted(tight.pages.free.tolist()) == [0, 1] and tight.pages.count.item() == 2
    for s in (tight, ample):
        s.close()


def test_prompts_wait_for_pages():
    """Pages for two of the five requests at a time: the others wait, all are served."""
    torch = torch_cuda()
    handle()
    m = example()
    lengths = (70, 1, 200, 130, 63)
    prompts = [torch.randn(n, m.HIDDEN, device="cuda").bfloat16() for n in lengths]
    results = []
    for pages in (6, 24):
        server = _server(m, torch, pages, slots=3)
        results.append(m.serve(server, prompts, 5))
        assert sorted(server.pages.free.tolist()) == list(range(pages))
        assert server.pages.count.item() == pages and (server.pages.table == -1).all()
        server.close()
    for x, y in zip(*results):
        assert (x.float() - y.float()).abs().max() <= 2.0 ** -4 * 6  # six steps


def test_a_prompt_that_never_fits_is_reported():
    torch = torch_cuda()
    handle()
    m = example()
    server = _server(m, torch, 2)
    with pytest.raises(gdn.GdnError) as e:
        m.serve(server, [torch.randn(200, m.HIDDEN, device="cuda").bfloat16()], 3)
    assert e.value.status == gdn.GDN_ERR_POOL_EXHAUSTED
    with pytest.raises(gdn.GdnError) as e:
        server.step({0: torch.randn(513, m.HIDDEN, device="cuda").bfloat16()})
    assert e.value.status == gdn.GDN_ERR_INVALID_ARGUMENT
    assert _pool(server) == [0, 1]
    server.close()
