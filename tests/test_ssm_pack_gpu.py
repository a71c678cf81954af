"""The selective scan: what a request's results and a call's workspace owe to the calls around them."""
import numpy as np
import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda
from step_util import empty_rows, i32, num, up
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
