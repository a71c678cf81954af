"""One prompt of the longest context that the linear layers serve, 262,144 tokens, beside a
decoding request behind it; sampled rows against fp64."""
import math

import pytest

from packed_linear_attention_gb300 import gdn

from gpu_util import handle, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,page", [(16, 2, 256, 64), (8, 2, 128, 128)])
def test_the_longest_prompt(hq, hkv, dim, page):
    torch = torch_cuda()
    n, group = 262144, hq // hkv
    kv = [n, 200001]
    tokens, pages, scale = n + 1, n // page, dim ** -0.5
    g = torch.Generator(device="cuda").manual_seed(11)
    up = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    codes = []
    for _ in range(2):
        x = torch.randint(0, 256, (pages, hkv, page, dim), dtype=torch.uint8, device="cuda",
                          generator=g)
        codes.append(torch.where((x & 127) == 127, x - 1, x))
    scales = [torch.exp2(torch.randint(-9, -6, (pages, hkv), device="cuda", generator=g).float())
              for _ in range(2)]
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.stack([order, order]).contiguous()  # the second request shares the first's pages
    q = torch.randn(tokens, hq, dim, device="cuda", generator=g).bfloat16()
    o = torch.empty_like(q)
    lse = torch.empty(tokens, hq, device="cuda")
    cache = gdn.make_kv_cache(*codes, *scales)
    cfg = gdn.make_attn_config(hq, scale=scale)
    size = gdn.gdn_attn_workspace_size(cfg, cache, 2, tokens, n, n)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    row = hq * dim
    gdn.gdn_attn_paged(handle(), cfg, cache, 2, tokens, n, n, up([0, n, n + 1]), up(kv), table,
                       pages, q, row, o, row, lse, work, size, status)
    torch.cuda.synchronize()
    assert status.item() == gdn.GDN_OK
    # row -> tokens it sees
    rows = {r: r + 1 for r in (0, 1, 63, 64, 15, 4097, 65535, 65536, 131073, 200000, 262079, n - 1)}
    rows[n] = kv[1]
    values = lambda x: x.view(torch.float8_e4m3fn).double()  # noqa: E731
    for h in range(hkv):
        k, v = ((values(c[order.long(), h]) * s[order.long(), h].double()[:, None, None])
                .reshape(-1, dim) for c, s in zip(codes, scales))
        heads = slice(h * group, (h + 1) * group)
        for r, see in rows.items():
            qr = q[r, heads].double()
            s = scale * (qr @ k[:see].T)
            p = (s - s.amax(1, keepdim=True)).exp()
            total = p.sum(1, keepdim=True)
            want, mean = p @ v[:see] / total, p @ v[:see].abs() / total
            # as the small cases' bound: scores of fp32 sums and 2^x, weights of 11 bits or 2^-31
            # of the largest, sums in fp32, the output's rounding
            size_ = scale * (qr.abs() @ k[:see].abs().T).amax(1, keepdim=True)
            prob = 2 * (dim + 8) * 2.0 ** -24 * size_ + 2.0 ** -21
            sums = (math.sqrt(see) + 64) * 2.0 ** -24 * 8
            tiny = see * 2.0 ** -31 * v[:see].abs().max() / total
            bound = want.abs() * 2.0 ** -8 + mean * (2.0 ** -11 + 2 * prob + 2 * sums) + tiny
            assert ((o[r, heads].double() - want).abs() <= bound).all(), r
            exact = (s.amax(1, keepdim=True) + total.log())[:, 0]
            err = (lse[r, heads].double() - exact).abs()
            assert (err <= prob[:, 0] + sums + exact.abs() * 2.0 ** -22).all(), r
