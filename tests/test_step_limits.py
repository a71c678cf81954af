"""The calls around the recurrent layers at the ends of what they take, on the host: no call gets as
far as a kernel (validation comes before any CUDA call, and a NULL handle is the last thing checked)."""
import random

import pytest

from packed_linear_attention_gb300 import build, gdn

from test_step_abi import (INVALID, P, SMALL, UNSUPPORTED, conv_config, norm_config, requests, ssm_config,
                           ssm_rows)

TOP = (1 << 31) - 4096
FAR = [(1 << 50) * (i + 1) for i in range(8)]  # room for 2^31 rows each


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return gdn.load()


def conv(tokens):
    return gdn.gdn_conv_packed(None, conv_config(), requests(num_tokens=tokens), FAR[0], 96, FAR[1], 96,
                               P(2), P(3), P(4), raise_on_error=False)


def ssm(tokens):
    rows = ssm_rows(x=FAR[0], delta=FAR[1], b=FAR[2], c=FAR[3], z=FAR[4], y=FAR[5])
    return gdn.gdn_ssm_packed(None, ssm_config(), requests(num_tokens=tokens), rows, P(6), P(7), FAR[6],
                              1 << 40, P(9), raise_on_error=False)


@pytest.mark.parametrize("call", [conv, ssm])
def test_rows_of_a_packed_call(call):
    """The kernels count rows in 32 bits, a block past the last one too."""
    assert call(TOP - 1) == INVALID  # the NULL handle
    assert call(TOP) == UNSUPPORTED and call((1 << 31) - 1) == UNSUPPORTED


def test_norm_of_no_rows():
    """Empty tensors have no address."""
    odd = norm_config(num_heads=4, dim=96)  # refused after everything else
    call = lambda n, **kw: gdn.gdn_rms_norm(None, odd, n, None, 384, raise_on_error=False, **kw)  # noqa: E731
    assert call(0) == UNSUPPORTED and call(1) == INVALID and call(-1) == INVALID
    for kw in (dict(sum=P(0), sum_stride=384), dict(codes=P(1), codes_stride=384), dict(scales=P(2))):
        assert call(0, **kw) == UNSUPPORTED and call(1, **kw) == INVALID, kw


@pytest.mark.gpu
def test_norm_of_empty_tensors():
    from gpu_util import handle, torch_cuda
    torch = torch_cuda()
    empty = lambda dtype: torch.empty(0, 256, dtype=dtype, device="cuda")  # noqa: E731
    x = empty(torch.bfloat16)
    cfg = gdn.make_norm_config(256, torch.ones(256, device="cuda"))
    gdn.gdn_rms_norm(handle(), cfg, 0, x, 256, x, 256, x, 256, y=x, y_stride=256)
    gdn.gdn_rms_norm(handle(), cfg, 0, x, 256, codes=empty(torch.uint8), codes_stride=256,
                     scales=torch.empty(0, 1, device="cuda"))
    torch.cuda.synchronize()


def scan_takes(cfg, seqs, tokens, max_len, size):
    ch, gn = cfg.channels, cfg.num_groups * cfg.state_dim
    rows = ssm_rows(x=FAR[0], delta=FAR[1], b=FAR[2], c=FAR[3], z=FAR[4], y=FAR[5], x_stride=ch,
                    delta_stride=ch, z_stride=ch, y_stride=ch, b_stride=gn, c_stride=gn)
    req = requests(num_seqs=seqs, num_tokens=tokens, max_len=max_len, num_slots=seqs, ckpt_cu=None)
    st = gdn.gdn_ssm_packed(None, cfg, req, rows, FAR[6], None, FAR[7], size, None, raise_on_error=False)
    assert st in (INVALID, SMALL)  # the NULL handle, or the workspace
    return st == INVALID


def test_a_workspace_for_the_largest_scan_serves_every_smaller_one():
    """Fewer and shorter requests may be cut where many are not."""
    rng = random.Random(3)
    far = lambda top: int(2.0 ** rng.uniform(0, top))  # noqa: E731
    for _ in range(300):
        cfg = ssm_config(channels=8 * far(11), num_groups=1, state_dim=rng.choice([3, 8, 16, 64, 128]))
        seqs, max_len = far(7), far(16)
        tokens = min((1 << 31) - 5000, int(seqs * max_len * rng.uniform(0.3, 1.2)) + 1)
        size = gdn.gdn_ssm_workspace_size(cfg, requests(num_seqs=seqs, num_tokens=tokens, max_len=max_len,
                                                        num_slots=seqs))
        assert size % 256 == 0
        for _ in range(20):
            n, m = rng.randint(1, seqs), rng.randint(1, max_len)
            t = rng.randint(1, tokens)
            assert scan_takes(cfg, n, t, m, size), (cfg.channels, cfg.state_dim, n, t, m)
        for n in (1, 2, 3, seqs):  # as many rows as such requests have
            n = min(n, seqs)
            assert scan_takes(cfg, n, min(tokens, n * max_len), max_len, size)
            assert scan_takes(cfg, n, tokens, max_len, size)


def test_one_prompt_beside_a_wave():
    cfg = ssm_config(channels=4096, num_groups=1)
    wave = dict(num_seqs=32, num_slots=32, num_tokens=32768, max_len=1024)
    size = gdn.gdn_ssm_workspace_size(cfg, requests(**wave))
    for n in (1, 2, 3, 8, 32):
        assert scan_takes(cfg, n, n * 1024, 1024, size) and scan_takes(cfg, n, 32768, 1024, size)
    assert not scan_takes(cfg, 1, 1024, 1024, 256)  # cut: it needs room
    assert size < 1 << 24
